// The work list of lf_attn_paged_chunk, shared by its kernels (private to the library).
//
// An item is (sequence, KV head, row tile): `toks` consecutive new tokens with all
// query heads of the KV head, row = token * group + head of the group.  It reads
// the keys that any of its tokens sees in tiles of KT positions, cut at
// multiples of KT of the sequence's positions, so a tile lies in whole pages or
// a page in whole tiles.  The tiles of all items, in the order sequence, head, row
// tile, key, form one list that is cut into equal contiguous shares, one per CTA.
// Everything is worked out on the device from starts and lens.
#pragma once

#include "lf_paged_attn.h"

namespace lf {

struct ChunkArgs {
    PagedView kv;
    const void *q;
    void *out;
    float *lse;
    long long ld_q, ld_out;
    int n_q, group;
    const int32_t *starts, *lens;
    int n_tokens, max_len, window;  // window 0: none
    float scale_log2;
    bool tc;                    // the tensor cores' kernel
    int toks, slot_rows;        // tokens of a row tile; rows of a partial in the workspace: at least toks * group
    int grid;                   // CTAs that share the list
    // A CTA works on at most two items that it does not see whole: one that an
    // earlier CTA began (partial 2 c), and one that it begins and does not
    // end (partial 2 c + 1).  joins[c]: that last item, where there is one.
    struct Join {
        int row0, rows, head, parts;  // first row of q (token), rows of the item, KV head, CTAs of the item (0: none)
    };
    Join *joins;
    float *part_o;     // [2 grid][slot_rows][head_dim], unnormalised
    float2 *part_ml;   // [2 grid][slot_rows] (max in the log2 domain, sum)
    uint32_t *err;
};

// The new tokens of a sequence.
struct Chunk {
    int row0, c;  // first row, how many
    int base;     // position of the first (below 0: a chunk longer than the sequence)
    bool bad;
};
__device__ __forceinline__ Chunk chunk_of(const ChunkArgs &a, int b) {
    Chunk k;
    const int s0 = a.starts[b], s1 = a.starts[b + 1];
    int len = a.lens[b];
    k.bad = len < 0 || len > a.max_len;
    if (k.bad) len = 0;
    const bool in = s0 >= 0 && s0 <= s1 && s1 <= a.n_tokens;
    k.bad |= !in;
    k.row0 = in ? s0 : 0;
    k.c = in ? s1 - s0 : 0;
    k.base = len - k.c;
    return k;
}

// sum_{i < n} floor((a i + b) / M) for a, b >= 0, M a power of two, a n + b < 2^32, by
// the Euclidean reduction of the lattice points under a line (each step swaps a and m).
template <unsigned M>
__host__ __device__ inline long long floor_sum(unsigned n, unsigned a, unsigned b) {
    long long sum = 0;
    unsigned m = M;
    bool power = true;  // (the first step divides by M: shifts)
    while (n) {
        const unsigned qa = power ? a / M : a / m, qb = power ? b / M : b / m;
        sum += (long long)n * (n - 1) / 2 * qa + (long long)n * qb;
        a -= qa * m;
        b -= qb * m;
        if (a == 0) break;  // (what is left lies below one step)
        const unsigned y = a * n + b;
        n = power ? y / M : y / m;
        b = y - n * m;
        const unsigned t = m;
        m = a;
        a = t;
        power = false;
    }
    return sum;
}

// Keys [lo, hi) that the row tile from token `tok` on sees.
struct Keys {
    int lo, hi;
};
__host__ __device__ inline Keys keys_of(int base, int c, int window, int toks, int tok) {
    const int last = base + (c - tok < toks ? c : tok + toks);
    const long long first = window > 0 ? (long long)base + tok - window + 1 : 0;
    Keys k;
    k.hi = last > 0 ? last : 0;
    k.lo = first > 0 ? (int)first : 0;
    return k;
}
// Key tiles of a row tile: at least one (a row tile that sees nothing writes zeros).
template <int KT>
__host__ __device__ inline int key_tiles(const Keys &k) {
    return k.hi <= 0 ? 1 : (int)((unsigned)(k.hi + KT - 1) / KT - (unsigned)k.lo / KT);
}
// Key tiles of the first n row tiles of a chunk, n at most ceil(c / toks).
template <int KT>
__host__ __device__ inline long long tiles_before(int base, int c, int window, int toks, int n) {
    if (n <= 0) return 0;
    const int full = c / toks < n ? c / toks : n;  // row tiles of `toks` tokens; one more is shorter
    // those that end before position 1 have one tile without keys
    int none = base < 0 ? -base / toks : 0;
    if (none > full) none = full;
    long long sum = none + floor_sum<KT>((unsigned)(full - none), (unsigned)toks,
                                         full > none ? (unsigned)(base + (none + 1) * toks + KT - 1) : 0u);
    if (n > full) sum += base + c <= 0 ? 1 : (unsigned)(base + c + KT - 1) / KT;
    if (window > 0) {  // less the tiles before each one's first key; none before token window - 1 - base
        const long long from = (long long)window - 1 - base;
        const long long z = from < 0 ? 0 : from / toks + 1;
        if (z < n) {
            const int f = (int)z;
            sum -= floor_sum<KT>((unsigned)(n - f), (unsigned)toks, (unsigned)(base + f * toks - window + 1));
        }
    }
    return sum;
}

// The list as one CTA walks it.
struct ChunkWork {
    int b, h, r, row_tiles;  // sequence, KV head, row tile of it, row tiles of the sequence
    Chunk ch;
    int tok, toks;           // first token of the row tile, tokens
    Keys k;
    int kt0, tile, tiles;    // first key tile (key / KT); this tile, and how many the item has
    template <int KT>
    __device__ void set(const ChunkArgs &a) {
        tok = r * a.toks;
        toks = min(a.toks, ch.c - tok);
        k = keys_of(ch.base, ch.c, a.window, a.toks, tok);
        kt0 = (unsigned)k.lo / KT;
        tiles = key_tiles<KT>(k);
    }
};

// Fills cum[b] = key tiles per KV head of the sequences before b (cum[n_seqs]: of
// all); a whole block calls it.  Returns the list's length.
template <int KT>
__device__ __forceinline__ int chunk_plan(const ChunkArgs &a, int *cum) {
    const int n = a.kv.n_seqs, lane = threadIdx.x & 31;
    int at = 0;
    for (int b0 = 0; b0 < n; b0 += 32) {  // (every warp for itself; the first fills the table)
        const int b = b0 + lane;
        int t = 0;
        if (b < n) {
            const Chunk k = chunk_of(a, b);
            t = (int)tiles_before<KT>(k.base, k.c, a.window, a.toks, (k.c + a.toks - 1) / a.toks);
            if (k.bad && blockIdx.x == 0 && threadIdx.x < 32) atomicExch(a.err, 1u);
        }
        int inc = t;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += y;
        }
        if (threadIdx.x < 32 && b < n) cum[b] = at + inc - t;
        at += __shfl_sync(0xffffffffu, inc, 31);
    }
    if (threadIdx.x == 0) cum[n] = at;
    __syncthreads();
    return at * a.kv.n_kv;
}

// The place of tile u; whole warps call it together.
template <int KT>
__device__ __forceinline__ ChunkWork chunk_place(const ChunkArgs &a, const int *cum, int u) {
    ChunkWork w;
    const int lane = threadIdx.x & 31;
    int lo = 0, hi = a.kv.n_seqs;  // the sequence with n_kv cum[b] <= u < n_kv cum[b + 1]
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (a.kv.n_kv * cum[mid] <= u)
            lo = mid;
        else
            hi = mid;
    }
    w.b = lo;
    const int per_head = cum[lo + 1] - cum[lo];
    u -= a.kv.n_kv * cum[lo];
    w.h = quotient(u, per_head);
    u -= w.h * per_head;
    w.ch = chunk_of(a, lo);
    w.row_tiles = (w.ch.c + a.toks - 1) / a.toks;
    // the row tile with before(r) <= u < before(r + 1): 32 places at a time
    lo = 0, hi = w.row_tiles;
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32, x = lo + lane * step;
        const bool in = x < hi && tiles_before<KT>(w.ch.base, w.ch.c, a.window, a.toks, x) <= u;
        const int last = 31 - __clz(__ballot_sync(0xffffffffu, in));  // (lane 0 always is)
        lo += last * step;
        hi = min(hi, lo + step);
    }
    w.r = lo;
    w.set<KT>(a);
    w.tile = u - (int)tiles_before<KT>(w.ch.base, w.ch.c, a.window, a.toks, lo);
    return w;
}

// The next tile of the list; true if it begins another item.
template <int KT>
__device__ __forceinline__ bool chunk_advance(const ChunkArgs &a, const int *cum, ChunkWork &w) {
    if (++w.tile < w.tiles) return false;
    w.tile = 0;
    if (++w.r == w.row_tiles) {
        w.r = 0;
        if (++w.h == a.kv.n_kv) {
            w.h = 0;
            do {
                ++w.b;
            } while (w.b < a.kv.n_seqs - 1 && cum[w.b + 1] == cum[w.b]);
            w.ch = chunk_of(a, w.b);
            w.row_tiles = (w.ch.c + a.toks - 1) / a.toks;
        }
    }
    w.set<KT>(a);
    return true;
}

// What CTA c leaves for the join: its last item, if it begins it and does not end
// it (its tiles from `tile` on lie behind this CTA's share, which ends at u1).
__device__ __forceinline__ ChunkArgs::Join chunk_join(const ChunkArgs &a, const ChunkWork &w, const Shares &sh, int c,
                                                      int u1, int next_tile, bool begun_here) {
    ChunkArgs::Join j = {0, 0, 0, 0};
    if (begun_here && next_tile < w.tiles) {
        const int left = w.tiles - next_tile;  // tiles of the item in the CTAs behind
        int parts = 1;
        for (int at = u1, k = c + 1; at < u1 + left; ++k, ++parts) at = sh.begin(k + 1);
        j.row0 = w.ch.row0 + w.tok;
        j.rows = w.toks * a.group;
        j.head = w.h;
        j.parts = parts;
    }
    return j;
}

// The list's kernel on the 5th-generation tensor cores (lf_paged_chunk_tc.cu): head_dim 64 and 128,
// toks even, slot_rows = kTcRows.
lf_status paged_chunk_tc(const ChunkArgs &a, int dtype, cudaStream_t st);

}  // namespace lf
