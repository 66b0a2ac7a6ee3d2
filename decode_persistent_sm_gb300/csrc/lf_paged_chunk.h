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
#ifdef LF_DEBUG
    int lose_cta, lose_warp, lose_wait;  // tensor cores' kernel: this warp of this CTA (-1: of each) gives up in its lose_wait-th wait (0: none)
#endif
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
// Row tiles of a chunk of c tokens.
__device__ __forceinline__ int row_tiles_of(int c, int toks) { return c <= toks ? (c > 0) : quotient(c + toks - 1, toks); }
// Key tiles of row tile r.
template <int KT>
__device__ __forceinline__ int key_tiles_of(const ChunkArgs &a, const Chunk &k, int r) {
    return key_tiles<KT>(keys_of(k.base, k.c, a.window, a.toks, r * a.toks));
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
// all); a whole block calls it.  Returns the list's length.  A lane adds up the few
// row tiles of its sequence, the warp together those of a long chunk.  Starts that
// decrease (bad where they do) can claim rows more than once: beyond n_tokens in all,
// which is what the host bounds the list by, there is no list.
template <int KT>
__device__ __forceinline__ int chunk_plan(const ChunkArgs &a, int *cum) {
    constexpr int kFew = 4;
    const int n = a.kv.n_seqs, lane = threadIdx.x & 31;
    long long claimed = 0;
    int at = 0;
    for (int b0 = 0; b0 < n; b0 += 32) {  // (every warp for itself; the first fills the table)
        const int b = b0 + lane;
        Chunk k = {0, 0, 0, false};
        if (b < n) {
            k = chunk_of(a, b);
            if (k.bad && blockIdx.x == 0 && threadIdx.x < 32) atomicExch(a.err, 1u);
        }
        claimed += __reduce_add_sync(0xffffffffu, (unsigned)k.c);  // (32 times 2^26 at most)
        if (claimed > a.n_tokens) break;
        const int rt = row_tiles_of(k.c, a.toks);
        int t = 0;
        for (int r = 0; r < min(rt, kFew); ++r) t += key_tiles_of<KT>(a, k, r);
        for (unsigned left = __ballot_sync(0xffffffffu, rt > kFew); left; left &= left - 1) {
            const int who = __ffs(left) - 1, rts = __shfl_sync(0xffffffffu, rt, who);
            Chunk y;
            y.base = __shfl_sync(0xffffffffu, k.base, who);
            y.c = __shfl_sync(0xffffffffu, k.c, who);
            int sum = 0;
            for (int r = kFew + lane; r < rts; r += 32) sum += key_tiles_of<KT>(a, y, r);
            sum = __reduce_add_sync(0xffffffffu, sum);
            if (lane == who) t += sum;
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
    if (claimed > a.n_tokens) at = 0;
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
    w.row_tiles = row_tiles_of(w.ch.c, a.toks);
    w.r = 0;
    w.tile = u;
    for (int r0 = 0; w.row_tiles > 1 && r0 < w.row_tiles; r0 += 32) {  // 32 row tiles at a time: how many end at or before u
        const int t = r0 + lane < w.row_tiles ? key_tiles_of<KT>(a, w.ch, r0 + lane) : 0;
        int inc = t;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += y;
        }
        const int ended = __popc(__ballot_sync(0xffffffffu, r0 + lane < w.row_tiles && inc <= u));
        if (ended < 32) {
            w.r = r0 + ended;
            w.tile = u - __shfl_sync(0xffffffffu, inc - t, ended);
            break;
        }
        u -= __shfl_sync(0xffffffffu, inc, 31);
    }
    w.set<KT>(a);
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
            w.row_tiles = row_tiles_of(w.ch.c, a.toks);
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

// Without the list: item `id` (row tile id / n_kv of all sequences, KV head id % n_kv); false if there are fewer.
// Whole warps call it together.
template <int KT>
__device__ __forceinline__ bool chunk_item(const ChunkArgs &a, int id, ChunkWork &w) {
    const int lane = threadIdx.x & 31, g = quotient(id, a.kv.n_kv);
    w.h = id - g * a.kv.n_kv;
    w.b = -1;
    for (int b0 = 0, at = 0; b0 < a.kv.n_seqs; b0 += 32) {
        const int b = b0 + lane;
        Chunk k = {0, 0, 0, false};
        if (b < a.kv.n_seqs) k = chunk_of(a, b);
        if (k.bad && blockIdx.x == 0 && threadIdx.x < 32) atomicExch(a.err, 1u);
        const int rt = row_tiles_of(k.c, a.toks);
        int inc = rt;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += y;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, at + inc > g);
        if (hit && w.b < 0) {
            const int who = __ffs(hit) - 1;
            w.b = b0 + who;
            w.r = g - at - __shfl_sync(0xffffffffu, inc - rt, who);
            w.ch.row0 = __shfl_sync(0xffffffffu, k.row0, who);
            w.ch.c = __shfl_sync(0xffffffffu, k.c, who);
            w.ch.base = __shfl_sync(0xffffffffu, k.base, who);
            if (blockIdx.x > 0) break;
        }
        at += __shfl_sync(0xffffffffu, inc, 31);
    }
    if (w.b < 0) return false;
    w.set<KT>(a);
    return true;
}

// The items that the chunks can have at most, in the list or a cluster to each (a chunk of c tokens has 1 + (c - 1) / toks
// row tiles; clusters without an item leave at once).
inline long long chunk_items(const ChunkArgs &a) {
    const int some = a.n_tokens < a.kv.n_seqs ? a.n_tokens : a.kv.n_seqs;  // sequences with new tokens
    return (long long)a.kv.n_kv * (some + (a.n_tokens - some) / a.toks);
}

// The kernel on the 5th-generation tensor cores (lf_paged_chunk_tc.cu): head_dim 64 and 128, toks even, slot_rows =
// kTcRows.  direct: CTAs to an item, 0 for the list.
lf_status paged_chunk_tc(const ChunkArgs &a, int dtype, int direct, cudaStream_t st);

}  // namespace lf
