// Decode attention over a paged cache for a batch whose sequences share their
// first positions: o = softmax(scale q K^T) V per query head, one query token
// per sequence.
//
// What bounds it is reading K and V: 4 head_dim bytes per (position, KV head)
// against 4 head_dim FLOP per (position, query head).  The common positions
// are therefore read once for all sequences: the rows (sequence, query head)
// of one KV head are the M side of one product with a tile of common keys,
// 64 rows at a time.  Only positions that every sharing sequence sees are
// treated so (from the latest window start to shared_len); what a sequence
// sees besides goes through its own items, so no masked position ever enters
// a product.
//
// Work is cut into tiles of 64 or 128 keys.  An item is (KV head, row tile) of the
// common range or (sequence, KV head) of the own ranges; all tiles of all
// items form one list, cut into equal contiguous shares, one per CTA, so ragged
// lengths and short batches fill the GPU alike.  A CTA walks its share with a
// cp.async ring of tiles that runs on across item borders, and leaves one
// partial (unnormalised o, max, sum) per item it touches: slot item + CTA,
// which is unique because both only grow along the list.  A second kernel,
// launched to overlap the first one's end, joins each row's partials in list
// order.  A call of few keys does without the list: a cluster of up to 8 CTAs
// per (sequence, KV head) reads all that the sequence sees and joins through
// distributed shared memory, in one launch.
//
// One tile: S = Q K^T and O += P V on warp-level MMAs (m16n8k16, fp32
// accumulators), softmax statistics in registers.  The four warps take 16-row
// blocks (rows > 16) and 16-key blocks (what is left), each warp its own
// running maximum; warps that shared rows join in shared memory at the item's
// end.  P is rounded to the cache's type for the second product: both operands of
// an MMA have one type, and a second product with what the rounding leaves would
// double the work.  Its sum is taken before the rounding.  Against 64 bits the
// output's error (mostly its own rounding) grows by 8 to 14 % on the timed cases, from
// 1.66e-3 to 2.31e-3 at the largest in BF16.
//
// Measured (us per call, both launches; in brackets the bytes it cannot do
// without at the copy rate): 8 sequences x 512 common + 40 .. 130 own positions, 32 / 16
// heads of 128: 10.0 (1.5); 16 x 3584 + 100 .. 512: 23.8 (10.4); 24 windowed
// sequences, 24 / 8 heads of 64: 15.1 (2.9); 2 short ones, by the direct kernel:
// 4.7 to 5.2 (6.5 by the list), the time of the call.  Between 2 and 3 us go to working out the list (lengths, then page
// numbers, then the first keys: three trips to L2), as much to the join; in
// between the keys and values stream at 5.7 TB/s.
#include <cooperative_groups.h>

#include <algorithm>
#include <climits>
#include <type_traits>

#include "lf_paged_attn.h"
#include "lf_ptx.cuh"

namespace cg = cooperative_groups;

namespace lf {
namespace {

constexpr int PA_THREADS = 128, PA_ROWS = 64, PA_MAX_SEQS = 1024, PA_MAX_GROUP = 16;
constexpr int PA_CTAS_PER_SM = 2;
// keys per tile: 32 KB of K and V at head_dim 64 and 128 (a 16 KB tile's barriers and softmax statistics cost more than its copy)
__host__ __device__ constexpr int tile_keys(int dim) { return dim == 128 ? 64 : 128; }
constexpr int PA_MERGE_THREADS = 128;
template <typename T>
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void mma<__half>(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    mma_16816(c, a, b0, b1);
}
template <>
__device__ __forceinline__ void mma<__nv_bfloat16>(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// 16 bytes global -> shared, or 16 zero bytes.
__device__ __forceinline__ void cp16_or_zero(uint32_t dst, const void *src, bool valid) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0) : "memory");
}

// Byte offset of 16-byte chunk c of row r of a tile: the chunk index is
// permuted by the row so that the 8 rows of a matrix load lie in 8 different
// 16-byte bank groups.
template <int DH>
__device__ __forceinline__ uint32_t tile_off(int r, int c) {
    return (uint32_t)(r * DH * 2 + ((c ^ (DH >= 64 ? (r & 7) : ((r >> 1) & 3))) << 4));
}

// The place of a tile in the list.
struct Place {
    int item;   // common: h * row_tiles + rt; own: b * n_kv + h
    int tile, tiles;
    bool common;
    int b, h, rt;
    // the item's keys: key k is position first + k, + gap from key gap_at on
    int keys, first, gap_at, gap;
};

// Three stages of 32 KB (six of 16 KB at head_dim 32), so that two CTAs share an
// SM with 128 KB of copies in flight.
template <typename T, int DH>
struct Smem {
    static constexpr int KT = tile_keys(DH);
    static constexpr int TILE = KT * DH * 2;  // bytes of K (or V) of one tile
    static constexpr int STAGES = DH == 32 ? 6 : 3;
    static constexpr int ML = 4 * 16 * 2 * 4;  // max and sum of the rows that the warps join
    static constexpr int Q = PA_MAX_GROUP * DH * 2;  // an own item's query rows, one buffer per stage
    static constexpr int CUM = (PA_MAX_SEQS + 4) * 4;
    static constexpr int BYTES = STAGES * (2 * TILE + Q) + ML + CUM;
    // the join of the warps' rows uses the stage of the item's last tile
    static_assert(4 * 16 * DH * 4 <= 2 * TILE, "the joined rows fit the stage");
    static_assert(PA_MAX_GROUP * DH * 4 <= STAGES * Q, "a cluster's partial fits the query rows' buffers");
};

// 1 / sum, 0 for a row that saw nothing (a NaN stays one).
__device__ __forceinline__ float inverse(float sum) { return sum > 0.f ? 1.f / sum : (sum == 0.f ? 0.f : sum); }

template <typename T, int DH>
class Walker {
  public:
    __device__ Walker(const AttnArgs &args, uint8_t *smem) : a(args), com(args, -1) {
        stage0 = smem;
        q0 = smem + L::STAGES * 2 * L::TILE;
        ml = reinterpret_cast<float2 *>(q0 + L::STAGES * L::Q);
        cum = reinterpret_cast<int *>(q0 + L::STAGES * L::Q + L::ML);
        tid = threadIdx.x;
        warp = tid >> 5;
        lane = tid & 31;
    }

    // The plan from the lengths: the common range and the own tiles before
    // each sequence.  Every warp works it out for itself, so that only the
    // table waits for a barrier; CTA 0 leaves the common range for
    // the join.
    __device__ void plan() {
        const int n = a.kv.n_seqs;
        com = Common(a, __reduce_max_sync(0xffffffffu, latest_start(a, lane)));
        tiles_c = (com.hi - com.lo + a.keys_c - 1) / a.keys_c;
        int at = 0;
        for (int b0 = 0; b0 < n; b0 += 32) {
            const int b = b0 + lane;
            int t = 0;
            if (b < n) {
                t = (own_count(span_of(a, b), com) + KT - 1) / KT;
                if (blockIdx.x == 0 && (a.lens[b] < 0 || a.lens[b] > a.max_len)) atomicExch(a.err, 1u);
            }
            int inc = t;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o) inc += y;
            }
            if (warp == 0 && b < n) cum[b] = at + inc - t;
            at += __shfl_sync(0xffffffffu, inc, 31);
        }
        if (tid == 0) cum[n] = at;
        common_total = a.tc ? 0 : a.kv.n_kv * a.row_tiles * tiles_c;
        total = common_total + a.kv.n_kv * at;
        if (blockIdx.x == 0 && tid == 0) {
            a.plan[0] = com.lo;
            a.plan[1] = com.hi;
        }
        __syncthreads();
    }

    __device__ void run() {
        const Shares sh(total, gridDim.x);
        if ((int)blockIdx.x >= min(total, (int)gridDim.x)) return;
        const int u0 = sh.begin(blockIdx.x), n = sh.begin(blockIdx.x + 1) - u0;
        Place work = place(u0), load = work;
        prepare(load);
        int loaded = 0;
        bool load_fresh = true;  // load is the first tile of its item in this CTA
        auto fetch_next = [&] {
            if (loaded < n) {
                fetch(loaded % L::STAGES, load, load_fresh);
                if (loaded + 1 < n) {
                    load_fresh = advance(load);
                    prepare(load);
                }
            }
            ++loaded;
            cp_async_commit();
        };
        for (int i = 0; i < L::STAGES - 1; ++i) fetch_next();
        bool fresh = true;
        for (int i = 0; i < n; ++i) {
            if (fresh && work.common) common_queries(work);
            fetch_next();
            asm volatile("cp.async.wait_group %0;" ::"n"(L::STAGES - 1) : "memory");
            __syncthreads();
            const bool last = i + 1 == n || work.tile + 1 == work.tiles;
            if (tid == 0) {  // for the join
                int2 *sp = a.span + (work.common ? work.item : a.items_c + work.item);
                if (work.tile == 0) sp->x = blockIdx.x;
                if (work.tile + 1 == work.tiles) sp->y = blockIdx.x;
            }
            if (work.common) {
                const int rows = min(PA_ROWS, a.kv.n_seqs * a.group - work.rt * PA_ROWS);
                if (rows <= 16)
                    tile<1>(work, rows, fresh, last, i % L::STAGES);
                else if (rows <= 32)
                    tile<2>(work, rows, fresh, last, i % L::STAGES);
                else
                    tile<4>(work, rows, fresh, last, i % L::STAGES);
            } else {
                tile<1>(work, a.group, fresh, last, i % L::STAGES);
            }
            __syncthreads();  // the stage may be written again
            fresh = last;
            if (i + 1 < n) advance(work);
        }
    }

    // One (sequence, KV head) by the CTAs of a cluster, result and all: each takes
    // an equal share of its tiles, and all join the partials through
    // distributed shared memory.
    __device__ void run_direct() {
        cg::cluster_group cl = cg::this_cluster();
        const int parts = (int)cl.num_blocks(), part = (int)cl.block_rank();
        Place p;
        p.common = false;
        p.item = quotient(blockIdx.x, parts);
        p.b = quotient(p.item, a.kv.n_kv);
        p.h = p.item - p.b * a.kv.n_kv;
        p.rt = 0;
        if (p.h == 0 && part == 0 && tid == 0 && (a.lens[p.b] < 0 || a.lens[p.b] > a.max_len)) atomicExch(a.err, 1u);
        set_keys(p);  // (com is empty: all that the sequence sees is its own)
        p.tiles = (p.keys + KT - 1) / KT;
        const Shares sh(p.tiles, parts);
        const bool some = part < p.tiles;
        const int t0 = some ? sh.begin(part) : 0, n = some ? sh.begin(part + 1) - t0 : 0;
        p.tile = t0;
        Place load = p;
        auto fetch_next = [&](int i) {
            if (i < n) {
                prepare(load);
                fetch(i % L::STAGES, load, i == 0);
                ++load.tile;
            }
            cp_async_commit();
        };
        for (int i = 0; i < L::STAGES - 1; ++i) fetch_next(i);
        for (int i = 0; i != n; ++i) {
            fetch_next(i + L::STAGES - 1);
            asm volatile("cp.async.wait_group %0;" ::"n"(L::STAGES - 1) : "memory");
            __syncthreads();
            tile<1, true>(p, a.group, i == 0, i + 1 == n, i % L::STAGES);
            __syncthreads();
            ++p.tile;
        }
        // this CTA's partial lies in shared memory (finish); an empty share leaves nothing
        float *mine = direct_o();
        float2 *stat = direct_ml();
        if (n == 0) {
            for (int x = tid; x < a.group * DH; x += PA_THREADS) mine[x] = 0.f;
            if (tid < a.group) stat[tid] = make_float2(-INFINITY, 0.f);
        }
        if (parts > 1)
            cl.sync();
        else
            __syncthreads();
        const int pairs = a.group * (DH / 2), per = (pairs + parts - 1) / parts;
        for (int x = part * per + tid; x < min(pairs, (part + 1) * per); x += PA_THREADS) {
            const int row = x / (DH / 2), c = (x % (DH / 2)) * 2;
            float2 w[8], v[8];
            float mx = -INFINITY;
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (k < parts) {
                    w[k] = parts > 1 ? *cl.map_shared_rank(stat + row, k) : stat[row];
                    v[k] = *reinterpret_cast<const float2 *>(parts > 1 ? cl.map_shared_rank(mine + row * DH + c, k)
                                                                       : mine + row * DH + c);
                    mx = fmaxf(mx, w[k].x);
                }
            const float off = mx == -INFINITY ? 0.f : mx;
            float sx = 0.f, sy = 0.f, sl = 0.f;
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (k < parts) {
                    const float f = ex2(w[k].x - off);
                    sx += f * v[k].x;
                    sy += f * v[k].y;
                    sl += f * w[k].y;
                }
            const float inv = inverse(sl);
            *reinterpret_cast<uint32_t *>(static_cast<T *>(a.out) + (long long)p.b * a.ld_out +
                                          (long long)(p.h * a.group + row) * DH + c) = pack2<T>(sx * inv, sy * inv);
            if (c == 0 && a.lse)
                a.lse[(long long)p.b * a.n_q + p.h * a.group + row] = mx * 0.69314718055994530942f + logf(sl);
        }
        if (parts > 1) cl.sync();  // nobody leaves while its partial is read
    }

  private:
    using L = Smem<T, DH>;
    static constexpr int KT = L::KT;
    const AttnArgs &a;
    uint8_t *stage0, *q0;
    float2 *ml;
    int *cum;
    int tid, warp, lane;
    Common com;
    int tiles_c;
    int common_total, total;
    // the tile to be fetched next: element offsets of rows lane + 32 i (-1: no such key)
    long long row_off[KT / 32];

    // running state of this warp's 16 rows (lane 4 g + t: rows g and g + 8)
    uint32_t qf[DH / 16][4];
    float o[DH / 8][4];
    float m[2], l[2];

    // The keys of p's item.
    __device__ void set_keys(Place &p) const {
        p.gap_at = INT_MAX;
        p.gap = 0;
        if (p.common) {
            p.first = com.lo;
            p.keys = com.hi - com.lo;
            return;
        }
        const Span s = span_of(a, p.b);
        p.first = s.lo;
        p.keys = own_count(s, com);
        if (s.member) {
            p.gap_at = max(0, com.lo - s.lo);
            p.gap = com.hi - max(com.lo, s.lo);
        }
    }

    __device__ Place place(int u) const {
        Place p;
        if (u < common_total) {
            p.common = true;
            p.item = quotient(u, tiles_c);
            p.tile = u - p.item * tiles_c;
            p.tiles = tiles_c;
            p.h = quotient(p.item, a.row_tiles);
            p.rt = p.item - p.h * a.row_tiles;
            p.b = 0;
        } else {
            const int v = u - common_total;
            int lo = 0, hi = a.kv.n_seqs;  // the sequence with n_kv cum[b] <= v < n_kv cum[b + 1]
            while (hi - lo > 1) {
                const int mid = (lo + hi) / 2;
                if (a.kv.n_kv * cum[mid] <= v)
                    lo = mid;
                else
                    hi = mid;
            }
            p.common = false;
            p.b = lo;
            p.tiles = cum[lo + 1] - cum[lo];
            const int r = v - a.kv.n_kv * cum[lo];
            p.h = quotient(r, p.tiles);
            p.tile = r - p.h * p.tiles;
            p.rt = 0;
            p.item = p.b * a.kv.n_kv + p.h;
        }
        set_keys(p);
        return p;
    }

    // The next tile of the list; true if it begins another item.
    __device__ bool advance(Place &p) const {
        if (++p.tile < p.tiles) return false;
        p.tile = 0;
        ++p.item;
        if (p.common) {
            if (++p.rt < a.row_tiles) return true;
            p.rt = 0;
            if (++p.h < a.kv.n_kv) return true;
            p.common = false;  // on to the own items
            p.b = -1;
        } else {
            if (++p.h < a.kv.n_kv) return true;
        }
        p.h = 0;
        do {
            ++p.b;
        } while (p.b < a.kv.n_seqs - 1 && cum[p.b + 1] == cum[p.b]);
        p.tiles = cum[p.b + 1] - cum[p.b];
        p.item = p.b * a.kv.n_kv;
        set_keys(p);
        return true;
    }

    // Looks up the pages of p's tile.
    __device__ void prepare(const Place &p) {
        int page[KT / 32], pos[KT / 32];
#pragma unroll
        for (int i = 0; i < KT / 32; ++i) {  // (the loads first: none of them may pass the flag's atomic)
            const int k = p.tile * KT + lane + 32 * i, j = p.first + k + (k >= p.gap_at ? p.gap : 0);
            const int row = j < a.shared ? 0 : p.b;
            pos[i] = j;
            page[i] = 0;
            if (k < p.keys) page[i] = a.kv.table[(long long)row * a.kv.max_pages + (j >> a.kv.ps_log2)];
        }
        bool bad = false;
#pragma unroll
        for (int i = 0; i < KT / 32; ++i) {
            const bool key = p.tile * KT + lane + 32 * i < p.keys, in = page[i] >= 0 && page[i] < a.kv.n_pages;
            bad |= key && !in;
            row_off[i] = key && in ? page[i] * a.kv.page_stride +
                                         ((((long long)p.h << a.kv.ps_log2) + (pos[i] & ((1 << a.kv.ps_log2) - 1))) * DH)
                                   : -1;
        }
        if (bad) atomicExch(a.err, 1u);
    }

    // Starts the copies of the prepared tile into stage s
    // and, with the first tile of an own item, of the item's query rows.
    __device__ void fetch(int s, const Place &p, bool first) {
        constexpr int CH = DH / 8;                  // 16-byte chunks per row
        if (first && !p.common) {
            const uint32_t qs = smem_u32(q0 + s * L::Q);
            const T *q = static_cast<const T *>(a.q) + (long long)p.b * a.ld_q + (long long)p.h * a.group * DH;
            for (int x = tid; x < a.group * CH; x += PA_THREADS)
                cp16_or_zero(qs + tile_off<DH>(x / CH, x % CH), q + (x / CH) * DH + (x % CH) * 8, true);
        }
        constexpr int RP = PA_THREADS / CH;         // rows per pass
        const int c = tid % CH, r0 = tid / CH;
        const uint32_t ks = smem_u32(stage0 + (size_t)s * 2 * L::TILE), vs = ks + L::TILE;
        const T *k = static_cast<const T *>(a.kv.k), *v = static_cast<const T *>(a.kv.v);
#pragma unroll
        for (int i = 0; i < KT / RP; ++i) {
            const int r = i * RP + r0;
            // (the RP rows of a pass lie in one group of 32: RP divides 32)
            const long long off = __shfl_sync(0xffffffffu, row_off[i * RP / 32], r & 31);
            const long long at = off < 0 ? 0 : off + c * 8;
            cp16_or_zero(ks + tile_off<DH>(r, c), k + at, off >= 0);
            cp16_or_zero(vs + tile_off<DH>(r, c), v + at, off >= 0);
        }
    }

    // Where a CTA of run_direct leaves its partial, the same place in all: o in the
    // query rows' buffers (the queries are in registers by then), the statistics
    // where the list's table would be.
    __device__ float *direct_o() const { return reinterpret_cast<float *>(q0); }
    __device__ float2 *direct_ml() const { return reinterpret_cast<float2 *>(cum); }

    // One tile of an item's rows: WR warps side by side in rows, 4 / WR in keys.
    // DIRECT: the item's end is the result, not a partial.
    template <int WR, bool DIRECT = false>
    __device__ void tile(const Place &p, int rows, bool fresh, bool last, int s) {
        constexpr int WK = 4 / WR, NB = KT / (16 * WK);  // NB blocks of 16 keys per warp
        const int wr = warp % WR, wk = warp / WR, t = lane & 3;
        if (fresh) {
            if (!p.common) {  // (rows past the group hold anything: their results are dropped)
                const uint32_t qs = smem_u32(q0 + s * L::Q);
#pragma unroll
                for (int kk = 0; kk < DH / 16; ++kk) ldsm_x4(qs + tile_off<DH>(lane & 15, 2 * kk + (lane >> 4)), qf[kk]);
            }
#pragma unroll
            for (int i = 0; i < DH / 8; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) o[i][j] = 0.f;
            m[0] = m[1] = -INFINITY;
            l[0] = l[1] = 0.f;
        }
        const uint32_t ks = smem_u32(stage0 + (size_t)s * 2 * L::TILE), vs = ks + L::TILE;
        const int left = p.keys - p.tile * KT;  // keys of this tile (may exceed it)
        float sc[2 * NB][4];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            const int key0 = (nb * WK + wk) * 16;
#pragma unroll
            for (int j = 0; j < 4; ++j) sc[2 * nb][j] = sc[2 * nb + 1][j] = 0.f;
#pragma unroll
            for (int kk = 0; kk < DH / 16; ++kk) {
                // matrices: keys 0-7 | dims 0-7, keys 0-7 | dims 8-15, keys 8-15 | dims 0-7, keys 8-15 | dims 8-15
                uint32_t r[4];
                ldsm_x4(ks + tile_off<DH>(key0 + (lane & 7) + ((lane >> 4) << 3), 2 * kk + ((lane >> 3) & 1)), r);
                mma<T>(sc[2 * nb], qf[kk], r[0], r[1]);
                mma<T>(sc[2 * nb + 1], qf[kk], r[2], r[3]);
            }
        }
        if (left < KT) {
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const int key = (nb * WK + wk) * 16 + x * 8 + 2 * t;
                    if (key >= left) sc[2 * nb + x][0] = sc[2 * nb + x][2] = -INFINITY;
                    if (key + 1 >= left) sc[2 * nb + x][1] = sc[2 * nb + x][3] = -INFINITY;
                }
        }
#pragma unroll
        for (int r = 0; r < 2; ++r) {  // rows g, g + 8
            float mx = -INFINITY;
#pragma unroll
            for (int i = 0; i < 2 * NB; ++i) mx = fmaxf(mx, fmaxf(sc[i][2 * r], sc[i][2 * r + 1]));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            const float mn = fmaxf(m[r], mx * a.scale_log2);
            const float off = mn == -INFINITY ? 0.f : mn;
            const float fac = ex2(m[r] - off);
            m[r] = mn;
            l[r] *= fac;
#pragma unroll
            for (int i = 0; i < DH / 8; ++i) {
                o[i][2 * r] *= fac;
                o[i][2 * r + 1] *= fac;
            }
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < 2 * NB; ++i)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const float e = ex2(fmaf(sc[i][2 * r + x], a.scale_log2, -off));
                    sc[i][2 * r + x] = e;
                    sum += e;
                }
            l[r] += sum;  // this lane's keys only: joined at the end
        }
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            const int key0 = (nb * WK + wk) * 16;
            uint32_t pf[4];
            pf[0] = pack2<T>(sc[2 * nb][0], sc[2 * nb][1]);
            pf[1] = pack2<T>(sc[2 * nb][2], sc[2 * nb][3]);
            pf[2] = pack2<T>(sc[2 * nb + 1][0], sc[2 * nb + 1][1]);
            pf[3] = pack2<T>(sc[2 * nb + 1][2], sc[2 * nb + 1][3]);
#pragma unroll
            for (int d = 0; d < DH / 16; ++d) {
                // transposed matrices: keys 0-7 | dims 0-7, keys 8-15 | dims 0-7, then dims 8-15
                uint32_t r[4];
                ldsm_x4_trans(vs + tile_off<DH>(key0 + (lane & 15), 2 * d + (lane >> 4)), r);
                mma<T>(o[2 * d], pf, r[0], r[1]);
                mma<T>(o[2 * d + 1], pf, r[2], r[3]);
            }
        }
        if (last) finish<WR, DIRECT>(p, wr, rows, s);
    }

    // Q fragments of this warp's 16 rows of a common item, straight from global
    // memory (rows past the item's are zero).
    __device__ void common_queries(const Place &p) {
        const int rows = min(PA_ROWS, a.kv.n_seqs * a.group - p.rt * PA_ROWS);
        const int wr = rows <= 16 ? 0 : rows <= 32 ? warp % 2 : warp, g = lane >> 2, t = lane & 3;
        const T *base[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int row = wr * 16 + g + 8 * r;
            base[r] = nullptr;
            if (row < rows) {
                const int all = p.rt * PA_ROWS + row, b = all / a.group;
                base[r] = static_cast<const T *>(a.q) + (long long)b * a.ld_q +
                          (long long)(p.h * a.group + all - b * a.group) * DH;
            }
        }
#pragma unroll
        for (int kk = 0; kk < DH / 16; ++kk)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const T *q = base[i & 1];
                qf[kk][i] = q ? *reinterpret_cast<const uint32_t *>(q + kk * 16 + (i >> 1) * 8 + 2 * t) : 0u;
            }
    }

    // The item's partial: (o, max, sum) per row, warps with the same rows joined.
    template <int WR, bool DIRECT>
    __device__ void finish(const Place &p, int wr, int rows, int s) {
        constexpr int WK = 4 / WR;
        const int g = lane >> 2, t = lane & 3;
        const long long slot0 = p.common ? (long long)(p.item + blockIdx.x) * PA_ROWS
                                         : (long long)a.slots_c * a.rows_c + (long long)(p.item + blockIdx.x) * a.group;
        float *dst = a.part_o + slot0 * DH;
        float2 *dst_ml = a.part_ml + slot0;
        const uint64_t keep = policy_evict_last();  // the keys and values that stream by shall not push it out of L2
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
            l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
        }
        if constexpr (WK == 1) {
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int row = wr * 16 + g + 8 * r;
                if (row >= rows) continue;
                float *d = dst + row * DH;
#pragma unroll
                for (int i = 0; i < DH / 8; ++i)
                    st_hint(reinterpret_cast<float2 *>(d + 8 * i + 2 * t), make_float2(o[i][2 * r], o[i][2 * r + 1]), keep);
                if (t == 0) dst_ml[row] = make_float2(m[r], l[r]);
            }
        } else {
            __syncthreads();  // every warp has read this stage's keys and values
            // row r of warp w at (w * 16 + r) * DH, its columns permuted by the row (8 rows of a warp write 8 bank groups)
            float *red = reinterpret_cast<float *>(stage0 + (size_t)s * 2 * L::TILE);
            auto col = [](int row, int c) { return c ^ ((row & (DH / 8 - 1) & 7) << 3); };
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int row = g + 8 * r;
                float *d = red + (warp * 16 + row) * DH;
#pragma unroll
                for (int i = 0; i < DH / 8; ++i)
                    *reinterpret_cast<float2 *>(d + col(row, 8 * i) + 2 * t) = make_float2(o[i][2 * r], o[i][2 * r + 1]);
                if (t == 0) ml[warp * 16 + row] = make_float2(m[r], l[r]);
            }
            __syncthreads();
            for (int x = tid; x < rows * (DH / 2); x += PA_THREADS) {
                const int row = x / (DH / 2), c = (x % (DH / 2)) * 2;
                float mx = -INFINITY;  // over the key shares k: warp row / 16 + k * WR
#pragma unroll
                for (int k = 0; k < WK; ++k) mx = fmaxf(mx, ml[row + k * WR * 16].x);
                const float off = mx == -INFINITY ? 0.f : mx;
                float sx = 0.f, sy = 0.f, sl = 0.f;
#pragma unroll
                for (int k = 0; k < WK; ++k) {
                    const float2 w = ml[row + k * WR * 16];
                    const float f = ex2(w.x - off);
                    const float2 v = *reinterpret_cast<const float2 *>(red + (row + k * WR * 16) * DH +
                                                                       col(row, c & ~7) + (c & 7));
                    sx += f * v.x;
                    sy += f * v.y;
                    sl += f * w.y;
                }
                if constexpr (DIRECT) {
                    *reinterpret_cast<float2 *>(direct_o() + row * DH + c) = make_float2(sx, sy);
                    if (c == 0) direct_ml()[row] = make_float2(mx, sl);
                } else {
                    st_hint(reinterpret_cast<float2 *>(dst + row * DH + c), make_float2(sx, sy), keep);
                    if (c == 0) dst_ml[row] = make_float2(mx, sl);
                }
            }
        }
    }
};

template <typename T, int DH>
__global__ void __launch_bounds__(PA_THREADS, PA_CTAS_PER_SM) paged_attn_kernel(const AttnArgs a) {
    extern __shared__ __align__(128) uint8_t pa_smem[];
    Walker<T, DH> w(a, pa_smem);
    // (Behind the tensor-core kernel too.  Its trigger lets these CTAs become
    // resident as its own leave, but only the wait makes visible what the kernels
    // before it wrote.)
    pdl_wait();
    pdl_trigger();
    w.plan();
    w.run();
}

// A cluster per (sequence, KV head) and no other launch: for few keys.
template <typename T, int DH>
__global__ void __launch_bounds__(PA_THREADS, PA_CTAS_PER_SM) paged_attn_direct(const AttnArgs a) {
    extern __shared__ __align__(128) uint8_t pa_smem[];
    pdl_wait();
    pdl_trigger();
    Walker<T, DH>(a, pa_smem).run_direct();
}

// One warp per (sequence, query head): the row's partials joined in list
// order (common item first), normalised and rounded once.
template <typename T, int DH>
__global__ void __launch_bounds__(PA_MERGE_THREADS) paged_attn_join(const AttnArgs a) {
    constexpr int V = DH / 32;  // values per lane
    constexpr int U = 8;        // partials in flight
    const int x = (int)((blockIdx.x * (long long)PA_MERGE_THREADS + threadIdx.x) >> 5), lane = threadIdx.x & 31;
    const int b = x / a.n_q, hq = x - b * a.n_q, h = hq / a.group, r = hq - h * a.group;
    const int row = b * a.group + r, item = h * a.row_tiles + row / a.rows_c, own = b * a.kv.n_kv + h;
    const bool active = x < a.kv.n_seqs * a.n_q;
    pdl_wait();
    pdl_trigger();
    if (!active) return;
    // (of earlier calls, or anything, where this one has no tiles or gave up)
    int2 at_c = a.span[item];
    const int2 at_o = a.span[a.items_c + own];
    at_c.x = max(0, min(at_c.x, a.grid_c - 1));
    at_c.y = max(at_c.x, min(at_c.y, a.grid_c - 1));
    Common com(a, -1);
    com.lo = a.plan[0];
    com.hi = a.plan[1];
    const Span s = span_of(a, b);
    // partial k < n_c of the common item, then n_o of the own one: their rows in the workspace
    const int n_c = s.member && com.lo < com.hi ? at_c.y - at_c.x + 1 : 0;
    const int n_o = own_count(s, com) > 0 ? at_o.y - at_o.x + 1 : 0;
    const long long row_c = (long long)(item + at_c.x) * a.rows_c + row % a.rows_c;
    const long long row_o = (long long)a.slots_c * a.rows_c + (long long)(own + at_o.x) * a.group + r;
    auto row_of = [&](int k) {
        return k < n_c ? row_c + (long long)k * a.rows_c : row_o + (long long)(k - n_c) * a.group;
    };
    float acc[V], mx = -INFINITY, sum = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = 0.f;
    const int n = n_c + n_o;
    for (int k0 = 0; k0 < n; k0 += 32) {
        const int c = min(32, n - k0);
        const long long mine = row_of(k0 + min(lane, c - 1));
        float2 w = a.part_ml[mine];
        if (lane >= c) w = make_float2(-INFINITY, 0.f);
        for (int k = 0; k < c; k += U) {
            float v[U][V];
#pragma unroll
            for (int j = 0; j < U; ++j) {
                const float *d = a.part_o + __shfl_sync(0xffffffffu, mine, min(k + j, c - 1)) * DH + lane * V;
                if constexpr (V == 4)
                    *reinterpret_cast<float4 *>(v[j]) = *reinterpret_cast<const float4 *>(d);
                else if constexpr (V == 2)
                    *reinterpret_cast<float2 *>(v[j]) = *reinterpret_cast<const float2 *>(d);
                else
                    v[j][0] = d[0];
            }
            // (the statistics arrive with the first of these loads)
            float f = 0.f;
            if (k == 0) {
                float mn = w.x;
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
                mn = fmaxf(mn, mx);
                const float off = mn == -INFINITY ? 0.f : mn, f0 = ex2(mx - off);
                w.x = ex2(w.x - off);  // from here on the partial's weight
                float add = w.y * w.x;
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) add += __shfl_xor_sync(0xffffffffu, add, o);
                mx = mn;
                sum = sum * f0 + add;
#pragma unroll
                for (int i = 0; i < V; ++i) acc[i] *= f0;
            }
#pragma unroll
            for (int j = 0; j < U; ++j) {
                f = __shfl_sync(0xffffffffu, w.x, (k + j) & 31);
                if (k + j < c) {
#pragma unroll
                    for (int i = 0; i < V; ++i) acc[i] += v[j][i] * f;
                }
            }
        }
    }
    const float inv = inverse(sum);
    T *dst = static_cast<T *>(a.out) + (long long)b * a.ld_out + (long long)hq * DH + lane * V;
    if constexpr (V == 1) {
        dst[0] = (T)(acc[0] * inv);
    } else {
#pragma unroll
        for (int i = 0; i < V; i += 2)
            *reinterpret_cast<uint32_t *>(dst + i) = pack2<T>(acc[i] * inv, acc[i + 1] * inv);
    }
    if (a.lse && lane == 0) a.lse[(long long)b * a.n_q + hq] = mx * 0.69314718055994530942f + logf(sum);
}

int sm_count() {
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
        (void)cudaGetLastError();
        return 0;
    }
    return n;
}

size_t al256(size_t n) { return (n + 255) & ~size_t(255); }

// How the common rows are cut: 64 rows a pass on warp-level MMAs, or 256 on the
// tensor cores of lf_paged_attn_tc.cu.
void common_shape(AttnArgs &a, bool tc, int n_sm) {
    const long long rows = (long long)a.kv.n_seqs * a.group;
    a.tc = tc;
    a.rows_c = tc ? kTcRows : PA_ROWS;
    a.keys_c = tc ? kTcKeys : tile_keys(a.kv.head_dim);
    a.row_tiles = (int)((rows + a.rows_c - 1) / a.rows_c);
    a.grid = n_sm * PA_CTAS_PER_SM;
    a.grid_c = tc ? n_sm : a.grid;
    a.page_align = tc ? 1 << a.kv.ps_log2 : 1;
    a.items_c = a.kv.n_kv * a.row_tiles;
    a.slots_c = a.items_c + a.grid_c;
}

// CTAs to a (sequence, KV head) of the direct kernel, 0 for the list and its
// join.  Without the list, its table and the second launch a call of few keys
// is 3 to 5 us shorter, but every sequence reads the common positions itself and a
// CTA's tiles follow one another (0.7 us each).  As many CTAs as there are tiles
// and as two per SM allow; then at most 512 keys a CTA, fewer where the grid
// takes more than one wave.  Measured (us, list | direct by 1, 2, 4, 8), head_dim 128, n
// (sequence, KV head) items x keys:
//    16 x 160   6.2 | 4.7 4.9 4.3 4.4       128 x 160   8.5 | 4.9 5.9 9.1 16.7
//    16 x 1000  7.4 | 14.2 9.1 6.5 5.3      128 x 512   9.5 | 8.6 7.9 11.4 18.4
//    16 x 4096 12.5 | 49.6 27.0 15.3 11.0   128 x 1000 11.9 | 14.5 11.5 14.3 21.5
//    64 x 2048 11.0 | 26.3 15.3 11.4 14.8   128 x 2048 14.1 | 26.5 19.0 22.4 29.0
//   256 x 512  12.6 | 10.9 15.3 21.8        512 x 160  11.0 | 10.6 20.1
//   256 x 1000 14.6 | 18.1 21.5 27.3        512 x 256  11.3 | 12.9 21.9
// (over 179 such sizes, 64 wide heads too, the rule is 1.2 % off the best choice, 21 %
// at most).
// Not where the common positions read once more by every sequence make over 16
// MB: alone that is L2's to give (64 x 1000 at 4 sequences: 10.4 | 7.7), but in a
// step that streams weights beside it the list is faster (the batched decode of 4
// and 8 samples, 3584 common positions: 0.868 | 0.876 and 0.890 | 0.905 ms a step).
int direct_parts(const AttnArgs &a, int n_sm) {
    const int bound = a.window > 0 ? std::min(a.window, a.max_len) : a.max_len, kt = tile_keys(a.kv.head_dim);
    const int tiles = bound / kt + (bound % kt != 0);
    const long long items = (long long)a.kv.n_seqs * a.kv.n_kv;
    if (items > 6 * n_sm) return 0;
    if ((items - a.kv.n_kv) * std::min(a.shared, bound) * a.kv.head_dim * 4 > (16 << 20)) return 0;
    int parts = 1;
    while (parts < 8 && parts < tiles && items * parts * 2 <= 2 * n_sm) parts *= 2;
    const long long waves = (items * parts + 2 * n_sm - 1) / (2 * n_sm);
    const int each = (tiles + parts - 1) / parts;
    return waves * each <= (waves == 1 ? 512 / kt : 6) ? parts : 0;
}

struct WsLayout {
    size_t span, ml, o, bytes;
};
WsLayout ws_layout(const AttnArgs &a) {
    WsLayout w;
    const size_t rows = (size_t)a.slots_c * a.rows_c + ((size_t)a.kv.n_seqs * a.kv.n_kv + a.grid) * a.group;
    w.span = 256;  // behind the plan
    w.ml = w.span + al256(((size_t)a.items_c + (size_t)a.kv.n_seqs * a.kv.n_kv) * sizeof(int2));
    w.o = w.ml + al256(rows * sizeof(float2));
    w.bytes = w.o + rows * a.kv.head_dim * sizeof(float);
    return w;
}

// The tensor-core kernel takes head_dim 64 and 128, pages of at least 8 positions
// (a TMA box) and page strides that a tensor map can hold (2^40 bytes).
bool tc_possible(const PagedView &v) { return v.head_dim >= 64 && v.ps_log2 >= 3 && v.page_stride < (1ll << 38); }
// It costs one more launch and a second start (8 to 10 us; the own items wait for
// all of it), its 128-row tiles idle where there are few rows, and each CTA leaves a
// partial of up to 256 rows; it gains as the common products grow.  Both measured
// (us, warp-level MMAs | tensor cores), 64 own positions, common ones in whole
// pages, by rows of a KV head x common positions:
//   head_dim 128, 8 KV heads:   64 x 15232 31.4 | 29.3   64 x 25920 41.8 | 39.9   33 x 29568 42.4 | 40.1
//                              128 x 4544  22.3 | 23.3  128 x 7616  28.0 | 25.3  128 x 18304 45.8 | 36.6
//                              256 x 3813  27.5 | 30.1  256 x 9189  43.3 | 33.5  512 x 3200 37.3 | 39.2
//   head_dim 128, 16 KV heads:  64 x 9856  34.4 | 34.6  128 x 3776  28.3 | 30.4  128 x 6464 37.8 | 33.4
//                              256 x 3237  37.3 | 41.8  256 x 4581  45.8 | 35.6   32 x 16384 37.3 | 42.2
//   head_dim 64, 8 KV heads:    64 x 39616 35.1 | 38.5  128 x 15232 28.3 | 26.4  256 x 7653 27.3 | 24.6
//   head_dim 64, 16 KV heads:  128 x 9856  33.0 | 30.1  512 x 3776 28.4 | 29.7 (8 KV heads), 512 x 2432 38.9 | 34.3
// so: by the size of the common products, not where half of a row tile (a quarter at
// head_dim 128) would be empty, and from three key tiles a CTA on, which pay for its
// partial.  With a window at most that many positions are common.  (Over 150
// such sizes from 0.5e9 to 2.4e9 the rule is 1 % off the better choice, 10 % at most.)
bool tc_pays(const AttnArgs &a, int n_sm) {
    const long long rows = (long long)a.kv.n_seqs * a.group, keys = a.window > 0 ? std::min(a.window, a.shared) : a.shared;
    const long long tiles = keys / kTcKeys * ((rows + kTcRows - 1) / kTcRows) * a.kv.n_kv;
    return rows > (a.kv.head_dim == 128 ? 32 : 64) && tiles >= 3 * n_sm &&
           (double)rows * (double)keys * a.kv.n_kv * a.kv.head_dim >= 9.5e8;
}

size_t ws_bytes(AttnArgs a, int n_sm) {
    common_shape(a, false, n_sm);
    size_t n = ws_layout(a).bytes;
    if (tc_possible(a.kv)) {
        common_shape(a, true, n_sm);
        n = std::max(n, ws_layout(a).bytes);
    }
    return n;
}

lf_status check_shape(const lf_paged_kv *kv, int n_q_heads, PagedView *v) {
    const lf_status st = paged_view(kv, v);
    if (st != LF_OK) return st;
    if (n_q_heads < 1 || n_q_heads % v->n_kv) return LF_ERR_INVALID_ARG;
    if ((v->head_dim != 32 && v->head_dim != 64 && v->head_dim != 128) || n_q_heads / v->n_kv > PA_MAX_GROUP ||
        v->n_seqs > PA_MAX_SEQS)
        return LF_ERR_UNSUPPORTED;
    if ((long long)v->n_seqs * n_q_heads > (1 << 26)) return LF_ERR_UNSUPPORTED;  // item numbers are 32-bit
    return LF_OK;
}

template <typename T, int DH>
lf_status launch_attn(const AttnArgs &a, int direct, cudaStream_t st) {
    constexpr int smem = Smem<T, DH>::BYTES;
    if (direct)
        return set_smem_once<paged_attn_direct<T, DH>>(smem) &&
                       launch_pdl_cluster(paged_attn_direct<T, DH>, (unsigned)direct,
                                          dim3((unsigned)(a.kv.n_seqs * a.kv.n_kv * direct)), PA_THREADS, smem, st, a)
                   ? LF_OK
                   : LF_ERR_CUDA;
    if (!set_smem_once<paged_attn_kernel<T, DH>>(smem)) return LF_ERR_CUDA;
    if constexpr (DH >= 64) {
        if (a.tc) {
            const lf_status ts = paged_attn_tc(a, std::is_same<T, __half>::value ? LF_F16 : LF_BF16, st);
            if (ts != LF_OK) return ts;
        }
    }
    if (!launch_pdl(paged_attn_kernel<T, DH>, a.grid, PA_THREADS, smem, st, a)) return LF_ERR_CUDA;
    const long long threads = (long long)a.kv.n_seqs * a.n_q * 32;
    const unsigned blocks = (unsigned)((threads + PA_MERGE_THREADS - 1) / PA_MERGE_THREADS);
    return launch_pdl(paged_attn_join<T, DH>, blocks, PA_MERGE_THREADS, 0, st, a) ? LF_OK : LF_ERR_CUDA;
}

template <typename T>
lf_status launch_attn_dim(const AttnArgs &a, int direct, cudaStream_t st) {
    return a.kv.head_dim == 32   ? launch_attn<T, 32>(a, direct, st)
           : a.kv.head_dim == 64 ? launch_attn<T, 64>(a, direct, st)
                                 : launch_attn<T, 128>(a, direct, st);
}

}  // namespace
}  // namespace lf

extern "C" size_t lf_attn_paged_shared_workspace(const lf_paged_kv *kv, int n_q_heads) {
    lf::AttnArgs a = {};
    if (lf::check_shape(kv, n_q_heads, &a.kv) != LF_OK) return 0;
    a.group = n_q_heads / a.kv.n_kv;
    const int n_sm = lf::sm_count();
    return n_sm ? lf::ws_bytes(a, n_sm) : 0;
}

extern "C" lf_status lf_attn_paged_shared(const lf_paged_kv *kv, const void *q_device, int64_t ld_q, void *out_device,
                                          int64_t ld_out, float *lse_device, int n_q_heads, const int32_t *lens_device,
                                          int max_len, int shared_len, int window, float scale, void *workspace_device,
                                          size_t workspace_bytes, uint32_t *err_device, void *cuda_stream) {
    lf::AttnArgs a = {};
    const lf_status cs = lf::check_shape(kv, n_q_heads, &a.kv);
    if (cs != LF_OK) return cs;
    const int64_t row = (int64_t)n_q_heads * kv->head_dim, cap = (int64_t)kv->max_pages * kv->page_size;
    auto off4 = [](const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) != 0; };
    if (!q_device || !out_device || !lens_device || !workspace_device || !err_device || !lf::aligned16(q_device) ||
        !lf::aligned16(out_device) || off4(lse_device) || off4(lens_device) || off4(err_device) ||
        (reinterpret_cast<uintptr_t>(workspace_device) & 255u) || ld_q < row || ld_out < row || ld_q % 8 ||
        ld_out % 8 || max_len < 0 || max_len > cap || shared_len < 0 || shared_len > max_len || window < 0 ||
        !(scale > 0.f && scale * lf::kLog2e < INFINITY))
        return LF_ERR_INVALID_ARG;
    a.group = n_q_heads / a.kv.n_kv;
    // tiles are counted in 32 bits
    const int kt = lf::tile_keys(kv->head_dim);
    const long long per_head = (long long)(shared_len / kt + 1) * (((long long)kv->n_seqs * a.group) / lf::PA_ROWS + 1) +
                               (long long)(max_len / kt + 2) * kv->n_seqs;
    if (per_head * kv->n_kv_heads > INT_MAX) return LF_ERR_UNSUPPORTED;
    const int n_sm = lf::sm_count();
    if (!n_sm) return LF_ERR_CUDA;
    if (workspace_bytes < lf::ws_bytes(a, n_sm)) return LF_ERR_INVALID_ARG;
    a.shared = shared_len;
    a.window = window;
    lf::common_shape(a, lf::tc_possible(a.kv) && lf::tc_pays(a, n_sm), n_sm);
    const lf::WsLayout w = lf::ws_layout(a);
    uint8_t *ws = static_cast<uint8_t *>(workspace_device);
    a.plan = reinterpret_cast<int *>(ws);
    a.span = reinterpret_cast<int2 *>(ws + w.span);
    a.part_ml = reinterpret_cast<float2 *>(ws + w.ml);
    a.part_o = reinterpret_cast<float *>(ws + w.o);
    a.q = q_device;
    a.out = out_device;
    a.lse = lse_device;
    a.ld_q = ld_q;
    a.ld_out = ld_out;
    a.n_q = n_q_heads;
    a.lens = lens_device;
    a.max_len = max_len;
    a.scale_log2 = scale * lf::kLog2e;
    a.err = err_device;
    const int direct = lf::direct_parts(a, n_sm);
    cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
    return kv->dtype == LF_F16 ? lf::launch_attn_dim<__half>(a, direct, st) : lf::launch_attn_dim<__nv_bfloat16>(a, direct, st);
}
