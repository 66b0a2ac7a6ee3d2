// Attention of each sequence's new tokens over a paged cache that holds them:
// o = softmax(scale q K^T) V per query head, causal (and windowed) by position.
//
// The rows (token, head of the group) of a few tokens are the M side of a product
// with a tile of keys (the list of such items: lf_paged_chunk.h).  Here: warp-level
// MMAs (m16n8k16, fp32 accumulators), 16, 32 or 64 rows an item, K and V tiles of 64
// or 128 keys through a cp.async ring that runs on across item borders, softmax
// statistics in registers.  Warps take 16-row blocks, and 16-key blocks where the
// rows are fewer; warps that shared rows join in shared memory at the item's end.
// An item that one CTA sees whole is written out at once; one that several share
// leaves partials (unnormalised o, max, sum) and a second launch joins them.  With
// few keys there is neither list nor second launch: a cluster of CTAs takes an
// item and joins it through distributed shared memory.  Many rows go to the
// tensor cores (lf_paged_chunk_tc.cu), which has both ways too.
//
// What bounds it: with few tokens the cache's bytes and, for short ones, the call's
// fixed parts: 8 sequences of 5 new tokens at 512 positions (32 heads on 16 of
// 128) move 38 MB in 14.1 us, 5.7 of them the bytes; one launch in a cluster took
// the place of list and join at 17.9.  8 sequences of one token at 4096 positions:
// 268 MB in 46.6 us, 85 % of the copy rate.
//
// Masks.  Only a tile that some row of the item does not see whole is masked, by
// position, scores set to -inf.  A weight of 0 times a value that is not finite
// would still be NaN, so in such a tile those values are taken out of the product
// and added to the rows that do see them.
//
// P is rounded to the cache's type for the second product: both operands of an MMA
// have one type.  Its sum is taken before the rounding.
#include <cooperative_groups.h>

#include <algorithm>
#include <climits>
#include <type_traits>

#include "lf_paged_chunk.h"

namespace cg = cooperative_groups;

namespace lf {
namespace {

constexpr int CK_THREADS = 128, CK_CTAS_PER_SM = 2, CK_MAX_SEQS = 1024, CK_MAX_GROUP = 16;
constexpr int CK_MAX_TOKENS = 1 << 26;

template <typename T, int DH>
struct CkSmem {
    static constexpr int KT = tile_keys(DH);
    static constexpr int TILE = KT * DH * 2;  // bytes of K (or V) of one tile
    static constexpr int STAGES = DH == 32 ? 6 : 3;
    static constexpr int ML = 4 * 16 * 2 * 4;  // max and sum of the rows that the warps join
    static constexpr int CUM = (CK_MAX_SEQS + 4) * 4;
    static constexpr int BYTES = STAGES * 2 * TILE + ML + CUM;
    static_assert(4 * 16 * DH * 4 <= 2 * TILE, "the joined rows fit the stage");
    static_assert(STAGES >= 2 && 64 * 8 <= CUM, "a cluster's partials have their places");
};

// A 16-bit value is infinite or NaN.
template <typename T>
__device__ __forceinline__ bool odd_one(uint32_t h) {
    constexpr uint32_t e = std::is_same<T, __half>::value ? 0x7c00u : 0x7f80u;
    return (h & e) == e;
}
// One of a word's two is.
template <typename T>
__device__ __forceinline__ bool odd_word(uint32_t w) {
    constexpr uint32_t one = std::is_same<T, __half>::value ? 0x04000400u : 0x00800080u;  // (carries out of a full exponent)
    return (((w & 0x7fff7fffu) + one) & 0x80008000u) != 0;
}

// WR warps side by side in rows, 4 / WR in keys: items of up to 16 WR rows.
template <typename T, int DH, int WR>
class ChunkWalker {
  public:
    __device__ ChunkWalker(const ChunkArgs &args, uint8_t *smem) : a(args) {
        stage0 = smem;
        ml = reinterpret_cast<float2 *>(smem + L::STAGES * 2 * L::TILE);
        cum = reinterpret_cast<int *>(smem + L::STAGES * 2 * L::TILE + L::ML);
        tid = threadIdx.x;
        warp = tid >> 5;
        lane = tid & 31;
    }

    __device__ void run() {
        const int total = chunk_plan<KT>(a, cum);
        const Shares sh(total, gridDim.x);
        const int cta = blockIdx.x;
        if (tid == 0) a.joins[cta].parts = 0;
        if (cta >= min(total, (int)gridDim.x)) return;
        const int u0 = sh.begin(cta), u1 = sh.begin(cta + 1), n = u1 - u0;
        ChunkWork work = chunk_place<KT>(a, cum, u0), load = work;
        prepare(load);
        int loaded = 0;
        auto fetch_next = [&] {
            if (loaded < n) {
                fetch(loaded % L::STAGES);
                if (loaded + 1 < n) {
                    chunk_advance<KT>(a, cum, load);
                    prepare(load);
                }
            }
            ++loaded;
            cp_async_commit();
        };
        for (int i = 0; i < L::STAGES - 1; ++i) fetch_next();
        bool fresh = true, whole = work.tile == 0;  // whole: this CTA has begun the item
        for (int i = 0; i < n; ++i) {
            if (fresh) begin(work);
            fetch_next();
            asm volatile("cp.async.wait_group %0;" ::"n"(L::STAGES - 1) : "memory");
            __syncthreads();
            const bool ends = work.tile + 1 == work.tiles, last = i + 1 == n || ends;
            tile(work, last, i % L::STAGES, whole && ends, 2 * cta + (whole ? 1 : 0));
            __syncthreads();  // the stage may be written again
            if (i + 1 == n) {
                if (tid == 0) a.joins[cta] = chunk_join(a, work, sh, cta, u1, work.tile + 1, whole);
            } else {
                fresh = chunk_advance<KT>(a, cum, work);
                if (fresh) whole = true;
            }
        }
    }

    // One item by the CTAs of a cluster, result and all: each takes an equal share of its
    // tiles, and all join the partials through distributed shared memory.
    __device__ void run_direct() {
        cg::cluster_group cl = cg::this_cluster();
        const int parts = (int)cl.num_blocks(), part = (int)cl.block_rank();
        ChunkWork w;
        if (!chunk_item<KT>(a, quotient(blockIdx.x, parts), w)) return;  // (the whole cluster: fewer row tiles than the grid allows for)
        const Shares sh(w.tiles, parts);
        const int t0 = part < w.tiles ? sh.begin(part) : 0, n = part < w.tiles ? sh.begin(part + 1) - t0 : 0;
        w.tile = t0;
        ChunkWork load = w;
        auto fetch_next = [&](int i) {
            if (i < n) {
                prepare(load);
                fetch(i % L::STAGES);
                ++load.tile;
            }
            cp_async_commit();
        };
        for (int i = 0; i < L::STAGES - 1; ++i) fetch_next(i);
        if (n > 0) begin(w);
        for (int i = 0; i < n; ++i) {
            fetch_next(i + L::STAGES - 1);
            asm volatile("cp.async.wait_group %0;" ::"n"(L::STAGES - 1) : "memory");
            __syncthreads();
            tile<true>(w, i + 1 == n, i % L::STAGES, false, 0);
            __syncthreads();
            ++w.tile;
        }
        // this CTA's partial lies in shared memory (finish); an empty share leaves nothing
        const int rows = w.toks * a.group;
        float *mine = direct_o();
        float2 *stat = direct_ml();
        if (n == 0) {
            for (int x = tid; x < rows * DH; x += CK_THREADS) mine[x] = 0.f;
            for (int x = tid; x < rows; x += CK_THREADS) stat[x] = make_float2(-INFINITY, 0.f);
        }
        if (parts > 1)
            cl.sync();
        else
            __syncthreads();
        const int quads = rows * (DH / 4), per = (quads + parts - 1) / parts;
        for (int x = part * per + tid; x < min(quads, (part + 1) * per); x += CK_THREADS) {
            const int row = x / (DH / 4), c = (x % (DH / 4)) * 4;
            float2 y[8];
            float4 v[8];
            float mx = -INFINITY;
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (k < parts) {
                    y[k] = parts > 1 ? *cl.map_shared_rank(stat + row, k) : stat[row];
                    v[k] = *reinterpret_cast<const float4 *>(parts > 1 ? cl.map_shared_rank(mine + row * DH + c, k)
                                                                       : mine + row * DH + c);
                    mx = fmaxf(mx, y[k].x);
                }
            const float off = mx == -INFINITY ? 0.f : mx;
            float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
            float sl = 0.f;
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (k < parts) {
                    const float f = ex2(y[k].x - off);
                    s.x += f * v[k].x;
                    s.y += f * v[k].y;
                    s.z += f * v[k].z;
                    s.w += f * v[k].w;
                    sl += f * y[k].y;
                }
            const float inv = inverse(sl);
            const int tok = quotient(row, a.group), head = w.h * a.group + row - tok * a.group;
            const long long q = w.ch.row0 + w.tok + tok;
            *reinterpret_cast<uint2 *>(static_cast<T *>(a.out) + q * a.ld_out + (long long)head * DH + c) =
                make_uint2(pack2<T>(s.x * inv, s.y * inv), pack2<T>(s.z * inv, s.w * inv));
            if (c == 0 && a.lse) a.lse[q * a.n_q + head] = mx * 0.69314718055994530942f + logf(sl);
        }
        if (parts > 1) cl.sync();  // nobody leaves while its partial is read
    }

  private:
    using L = CkSmem<T, DH>;
    static constexpr int KT = L::KT, WK = 4 / WR, NB = KT / (16 * WK);  // NB blocks of 16 keys per warp
    const ChunkArgs &a;
    uint8_t *stage0;
    float2 *ml;
    int *cum;
    int tid, warp, lane;
    // the tile to be fetched next: element offsets of rows lane + 32 i (-1: no such key)
    long long row_off[KT / 32];
    // running state of this warp's 16 rows (lane 4 g + t: rows g and g + 8)
    uint32_t qf[DH / 16][4];
    float o[DH / 8][4];
    float m[2], l[2];
    int pos[2];  // their tokens' positions; INT_MIN: no such row

    // element offset of position j of w's KV head in K and V, -1 for a page outside the cache
    __device__ long long offset_of(const ChunkWork &w, int j) const {
        const int page = a.kv.table[(long long)w.b * a.kv.max_pages + (j >> a.kv.ps_log2)];
        return page >= 0 && page < a.kv.n_pages
                   ? page * a.kv.page_stride +
                         ((((long long)w.h << a.kv.ps_log2) + (j & ((1 << a.kv.ps_log2) - 1))) * DH)
                   : -1;
    }

    // Looks up the pages of w's tile.
    __device__ void prepare(const ChunkWork &w) {
        bool bad = false;
#pragma unroll
        for (int i = 0; i < KT / 32; ++i) {
            const int j = (w.kt0 + w.tile) * KT + lane + 32 * i;
            const bool key = j >= w.k.lo && j < w.k.hi;
            row_off[i] = -1;
            if (key) {
                row_off[i] = offset_of(w, j);
                bad |= row_off[i] < 0;
            }
        }
        if (bad) atomicExch(a.err, 1u);
    }

    // Starts the copies of the prepared tile into stage s; keys outside the item are zeros.
    __device__ void fetch(int s) {
        constexpr int CH = DH / 8;           // 16-byte chunks per row
        constexpr int RP = CK_THREADS / CH;  // rows per pass
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

    // A new item: its queries, straight from global memory (rows past the item's are zero).
    __device__ void begin(const ChunkWork &w) {
        const int rows = w.toks * a.group, wr = warp % WR, g = lane >> 2, t = lane & 3;
        const T *base[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int row = wr * 16 + g + 8 * r;
            base[r] = nullptr;
            pos[r] = INT_MIN;
            if (row < rows) {
                const int tok = quotient(row, a.group);
                base[r] = static_cast<const T *>(a.q) + (long long)(w.ch.row0 + w.tok + tok) * a.ld_q +
                          (long long)(w.h * a.group + row - tok * a.group) * DH;
                pos[r] = w.ch.base + w.tok + tok;
            }
        }
#pragma unroll
        for (int kk = 0; kk < DH / 16; ++kk)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const T *q = base[i & 1];
                qf[kk][i] = q ? *reinterpret_cast<const uint32_t *>(q + kk * 16 + (i >> 1) * 8 + 2 * t) : 0u;
            }
#pragma unroll
        for (int i = 0; i < DH / 8; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) o[i][j] = 0.f;
        m[0] = m[1] = -INFINITY;
        l[0] = l[1] = 0.f;
    }

    // This lane's row r sees position j.
    __device__ bool sees(int r, int j) const {
        return j <= pos[r] && (a.window == 0 || j > (long long)pos[r] - a.window);
    }

    // Where a CTA of run_direct leaves its partial, the same place in all: o in the ring's first stage (no copy is under
    // way by then), the statistics where the list's table would be.
    __device__ float *direct_o() const { return reinterpret_cast<float *>(stage0); }
    __device__ float2 *direct_ml() const { return reinterpret_cast<float2 *>(cum); }

    // One tile of the item.  DIRECT: the item's end is a partial in shared memory.
    template <bool DIRECT = false>
    __device__ void tile(const ChunkWork &w, bool last, int s, bool whole, int slot) {
        const int wk = warp / WR, t = lane & 3;
        const int j0 = (w.kt0 + w.tile) * KT;  // position of the tile's first key
        const uint32_t ks = smem_u32(stage0 + (size_t)s * 2 * L::TILE), vs = ks + L::TILE;
        // every row sees every key: up to the first token, from the last one's window on
        const int first = w.ch.base + w.tok, end = first + w.toks - 1;
        const bool full = j0 + KT - 1 <= first && j0 >= w.k.lo && (a.window == 0 || j0 > (long long)end - a.window);
        bool odd = false;
        if (!full) {  // values that are not finite leave the product
            uint8_t *v = stage0 + (size_t)s * 2 * L::TILE + L::TILE;
            for (int x = tid; x < L::TILE / 16; x += CK_THREADS) {
                uint4 y = reinterpret_cast<uint4 *>(v)[x];
                if (!(odd_word<T>(y.x) | odd_word<T>(y.y) | odd_word<T>(y.z) | odd_word<T>(y.w))) continue;
                uint32_t *p = reinterpret_cast<uint32_t *>(&y);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (odd_one<T>(p[i] & 0xffffu)) p[i] &= 0xffff0000u;
                    if (odd_one<T>(p[i] >> 16)) p[i] &= 0xffffu;
                }
                reinterpret_cast<uint4 *>(v)[x] = y;
                odd = true;
            }
            odd = __syncthreads_or(odd);
        }
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
        if (!full) {
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int x = 0; x < 2; ++x)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (!sees(i >> 1, j0 + (nb * WK + wk) * 16 + x * 8 + 2 * t + (i & 1))) sc[2 * nb + x][i] = -INFINITY;
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
        if (odd) add_odd(w, j0, wk, t);
        if (last) finish<DIRECT>(w, s, whole, slot);
    }

    // Adds the tile's values that are not finite to the rows that see them.
    __device__ __forceinline__ void add_odd(const ChunkWork &w, int j0, int wk, int t) {
#pragma unroll 1
        for (int key = 0; key < KT; ++key) {
            const int j = j0 + key;
            if ((key / 16) % WK != wk || j < w.k.lo || j >= w.k.hi) continue;
            const long long off = offset_of(w, j);
            if (off < 0) continue;
            const uint16_t *v = static_cast<const uint16_t *>(a.kv.v) + off;
#pragma unroll
            for (int i = 0; i < DH / 8; ++i)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const uint16_t h = v[8 * i + 2 * t + x];
                    if (!odd_one<T>(h)) continue;
                    const float f = (float)*reinterpret_cast<const T *>(&h);
                    if (sees(0, j)) o[i][x] += f;
                    if (sees(1, j)) o[i][2 + x] += f;
                }
        }
    }

    // The item's end in this CTA: the result where it has seen all of it, a partial otherwise; warps with the same rows
    // joined.
    template <bool DIRECT>
    __device__ void finish(const ChunkWork &w, int s, bool whole, int slot) {
        const int wr = warp % WR, g = lane >> 2, t = lane & 3, rows = w.toks * a.group;
        const long long at = (long long)slot * a.slot_rows;
        float *dst = a.part_o + at * DH;
        float2 *dst_ml = a.part_ml + at;
        auto result = [&](int row, int c, float x, float y, float mx, float sum) {  // dims c, c + 1
            if constexpr (DIRECT) {
                *reinterpret_cast<float2 *>(direct_o() + row * DH + c) = make_float2(x, y);
                if (c == 0) direct_ml()[row] = make_float2(mx, sum);
            } else if (whole) {
                const int tok = row / a.group, head = w.h * a.group + row - tok * a.group;
                const long long q = w.ch.row0 + w.tok + tok;
                const float inv = inverse(sum);
                *reinterpret_cast<uint32_t *>(static_cast<T *>(a.out) + q * a.ld_out + (long long)head * DH + c) =
                    pack2<T>(x * inv, y * inv);
                if (c == 0 && a.lse) a.lse[q * a.n_q + head] = mx * 0.69314718055994530942f + logf(sum);
            } else {
                *reinterpret_cast<float2 *>(dst + (long long)row * DH + c) = make_float2(x, y);
                if (c == 0) dst_ml[row] = make_float2(mx, sum);
            }
        };
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
            l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
        }
        if constexpr (WK == 1) {
            if (DIRECT) __syncthreads();  // every warp has read the keys and values
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int row = wr * 16 + g + 8 * r;
                if (row >= rows) continue;
#pragma unroll
                for (int i = 0; i < DH / 8; ++i) result(row, 8 * i + 2 * t, o[i][2 * r], o[i][2 * r + 1], m[r], l[r]);
            }
        } else {
            __syncthreads();  // every warp has read this stage's keys and values
            // row r of warp w at (w * 16 + r) * DH, its columns permuted by the row (8 rows of a warp write 8 bank groups)
            float *red = reinterpret_cast<float *>(stage0 + (size_t)(DIRECT ? 1 : s) * 2 * L::TILE);
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
            for (int x = tid; x < rows * (DH / 2); x += CK_THREADS) {
                const int row = x / (DH / 2), c = (x % (DH / 2)) * 2;
                float mx = -INFINITY;  // over the key shares k: warp row / 16 + k * WR
#pragma unroll
                for (int k = 0; k < WK; ++k) mx = fmaxf(mx, ml[row + k * WR * 16].x);
                const float off = mx == -INFINITY ? 0.f : mx;
                float sx = 0.f, sy = 0.f, sl = 0.f;
#pragma unroll
                for (int k = 0; k < WK; ++k) {
                    const float2 y = ml[row + k * WR * 16];
                    const float f = ex2(y.x - off);
                    const float2 v = *reinterpret_cast<const float2 *>(red + (row + k * WR * 16) * DH +
                                                                       col(row, c & ~7) + (c & 7));
                    sx += f * v.x;
                    sy += f * v.y;
                    sl += f * y.y;
                }
                result(row, c, sx, sy, mx, sl);
            }
        }
    }
};

template <typename T, int DH, int WR>
__global__ void __launch_bounds__(CK_THREADS, CK_CTAS_PER_SM) paged_chunk_kernel(const ChunkArgs a) {
    extern __shared__ __align__(128) uint8_t ck_smem[];
    pdl_wait();
    pdl_trigger();
    ChunkWalker<T, DH, WR>(a, ck_smem).run();
}

// A cluster per item and no other launch: for few keys.
template <typename T, int DH, int WR>
__global__ void __launch_bounds__(CK_THREADS, CK_CTAS_PER_SM) paged_chunk_direct(const ChunkArgs a) {
    extern __shared__ __align__(128) uint8_t ck_smem[];
    pdl_wait();
    pdl_trigger();
    ChunkWalker<T, DH, WR>(a, ck_smem).run_direct();
}

// The items that several CTAs share, half a warp to a row: block (c, y) takes rows
// 16 y .. 16 y + 15 of the item that CTA c began and did not end, its partials in the
// list's order, several in flight.
constexpr int CJ_THREADS = 256, CJ_ROWS = CJ_THREADS / 16;
template <typename T, int DH>
__global__ void __launch_bounds__(CJ_THREADS) paged_chunk_join(const ChunkArgs a) {
    constexpr int V = DH / 16, U = 4;  // values per lane; partials in flight
    const int c = blockIdx.x, lane = threadIdx.x & 15, row = blockIdx.y * CJ_ROWS + (threadIdx.x >> 4);
    pdl_wait();
    pdl_trigger();
    const ChunkArgs::Join j = a.joins[c];
    if (j.parts == 0 || row >= j.rows) return;
    // partial p of the item: the CTA that begins it leaves it second, those behind first
    auto at = [&](int p) { return (long long)(p == 0 ? 2 * c + 1 : 2 * (c + p)) * a.slot_rows + row; };
    float acc[V], mx = -INFINITY, sum = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = 0.f;
    for (int p0 = 0; p0 < j.parts; p0 += U) {
        float2 y[U];
        float v[U][V];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const long long s = at(min(p0 + u, j.parts - 1));
            y[u] = a.part_ml[s];
            const float *d = a.part_o + s * DH + lane * V;
#pragma unroll
            for (int i = 0; i < V; i += V >= 4 ? 4 : V) {
                if constexpr (V >= 4)
                    *reinterpret_cast<float4 *>(v[u] + i) = *reinterpret_cast<const float4 *>(d + i);
                else
                    *reinterpret_cast<float2 *>(v[u] + i) = *reinterpret_cast<const float2 *>(d + i);
            }
        }
        float mn = mx;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (p0 + u >= j.parts) y[u] = make_float2(-INFINITY, 0.f);
            mn = fmaxf(mn, y[u].x);
        }
        const float off = mn == -INFINITY ? 0.f : mn, f0 = ex2(mx - off);
        mx = mn;
        sum *= f0;
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] *= f0;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (p0 + u >= j.parts) break;
            const float f = ex2(y[u].x - off);
            sum += f * y[u].y;
#pragma unroll
            for (int i = 0; i < V; ++i) acc[i] += f * v[u][i];
        }
    }
    const int tok = row / a.group, head = j.head * a.group + row - tok * a.group;
    const long long q = j.row0 + tok;
    const float inv = inverse(sum);
    uint32_t h[V / 2];
#pragma unroll
    for (int i = 0; i < V; i += 2) h[i / 2] = pack2<T>(acc[i] * inv, acc[i + 1] * inv);
    uint32_t *dst = reinterpret_cast<uint32_t *>(static_cast<T *>(a.out) + q * a.ld_out + (long long)head * DH + lane * V);
    if constexpr (V == 8)
        *reinterpret_cast<uint4 *>(dst) = make_uint4(h[0], h[1], h[2], h[3]);
    else if constexpr (V == 4)
        *reinterpret_cast<uint2 *>(dst) = make_uint2(h[0], h[1]);
    else
        *dst = h[0];
    if (a.lse && lane == 0) a.lse[q * a.n_q + head] = mx * 0.69314718055994530942f + logf(sum);
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

// The tensor-core kernel takes head_dim 64 and 128, pages of at least 8 positions
// (a TMA box) and page strides that a tensor map can hold (2^40 bytes).
bool tc_fits(const PagedView &v) { return v.head_dim >= 64 && v.ps_log2 >= 3 && v.page_stride < (1ll << 38); }

// Rows of a sequence and KV head, on average.
long long rows_of(const ChunkArgs &a) { return ((long long)a.n_tokens * a.group + a.kv.n_seqs - 1) / a.kv.n_seqs; }

// Items of 16, 32 or 64 rows on warp-level MMAs, as the sequences have, or of 256 on the tensor cores.
void shape(ChunkArgs &a, bool tc, int n_sm) {
    const long long rows = rows_of(a);
    a.tc = tc;
    a.slot_rows = tc ? kTcRows : rows <= 16 ? 16 : rows <= 32 ? 32 : 64;
    a.toks = tc ? 2 * (128 / a.group) : a.slot_rows / a.group;  // (a 128-row tile holds whole tokens)
    a.grid = tc ? n_sm : n_sm * CK_CTAS_PER_SM;
}

// How a call on warp-level MMAs would run: items, tiles of keys each, and the CTAs to an item that take the fewest tiles
// one after another (every further wave of CTAs costs its start, about six tiles).
struct MmaPlan {
    long long items, tiles, each;  // each: tiles one after another of the direct kernel, starts of further waves included
    int parts;
    bool one_wave;
};
MmaPlan mma_plan(const ChunkArgs &a, int n_sm) {
    MmaPlan p;
    const int kt = tile_keys(a.kv.head_dim), toks = (a.n_tokens + a.kv.n_seqs - 1) / a.kv.n_seqs;  // tokens of a sequence
    const int bound = a.window > 0 ? std::min(a.window + a.toks, a.max_len) : a.max_len;
    const long long ctas = (long long)n_sm * CK_CTAS_PER_SM;
    p.tiles = bound / kt + 1;
    p.items = (long long)a.kv.n_seqs * a.kv.n_kv * ((toks + a.toks - 1) / a.toks);
    p.each = LLONG_MAX;
    for (int k = 1; k <= 8; k *= 2) {
        const long long room = k > 2 ? ctas * 7 / 8 : ctas;  // (larger clusters do not fill every SM of a GPC)
        const long long waves = (p.items * k + room - 1) / room, t = waves * ((p.tiles + k - 1) / k + 6) - 6;
        if (t < p.each) p.each = t, p.parts = k, p.one_wave = waves == 1;
    }
    return p;
}

// CTAs to an item of the direct kernel, 0 for the list and its join.  The list is even however the lengths are, but its
// table, its partials and the second launch take longer than six key tiles of a CTA, and the more CTAs share an item, the
// longer its join: about 0.3 tiles for each.  us, list | clusters of 1, 2, 4, 8, 32 heads on 16 of 128, one new token:
//   1 sequence   512 keys  10.2 | 13.1  9.8  8.2  7.7    4096 keys  22.9 | 63.8 35.3 21.0 15.7
//   8 sequences  512 keys  15.8 | 15.3 13.4 18.4 27.3    4096 keys  49.4 | 70.9 46.6 52.3 61.2
// and 16 rows (8 new tokens), 32 sequences: 512 keys 39.7 | 39.0 51.0 70.8 124, 4096 keys 171 | 176 190 189 236.
// Over 404 sizes this rule and tc_pays' together lose 2 % to the best choice of each.  These were batches of equal chunks and
// lengths, without windows; all the host knows of others is their mean, see tc_pays.
int direct_parts(const ChunkArgs &a, const MmaPlan &p, int n_sm) {
    const long long ctas = (long long)n_sm * CK_CTAS_PER_SM;
    return p.each * 10 <= p.items * p.tiles * 10 / ctas + 60 + 3 * std::min(p.tiles, ctas / p.items) ? p.parts : 0;
}

// CTAs to an item of the tensor-core kernel in a cluster, 0 for the list and its join.  A cluster's start, end and join take
// as long as 8, 9 or 12 key tiles of a CTA with 1, 2 or 4 CTAs; those of the list as 19, and 4 for each item of a CTA, and its
// tiles a tenth longer (their partials go through L2).  But the list is even, and of clusters the item with the most keys
// sets the time; several waves come only of CTAs that take an item each, whose ends overlap.  us, list | clusters
// of 1, 2, 4, one sequence, 32 heads on 16 of 128 (16 items for 128 new tokens):
//    128 new, 128 keys  18.7 | 10.9 12.7 14.5    640 keys  23.6 | 16.4 15.1 16.3    16128 keys  46.6 | 180 97 58
//    256 new, 256 keys  21.6 | 12.7 13.0 14.5   3840 keys  34.8 | 50.8 33.3 27.1    16256 keys  66.2 | 178 98 59
//    512 new, 512 keys  24.6 | 15.2 15.4 29.6   4096 keys  43.8 | 53.8 36.1 52.4    16512 keys   111 | 181 102 117
//   1024 new, 1024 keys 33.4 | 23.1 32.6 62.2   4608 keys  67.0 | 62.0 70.5 102     17024 keys   207 | 190 205 235
// (Equal chunks and lengths: 200 sizes.)
// Clusters of 8 find room for eight at most and were the best of one size in a hundred.
int tc_parts(const ChunkArgs &a, int n_sm) {
    const long long items = chunk_items(a);
    const int toks = (a.n_tokens + a.kv.n_seqs - 1) / a.kv.n_seqs;  // tokens of a sequence
    const int bound = a.window > 0 ? std::min(a.window + a.toks, a.max_len) : a.max_len;
    const long long tiles = bound / kTcKeys + 1, mean = a.window > 0 ? tiles : std::max(1ll, tiles - toks / (2 * kTcKeys));
    const long long even = (long long)a.kv.n_seqs * a.kv.n_kv * ((toks + a.toks - 1) / a.toks);
    long long best = 190 + 11 * even * mean / n_sm + 40 * even / n_sm;
    int parts = 0;
    const int fixed[3] = {80, 90, 120};
    for (int i = 0, k = 1; i < 3; ++i, k *= 2) {
        const long long room = (k > 1 ? n_sm * 7 / 8 : n_sm) / k;
        long long t = fixed[i] + 10 * ((tiles + k - 1) / k);
        if (even <= room)
            t += items > room ? t / 2 : 0;  // (chunks of uneven lengths may take a second wave)
        else if (k == 1)
            t = (items + n_sm - 1) / n_sm * fixed[0] + 10 * items * mean / n_sm + 5 * tiles;
        else
            continue;
        if (t < best) best = t, parts = k;
    }
    return parts;
}

// The tensor cores pay beyond 64 rows of a sequence and KV head, with many sequences from 41 on, but not where one wave of
// the direct kernel has three key tiles to a CTA at most (two where an item has one CTA); with few sequences and 41 to 64
// rows from 4096 keys on; and below 256 keys (with over 256 rows 512) wherever clusters take the items (64 rows of one
// sequence, 32 keys: 9.0 us where the direct kernel takes 13.8; 512 rows, 356 keys: 14.2 and 19.5).  us, the better of list and clusters | tensor cores by their list, 32 heads
// on 16 of 128:
//   1 sequence,    64 rows   512 keys  12.2 | 17.5   4096  26.7 | 25.0     128 rows  512  12.7 | 18.6   4096  26.9 | 26.1
//   8 sequences,   16 rows   512 keys  15.3 | 21.9   4096  48.4 | 57.2      64 rows  512  22.8 | 23.7   4096  74.7 | 59.5
//                 128 rows   512 keys  33.7 | 26.2   4096 130.7 | 63.8
//   32 sequences,  16 rows   512 keys  39.0 | 50.0   4096 171   | 180       32 rows  512  48.3 | 51.5   4096 187   | 184
//                  64 rows   512 keys  58.9 | 52.1   4096 246   | 187
// and 24 on 8 of 64: 1 sequence, 96 rows, 512 keys 10.0 | 13.8; 8 sequences, 48 rows, 4096 keys 28.9 | 28.4, 512 keys
// 11.1 | 15.5; 32 sequences, 48 rows, 4096 keys 81.8 | 74.1, 512 keys 22.8 | 26.3.
// One choice for the batch, by the mean rows of a sequence, those without new tokens among them: a chunk of 512 at 3584 (35
// us alone) takes 260 us on warp-level MMAs in a batch of 64 places whose others are without new tokens, and beside 63
// single tokens at 512 to 3584 (164 us by themselves) 270.
bool tc_pays(const ChunkArgs &a, int n_sm) {
    const long long rows = rows_of(a);
    if (!tc_fits(a.kv) || rows <= 40) return false;
    const int bound = a.window > 0 ? std::min(a.window + a.toks, a.max_len) : a.max_len;
    ChunkArgs t = a;
    shape(t, true, n_sm);
    if (bound < (rows > 256 ? 4 : 2) * kTcKeys && tc_parts(t, n_sm) > 0) return true;
    if (rows <= 64 && (long long)a.kv.n_seqs * a.kv.n_kv < 48 && bound < 4096) return false;
    ChunkArgs m = a;
    shape(m, false, n_sm);
    const MmaPlan p = mma_plan(m, n_sm);
    return !(p.one_wave && (p.parts > 1 ? (p.tiles + p.parts - 1) / p.parts <= 3 : p.tiles <= 2));
}

struct CkWs {
    size_t ml, o, bytes;
};
CkWs ck_layout(const ChunkArgs &a) {
    CkWs w;
    const size_t rows = 2 * (size_t)a.grid * a.slot_rows;
    w.ml = al256((size_t)a.grid * sizeof(ChunkArgs::Join));
    w.o = w.ml + al256(rows * sizeof(float2));
    w.bytes = w.o + rows * a.kv.head_dim * sizeof(float);
    return w;
}

lf_status check_chunk(const lf_paged_kv *kv, int n_q_heads, int n_tokens, PagedView *v) {
    const lf_status st = paged_view(kv, v);
    if (st != LF_OK) return st;
    if (n_q_heads < 1 || n_q_heads % v->n_kv || n_tokens < 0) return LF_ERR_INVALID_ARG;
    if ((v->head_dim != 32 && v->head_dim != 64 && v->head_dim != 128) || n_q_heads / v->n_kv > CK_MAX_GROUP ||
        v->n_seqs > CK_MAX_SEQS || n_tokens > CK_MAX_TOKENS)
        return LF_ERR_UNSUPPORTED;
    return LF_OK;
}

// The largest a call of up to this many tokens needs (fewer tokens may take smaller items, never larger ones).
size_t ck_bytes(ChunkArgs a, int n_sm) {
    shape(a, false, n_sm);
    size_t n = ck_layout(a).bytes;
    if (tc_fits(a.kv) && rows_of(a) > 40) {
        shape(a, true, n_sm);
        n = std::max(n, ck_layout(a).bytes);
    }
    return n;
}

template <typename T, int DH, int WR>
bool launch_rows(const ChunkArgs &a, int direct, cudaStream_t st) {
    constexpr int smem = CkSmem<T, DH>::BYTES;
    if (!direct)
        return set_smem_once<paged_chunk_kernel<T, DH, WR>>(smem) &&
               launch_pdl(paged_chunk_kernel<T, DH, WR>, a.grid, CK_THREADS, smem, st, a);
    return set_smem_once<paged_chunk_direct<T, DH, WR>>(smem) &&
           launch_pdl_cluster(paged_chunk_direct<T, DH, WR>, (unsigned)direct, dim3((unsigned)(chunk_items(a) * direct)), CK_THREADS, smem, st, a);
}

template <typename T, int DH>
lf_status launch_chunk(const ChunkArgs &a, int direct, cudaStream_t st) {
    bool ok = false;
    if constexpr (DH >= 64) {
        if (a.tc) {
            const lf_status ts = paged_chunk_tc(a, std::is_same<T, __half>::value ? LF_F16 : LF_BF16, direct, st);
            if (ts != LF_OK) return ts;
            ok = true;
        }
    }
    if (!a.tc)
        ok = a.slot_rows == 16   ? launch_rows<T, DH, 1>(a, direct, st)
             : a.slot_rows == 32 ? launch_rows<T, DH, 2>(a, direct, st)
                                 : launch_rows<T, DH, 4>(a, direct, st);
    if (ok && !direct)
        ok = launch_pdl(paged_chunk_join<T, DH>, dim3((unsigned)a.grid, (unsigned)(a.slot_rows / CJ_ROWS)), CJ_THREADS, 0, st, a);
    return ok ? LF_OK : LF_ERR_CUDA;
}

#ifdef LF_DEBUG
std::atomic<int> g_lose_cta{-1}, g_lose_warp{0}, g_lose_wait{0};
#endif

template <typename T>
lf_status launch_chunk_dim(const ChunkArgs &a, int direct, cudaStream_t st) {
    return a.kv.head_dim == 32   ? launch_chunk<T, 32>(a, direct, st)
           : a.kv.head_dim == 64 ? launch_chunk<T, 64>(a, direct, st)
                                 : launch_chunk<T, 128>(a, direct, st);
}

}  // namespace
}  // namespace lf

extern "C" size_t lf_attn_paged_chunk_workspace(const lf_paged_kv *kv, int n_q_heads, int n_tokens) {
    lf::ChunkArgs a = {};
    if (lf::check_chunk(kv, n_q_heads, n_tokens, &a.kv) != LF_OK) return 0;
    a.group = n_q_heads / a.kv.n_kv;
    a.n_tokens = n_tokens;
    const int n_sm = lf::sm_count();
    return n_sm ? lf::ck_bytes(a, n_sm) : 0;
}

extern "C" lf_status lf_attn_paged_chunk(const lf_paged_kv *kv, const void *q_device, int64_t ld_q, void *out_device,
                                         int64_t ld_out, float *lse_device, int n_q_heads,
                                         const int32_t *starts_device, int n_tokens, const int32_t *lens_device,
                                         int max_len, int window, float scale, void *workspace_device,
                                         size_t workspace_bytes, uint32_t *err_device, void *cuda_stream) {
    lf::ChunkArgs a = {};
    const lf_status cs = lf::check_chunk(kv, n_q_heads, n_tokens, &a.kv);
    if (cs != LF_OK) return cs;
    const int64_t row = (int64_t)n_q_heads * kv->head_dim, cap = (int64_t)kv->max_pages * kv->page_size;
    auto off4 = [](const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) != 0; };
    if (!q_device || !out_device || !starts_device || !lens_device || !workspace_device || !err_device ||
        !lf::aligned16(q_device) || !lf::aligned16(out_device) || off4(lse_device) || off4(starts_device) ||
        off4(lens_device) || off4(err_device) || (reinterpret_cast<uintptr_t>(workspace_device) & 255u) || ld_q < row ||
        ld_out < row || ld_q % 8 || ld_out % 8 || (q_device == out_device && ld_q != ld_out) || max_len < 0 ||
        max_len > cap || window < 0 || !(scale > 0.f && scale * lf::kLog2e < INFINITY))
        return LF_ERR_INVALID_ARG;
    a.group = n_q_heads / a.kv.n_kv;
    a.n_tokens = n_tokens;
    const int n_sm = lf::sm_count();
    if (!n_sm) return LF_ERR_CUDA;
    if (workspace_bytes < lf::ck_bytes(a, n_sm)) return LF_ERR_INVALID_ARG;
    a.max_len = max_len;
    a.window = window >= max_len ? 0 : window;  // (every position lies less than max_len back)
    lf::shape(a, lf::tc_pays(a, n_sm), n_sm);
    // tiles are counted in 32 bits: those of the items that the new tokens can have (a sequence without any has none)
    const int kt = a.tc ? lf::kTcKeys : lf::tile_keys(kv->head_dim);
    const long long items = lf::chunk_items(a);
    if (items > INT_MAX || items * (max_len / kt + 2) > INT_MAX) return LF_ERR_UNSUPPORTED;
    if (n_tokens == 0) return LF_OK;
    const lf::CkWs w = lf::ck_layout(a);
    uint8_t *ws = static_cast<uint8_t *>(workspace_device);
    a.joins = reinterpret_cast<lf::ChunkArgs::Join *>(ws);
    a.part_ml = reinterpret_cast<float2 *>(ws + w.ml);
    a.part_o = reinterpret_cast<float *>(ws + w.o);
    a.q = q_device;
    a.out = out_device;
    a.lse = lse_device;
    a.ld_q = ld_q;
    a.ld_out = ld_out;
    a.n_q = n_q_heads;
    a.starts = starts_device;
    a.lens = lens_device;
    a.scale_log2 = scale * lf::kLog2e;
    a.err = err_device;
#ifdef LF_DEBUG
    a.lose_cta = lf::g_lose_cta;
    a.lose_warp = lf::g_lose_warp;
    a.lose_wait = lf::g_lose_wait;
#endif
    const int direct = a.tc ? lf::tc_parts(a, n_sm) : lf::direct_parts(a, lf::mma_plan(a, n_sm), n_sm);
    cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
    return kv->dtype == LF_F16 ? lf::launch_chunk_dim<__half>(a, direct, st)
                               : lf::launch_chunk_dim<__nv_bfloat16>(a, direct, st);
}

extern "C" lf_status lf_debug_chunk_wait(int cta, int warp, int nth) {
    if (cta < -1 || warp < 0 || warp > 9 || nth < 0) return LF_ERR_INVALID_ARG;
#ifdef LF_DEBUG
    lf::g_lose_cta = cta;
    lf::g_lose_warp = warp;
    lf::g_lose_wait = nth;
    return LF_OK;
#else
    return LF_ERR_UNSUPPORTED;
#endif
}
