// lf_attn_paged_chunk on the 5th-generation tensor cores (tcgen05 + TMA + TMEM), for
// chunks whose rows (token, query head) of one KV head are many.
//
// An item is two M = 128 row tiles of consecutive tokens of one sequence and KV head.
// Many items: the list of their tiles of 128 keys in even shares (lf_paged_chunk.h),
// one CTA per SM, and a join behind.  Few: a cluster of 1, 2 or 4 CTAs to an item, an
// equal share of its tiles each; at the end each softmax warp's 32 rows belong to one
// of the CTAs, which the others push their partials to (shared memory, where Q, K
// and V lay), so that nothing goes through L2 and nothing is launched behind.  Which
// of the two is taken, and both sides' times: tc_parts in lf_paged_chunk.cu.
// Per key tile and row tile x:
//   S = Q K^T into TMEM; the row tile's softmax warpgroup, a row per thread,
//   reads S, moves the row's running max (only when it grows by more than 2^8,
//   so P stays below 256), and writes P in the cache's type back over S;
//   O += P V with P as the A operand from TMEM.
// The two row tiles take turns: one's softmax runs under the other's products.  P is
// handed over in two pieces: the products with its first 96 keys run while the
// exponentials of the last 32 are still computed.
//
// K and V pages come by TMA (one box of min(page size, 128) positions x 64 dims
// each), double-buffered; V is read as it lies, [key][dim], as an MN-major B
// operand.  Tiles are cut at multiples of 128 positions, so boxes never cross a page;
// pages without a key of the item are loaded from outside the tensor, as zeros.
//
// Masks.  A tile that some row does not see whole has its scores masked by position.
// What lies behind the sequence's end in the last page, before a window's start, or
// is not finite would still reach the product as 0 times itself: in such a tile
// the first warpgroup zeroes those values in shared memory (a thread per key, before
// it hands over P), and at the item's end the values that are not finite are
// added to the rows that do see them.
//
// Q comes by TMA, a box of (64 dims, the group's heads, tokens): its rows lie as the
// products want them, and it loads under the item before.  Rows leave through
// shared memory, 64 bytes of a row to four lanes.  Both together took 512 new tokens
// at 3584 from 54 us to 45.
//
// What bounds it: over long keys the tensor cores (2 x 2048 new tokens at 14336, 64
// heads on 8 of 128, bf16: 961 us, 1672 TFLOP/s, their pipe 72 % full; in calls back to
// back the board's power, 1120 to 1150 us), else the items' starts and ends (512 at
// 3584: 35 us by clusters of two, 44 by the list, of which 11 were the join of 215
// pieces; its products take 17) and, with few rows to an item, the way of a tile
// from one product through the softmax to the next, 1.7 us (a mixed windowed
// batch, 144 items: 23.5 us by a CTA to each, 36 by the list).  Of a softmax warp's
// 168 registers 128 hold a row's scores.
//
// Tried: P's first piece of 64 or 32 keys, no better; shares of at least four tiles
// instead of two, slower for short keys; the key tiles of an item of one row tile in
// turn on both warpgroups, with a join of their sums at the end (36 us to 56 for
// a mixed batch, 1 to 9 us more for short keys).
//
// Every wait is bounded; a CTA that ran out of time flags it, lets its copies
// and products finish (bounded), frees its TMEM and exits.
#include <climits>

#include "lf_paged_chunk.h"
#include "lf_paged_tc.cuh"

namespace lf {
namespace {

constexpr int C_THREADS = 320;         // copy warp, MMA warp, 2 x 4 softmax warps
constexpr uint32_t C_TMEM_COLS = 512;  // S / P of row tile x at 128 x, O at 256 + 128 x
constexpr uint32_t C_O = 256;
constexpr int kLeast = 2;              // key tiles of a CTA, at least
constexpr int C_FIRST = 96;            // keys of P's first piece (a multiple of 32)
constexpr unsigned long long kChunkTimeoutNs = 2000000000ull;

// Every barrier completes once per use of what it guards, and no waiter can
// fall two phases behind, so parity waits are unambiguous.
struct CtShared {
    uint64_t bq[2];     // Q of row tile x loaded
    uint64_t bk0;       // K of the first tile loaded
    uint64_t bl[2];     // V of tile p and K of tile p + 1 loaded (p = 0, 2, .. and 1, 3, ..)
    uint64_t bf[2];     // done: the S products of tile p and the P V products of tile p - 1 (p = 0, 2, .. and 1, 3, ..)
    uint64_t bs[2];     // row tile x: S of the next tile computed (and its earlier P V done)
    uint64_t bp[2][2];  // row tile x: first and last piece of P written to TMEM (128 arrivals)
    uint64_t bo[2];     // row tile x: the last P V of an item done
    uint64_t bdone;     // every product this CTA issued is done (one commit at the end)
    uint32_t tmem;
    volatile int abort_;
    volatile int issued_;   // 1 once any product was issued (then bdone gets its commit)
    volatile int odd_[8];   // item it's masked tiles hold values that are not finite: odd_[it & 7] is it + 1
};

// A thread's waits.  (The limit counts from the first probe that fails: a wait that is over costs no look at the clock.)
struct CtWaits {
    CtShared &S;
    uint32_t *err;
#ifdef LF_DEBUG
    int lose;  // it gives up in this wait from here on
#endif
    __device__ __forceinline__ bool operator()(uint64_t *bar, uint32_t parity) {
#ifdef LF_DEBUG
        if (--lose == 0) return give_up();
#endif
        if (mbar_test_wait(bar, parity)) return true;
        const uint64_t deadline = global_timer_ns() + kChunkTimeoutNs;
        while (!mbar_try_wait(bar, parity)) {
            if (S.abort_) return false;
            if (global_timer_ns() > deadline) return give_up();
        }
        return true;
    }
    __device__ __forceinline__ bool give_up() {
        atomicExch(err, 2u);
        S.abort_ = 1;
        return false;
    }
};

// (x, y) * c + d and x + y, two values to an instruction
__device__ __forceinline__ float2 fma2(float2 x, float2 c, float2 d) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(r)
        : "l"(*reinterpret_cast<const uint64_t *>(&x)), "l"(*reinterpret_cast<const uint64_t *>(&c)),
          "l"(*reinterpret_cast<const uint64_t *>(&d)));
    return *reinterpret_cast<float2 *>(&r);
}
__device__ __forceinline__ float2 add2(float2 x, float2 y) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;"
        : "=l"(r)
        : "l"(*reinterpret_cast<const uint64_t *>(&x)), "l"(*reinterpret_cast<const uint64_t *>(&y)));
    return *reinterpret_cast<float2 *>(&r);
}

// Bits 15 and 31: of the two 16-bit values of a word, those that are infinite or NaN.
template <typename T>
__device__ __forceinline__ uint32_t odd_bits(uint32_t w) {
    constexpr uint32_t one = std::is_same<T, __half>::value ? 0x04000400u : 0x00800080u;  // (carries out of a full exponent)
    return ((w & 0x7fff7fffu) + one) & 0x80008000u;
}

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t y;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(y));
    return y;
}
__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t y;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(y));
    return y;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// The place in CTA `rank` of the cluster of a place in this one's shared memory, and stores there.
__device__ __forceinline__ uint32_t cluster_address(uint32_t mine, int rank) {
    uint32_t y;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(y) : "r"(mine), "r"(rank));
    return y;
}
__device__ __forceinline__ void cluster_store(uint32_t at, float2 v) {
    asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(at), "f"(v.x), "f"(v.y) : "memory");
}
__device__ __forceinline__ void cluster_store(uint32_t at, float4 v) {
    asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(at), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w) : "memory");
}

template <int DH>
struct CtSmem {
    static constexpr int HALVES = DH / 64;
    static constexpr int TILE = HALVES * T_HALF;  // one row tile of Q, one buffer of K or V
    static constexpr int Q = 0, K = 2 * TILE, V = 4 * TILE, TILES = 6 * TILE;
    static constexpr int CUM = TILES + 256;
    static constexpr int OUT = CUM + (1024 + 4) * 4;  // 32 rows of 64 bytes of each softmax warp, on their way out
    static constexpr int OUT_ROW = 80;                // (apart so that 8 rows lie in 8 different groups of banks)
    static constexpr int WORK = OUT + 8 * 32 * OUT_ROW;  // two items of each softmax warp
    static constexpr int BYTES = WORK + 16 * (int)sizeof(ChunkWork) + 1024;
    static_assert(sizeof(CtShared) <= 256, "the barriers' place");
    static_assert(6 * DH * 128 <= TILES && 6 * 32 * 8 <= 1024 * 4, "a cluster's partials and statistics");
};

// CL: a cluster to an item instead of the list.
template <typename T, int DH, bool CL>
__global__ void __launch_bounds__(C_THREADS, 1)
    paged_chunk_tc_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                          const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ ChunkArgs a) {
    using L = CtSmem<DH>;
    extern __shared__ __align__(1024) uint8_t ct_raw[];
    uint8_t *t = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(ct_raw) + 1023) & ~uintptr_t(1023));
    CtShared &S = *reinterpret_cast<CtShared *>(t + L::TILES);
    int *cum = reinterpret_cast<int *>(t + L::CUM);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, cta = blockIdx.x;

    if (threadIdx.x == 0) {
        for (int b = 0; b < 2; ++b) {
            mbar_init(&S.bq[b], 1);
            mbar_init(&S.bl[b], 1);
            mbar_init(&S.bf[b], 1);
            mbar_init(&S.bs[b], 1);
            mbar_init(&S.bp[b][0], 128);
            mbar_init(&S.bp[b][1], 128);
            mbar_init(&S.bo[b], 1);
            for (int i = 0; i < 4; ++i) S.odd_[4 * b + i] = 0;
        }
        mbar_init(&S.bk0, 1);
        mbar_init(&S.bdone, 1);
        S.abort_ = 0;
        S.issued_ = 0;
        fence_barrier_init();
        tma_prefetch_map(&tmK);
        tma_prefetch_map(&tmV);
        tma_prefetch_map(&tmQ);
    }
    pdl_wait();
    pdl_trigger();
    const int tx = a.toks / 2;  // tokens of a row tile
    int parts = 1, rank = 0, u1 = 0, n;  // n: tiles of this CTA
    ChunkWork w;                         // every warp walks the list for itself
    Shares sh(1, 1);
    if constexpr (CL) {
        parts = (int)cluster_size();
        rank = (int)cluster_rank();
        if (!chunk_item<kTcKeys>(a, quotient(cta, parts), w)) return;  // (the whole cluster, before it holds any TMEM)
        sh = Shares(w.tiles, parts);
        w.tile = rank < w.tiles ? sh.begin(rank) : 0;
        n = rank < w.tiles ? sh.begin(rank + 1) - w.tile : 0;
    } else {
        const int total = chunk_plan<kTcKeys>(a, cum);
        // (a share is at least kLeast tiles: below, the partials would cost more than the tiles)
        const int ctas = min((int)gridDim.x, max(1, (total + kLeast - 1) / kLeast));
        sh = Shares(total, ctas);
        if (threadIdx.x == 0) a.joins[cta].parts = 0;
        if (cta >= min(total, ctas)) return;  // (the whole block, before it holds any TMEM)
        const int u0 = sh.begin(cta);
        u1 = sh.begin(cta + 1);
        n = u1 - u0;
        w = chunk_place<kTcKeys>(a, cum, u0);
    }
    float cl_m = -INFINITY, cl_l = 0.f;  // CL: the row's max and sum in this CTA
    CtWaits waits{S, a.err};
#ifdef LF_DEBUG
    waits.lose = (a.lose_cta < 0 || a.lose_cta == cta) && a.lose_warp == warp ? a.lose_wait : 0;
#endif
    int started = 0, loads[2] = {0, 0};  // the copying warp: loads on bl and on bq so far
    if (warp == 1) tc_alloc(&S.tmem, C_TMEM_COLS);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = S.tmem;

    if (warp == 0) {
        // copies: lane i < boxes looks up and loads the tile's i-th box
        const int box = min(1 << a.kv.ps_log2, kTcKeys), boxes = kTcKeys / box;
        struct Box {
            int h, page, row;
        };
        auto place = [&] {  // this lane's box of w's tile
            const int at = (w.kt0 + w.tile) * kTcKeys + lane * box;
            Box x;
            x.h = w.h;
            x.page = a.kv.n_pages;  // outside the tensor: zeros
            x.row = at & ((1 << a.kv.ps_log2) - 1);
            if (lane < boxes && at < w.k.hi && at + box > w.k.lo) {
                const int p = a.kv.table[(long long)w.b * a.kv.max_pages + (at >> a.kv.ps_log2)];
                if (p >= 0 && p < a.kv.n_pages)
                    x.page = p;
                else
                    atomicExch(a.err, 1u);
            }
            return x;
        };
        auto load = [&](int tile_at, const CUtensorMap *map, const Box &x, uint64_t *bar) {
            if (lane < boxes)
                for (int i = 0; i < L::HALVES; ++i)
                    tma_load_4d(t + tile_at + lane * box * 128 + i * T_HALF, map, 64 * i, x.row, x.h, x.page, bar);
        };
        // An item's queries, a box of (64 dims, heads of the group, tokens) for each half of a row tile: its rows lie as the
        // products want them (rows of tokens behind the item's are of others, or zeros past the last: nobody reads their
        // results).
        struct Queries {
            int head, row, nx;
        };
        auto queries_of = [&] { return Queries{w.h * a.group, w.ch.row0 + w.tok, w.toks > tx ? 2 : 1}; };
        auto load_queries = [&](const Queries &q) {
            if (lane < q.nx) {
                mbar_arrive_expect_tx(&S.bq[lane], L::HALVES * 64 * 2 * a.group * tx);
                for (int i = 0; i < L::HALVES; ++i)
                    tma_load_3d(t + L::Q + lane * L::TILE + i * T_HALF, &tmQ, 64 * i, q.head, q.row + lane * tx, &S.bq[lane]);
            }
            __syncwarp();
        };
        Box now = place(), then = now;
        Queries q_now = queries_of(), q_then = q_now;
        bool fresh_now = true, fresh_then = false;  // tile j, tile j + 1 begin an item
        if (lane == 0) mbar_arrive_expect_tx(&S.bk0, L::TILE);
        __syncwarp();
        load(L::K, &tmK, now, &S.bk0);
        bool ok = true;
        for (int j = 0; j < n; ++j) {  // V of tile j and K of the next
            if (j + 1 < n) {
                fresh_then = chunk_advance<kTcKeys>(a, cum, w);
                then = place();
                if (fresh_then) q_then = queries_of();
            }
            // their buffers are free once the S products of tile j - 1 and the P V products of tile j - 2 are done, and so
            // are the queries of the item before
            if (j >= 1) ok = waits(&S.bf[(j - 1) & 1], ((j - 1) >> 1) & 1u);
            if (!__all_sync(0xffffffffu, ok)) break;
            if (fresh_now) {
                load_queries(q_now);
                ++loads[0];
                loads[1] += q_now.nx > 1;
            }
            uint64_t *bar = &S.bl[j & 1];
            if (lane == 0) mbar_arrive_expect_tx(bar, j + 1 < n ? 2 * L::TILE : L::TILE);
            __syncwarp();
            load(L::V + (j & 1) * L::TILE, &tmV, now, bar);
            if (j + 1 < n) load(L::K + ((j + 1) & 1) * L::TILE, &tmK, then, bar);
            ++started;
            now = then;
            q_now = q_then;
            fresh_now = fresh_then;
        }
    } else if (warp == 1) {
        // products, issued in order by one lane (the whole warp walks along: what the instructions take stays in uniform
        // registers, and nothing but them stands between two of them)
        const bool leader = elect_one();
        constexpr uint32_t kIdescS = idesc<T>(128, kTcKeys, false), kIdescO = idesc<T>(128, DH, true);
        // (descriptors of what lies `bytes` further: the address is in the low word)
        auto on = [](uint64_t d, uint32_t bytes) {
            return (d & 0xffffffff00000000ull) | (uint32_t)((uint32_t)d + (bytes >> 4));
        };
        const uint64_t q0 = smem_desc_sw128(smem_u32(t + L::Q)), k0 = smem_desc_sw128(smem_u32(t + L::K)),
                       v0 = desc_mn_sw128(smem_u32(t + L::V));
        auto qk = [&](int x, int j) {
            const uint64_t q = on(q0, (uint32_t)x * L::TILE), k = on(k0, (uint32_t)(j & 1) * L::TILE);
#pragma unroll
            for (int kk = 0; kk < DH / 16; ++kk) {
                const uint32_t off = (uint32_t)(kk >> 2) * T_HALF + (uint32_t)(kk & 3) * 32;
                tc_mma(tmem + (uint32_t)x * kTcKeys, on(q, off), on(k, off), kIdescS, kk > 0);
            }
            tc_commit(&S.bs[x]);
        };
        auto pv = [&](int x, int j, bool first, int kk0, int kk1) {  // steps of 16 keys
            const uint64_t v = on(v0, (uint32_t)(j & 1) * L::TILE);
#pragma unroll
            for (int kk = kk0; kk < kk1; ++kk)
                tc_mma_tmem_a(tmem + C_O + (uint32_t)x * 128, tmem + (uint32_t)x * kTcKeys + (uint32_t)kk * 8,
                              on(v, (uint32_t)kk * 16 * 128), kIdescO, (!first || kk > 0) ? 1u : 0u);
        };
        auto await = [&](uint64_t *bar, uint32_t parity) {
            const bool got = __all_sync(0xffffffffu, waits(bar, parity));
            tc_fence_after();
            return got;
        };
        uint32_t np[2] = {0, 0}, nq[2] = {0, 0};  // uses of bp and bq so far
        int nx = w.toks > tx ? 2 : 1;             // row tiles in use
        int to_go = w.tiles - w.tile;             // tiles of the item from this one on
        bool first = true, ok = await(&S.bk0, 0) && n > 0;  // (CL: a share may be empty)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            if (!ok || x >= nx) break;
            ok = await(&S.bq[x], nq[x]++ & 1u);
            if (ok && leader) {
                qk(x, 0);
                S.issued_ = 1;
            }
            __syncwarp();
        }
        if (ok && leader) tc_commit(&S.bf[0]);
        ok = ok && await(&S.bl[0], 0);
        for (int j = 0; ok && j < n; ++j) {
            const bool ends = to_go == 1, more = j + 1 < n;  // ends: the next tile belongs to another item
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                if (!ok || x >= nx) break;
                const uint32_t ph = np[x]++ & 1u;
                ok = await(&S.bp[x][0], ph);
                if (!ok) break;
                if (leader) pv(x, j, first, 0, C_FIRST / 16);
                __syncwarp();
                ok = await(&S.bp[x][1], ph);
                if (!ok) break;
                if (leader) {
                    pv(x, j, false, C_FIRST / 16, kTcKeys / 16);
                    if (ends || !more) tc_commit(&S.bo[x]);
                    if (more && !ends) qk(x, j + 1);  // after the P V that read P from the same columns
                    if (x + 1 == nx && more && !ends) tc_commit(&S.bf[(j + 1) & 1]);
                }
                __syncwarp();
            }
            if (!ok) break;
            first = false;
            --to_go;
            if (ends && more) {  // both row tiles are on their way out; the next item's Q follows
                w.tile = w.tiles - 1;
                chunk_advance<kTcKeys>(a, cum, w);
                first = true;
                nx = w.toks > tx ? 2 : 1;
                to_go = w.tiles;
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    if (!ok || x >= nx) break;
                    ok = await(&S.bq[x], nq[x]++ & 1u);
                    if (ok && leader) qk(x, j + 1);
                    __syncwarp();
                }
                if (ok && leader) tc_commit(&S.bf[(j + 1) & 1]);
                __syncwarp();
            }
            if (more) ok = ok && await(&S.bl[(j + 1) & 1], ((j + 1) >> 1) & 1u);
        }
        if (leader && S.issued_) tc_commit(&S.bdone);  // tracks everything issued above
        __syncwarp();
    } else {  // softmax warpgroup x: warp w owns TMEM lanes (rows) 32 * (w % 4) .. + 31
        const int x = (warp - 2) >> 2, quarter = warp & 3, row = 32 * quarter + lane;
        const uint32_t trow = tmem + ((uint32_t)(32 * quarter) << 16);
        const uint32_t ts = trow + (uint32_t)x * kTcKeys, to = trow + C_O + (uint32_t)x * 128;
        const float sc2 = a.scale_log2;
        constexpr float kLazy = 8.f;  // log2 of the largest P before the max moves
        // this item and the next one, in shared memory: the row's scores need the registers
        ChunkWork *const works = reinterpret_cast<ChunkWork *>(t + L::WORK) + 2 * (warp - 2);
        if (lane == 0) works[0] = w;
        __syncwarp();
        int left = n, at_tile = 0, ns = 0, no = 0;  // ns, no: uses of bs and bo so far
        bool ok = true, whole = w.tile == 0;        // whole: this CTA has begun the item
        for (int it = 0; ok && left > 0; ++it) {
            const ChunkWork &y = works[it & 1];
            auto next_item = [&] {
                if (lane == 0) {
                    ChunkWork z = y;
                    z.tile = z.tiles - 1;
                    chunk_advance<kTcKeys>(a, cum, z);
                    works[(it + 1) & 1] = z;
                }
                __syncwarp();
            };
            const int count = min(left, y.tiles - y.tile);  // tiles of this item in this CTA
            if (!CL && x == 0 && row == 0 && count == left) a.joins[cta] = chunk_join(a, y, sh, cta, u1, y.tile + count, whole);
            const int rows = min(tx, y.toks - x * tx) * a.group;
            const bool warp_used = 32 * quarter < rows;
            if (rows > 0) {
                const int j00 = (y.kt0 + y.tile) * kTcKeys;  // the first tile's first position
                // tiles that every row of the item sees whole: up to its first token, from its last one's window on
                const int first_pos = y.ch.base + y.tok, last_pos = first_pos + y.toks - 1;
                const int full_to = (max(first_pos + 1, 0) >> 7) - (j00 >> 7);
                const int full_from = a.window == 0 || last_pos < a.window ? 0 : ((last_pos - a.window) >> 7) + 1 - (j00 >> 7);
                static_assert(kTcKeys == 128, "shifts above");
                const int pos = row < rows ? first_pos + x * tx + quotient(row, a.group) - j00 : INT_MIN;  // from there on
                const int lo = y.k.lo - j00, hi = y.k.hi - j00;
                float m2 = -INFINITY, l = 0.f;
                for (int j = 0; j < count; ++j, ++ns) {
                    const bool full = j >= full_from && j < full_to;
                    if (!full && x == 0) {  // V of this tile: a key per thread
                        const int vj = at_tile + j, key = j * kTcKeys + row;
                        ok = ok && waits(&S.bl[vj & 1], (vj >> 1) & 1u);
                        if (ok) {
                            const bool none = key < lo || key >= hi;
                            uint8_t *v = t + L::V + (vj & 1) * L::TILE + row * 128;
                            uint32_t odd = 0;
                            if (none) {
#pragma unroll
                                for (int i = 0; i < DH / 8; ++i)  // (lanes begin at different pieces: different banks)
                                    *reinterpret_cast<uint4 *>(v + (i >> 3) * T_HALF + (((i & 7) ^ (lane & 7)) << 4)) = make_uint4(0u, 0u, 0u, 0u);
                            } else {
                                uint4 z[DH / 8];
#pragma unroll
                                for (int i = 0; i < DH / 8; ++i)
                                    z[i] = *reinterpret_cast<const uint4 *>(v + (i >> 3) * T_HALF + (((i & 7) ^ (lane & 7)) << 4));
#pragma unroll
                                for (int i = 0; i < DH / 8; ++i)
                                    odd |= odd_bits<T>(z[i].x) | odd_bits<T>(z[i].y) | odd_bits<T>(z[i].z) | odd_bits<T>(z[i].w);
                                if (odd) {
                                    uint16_t *h = reinterpret_cast<uint16_t *>(v);
                                    for (int i = 0; i < DH; ++i) {
                                        uint16_t &e = h[(i >> 6) * (T_HALF / 2) + (i & 63)];
                                        if (odd_bits<T>(e)) e = 0;
                                    }
                                }
                            }
                            if (odd) S.odd_[it & 7] = it + 1;
                            fence_proxy_async_shared();
                        }
                    }
                    ok = __all_sync(0xffffffffu, ok && waits(&S.bs[x], ns & 1u));
                    if (!ok) break;
                    tc_fence_after();
                    if (!warp_used) {  // (rows of nobody: whatever their P is)
                        tc_fence_before();
                        mbar_arrive(&S.bp[x][0]);
                        mbar_arrive(&S.bp[x][1]);
                        continue;
                    }
                    float2 r[kTcKeys / 2];
                    uint32_t *ri = reinterpret_cast<uint32_t *>(r);
                    float *rf = reinterpret_cast<float *>(r);
#pragma unroll
                    for (int c0 = 0; c0 < kTcKeys; c0 += 32) tc_ld32_nowait(ts + (uint32_t)c0, ri + c0);
#pragma unroll
                    for (int c0 = 0; c0 < kTcKeys; c0 += 32) tc_wait_ld32(ri + c0);
                    if (!full) {  // this row sees keys c with clo < c <= chi
                        const int chi = pos < j * kTcKeys ? -1 : min(pos - j * kTcKeys, kTcKeys);
#pragma unroll
                        for (int c = 0; c < kTcKeys; ++c) ri[c] = c <= chi ? ri[c] : 0xff800000u;  // -inf
                        if (a.window > 0) {
                            const int clo = (int)max(-1ll, min((long long)kTcKeys, (long long)pos - a.window - j * kTcKeys));
#pragma unroll
                            for (int c = 0; c < kTcKeys; ++c) ri[c] = c > clo ? ri[c] : 0xff800000u;
                        }
                    }
                    // the tile's max of the row in eight independent chains of three-input maxima
                    float mp[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) mp[i] = rf[i];
#pragma unroll
                    for (int c = 8; c < kTcKeys; c += 16)
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            mp[i] = c + 8 + i < kTcKeys ? max3(mp[i], rf[c + i], rf[c + 8 + i]) : fmaxf(mp[i], rf[c + i]);
                    const float mr = max3(max3(mp[0], mp[1], mp[2]), max3(mp[3], mp[4], mp[5]), fmaxf(mp[6], mp[7]));
                    float fac = 1.f;
                    if (mr != -INFINITY && mr * sc2 > m2 + kLazy) {
                        const float mn = mr * sc2;
                        fac = ex2(m2 - mn);  // 0 while the row had no key yet (O and l are 0 then)
                        l *= fac;
                        m2 = mn;
                    }
                    if (j > 0 && __any_sync(0xffffffffu, fac != 1.f)) {
                        // the commit that published S of this tile covers the row tile's
                        // previous P V, and this tile's waits for the arrivals below: O is idle
#pragma unroll 1
                        for (int c0 = 0; c0 < DH; c0 += 16) {
                            float o[16];
                            tc_ld16(to + (uint32_t)c0, o);
                            uint32_t ob[16];
#pragma unroll
                            for (int i = 0; i < 16; ++i) ob[i] = __float_as_uint(o[i] * fac);
                            tc_st16_nowait(to + (uint32_t)c0, ob);
                        }
                    }
                    // P over the first 64 columns of S (S is in registers now)
                    const float neg = m2 == -INFINITY ? 0.f : -m2;
                    const float2 neg2 = make_float2(neg, neg), scale2 = make_float2(sc2, sc2);
                    float2 ls[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                    for (int c0 = 0; c0 < kTcKeys; c0 += 32) {
                        uint32_t pk[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const float2 d = fma2(r[c0 / 2 + i], scale2, neg2);
                            const float2 p = make_float2(ex2(d.x), ex2(d.y));
                            ls[i & 1] = add2(ls[i & 1], p);
                            pk[i] = pack2<T>(p.x, p.y);
                        }
                        tc_st16_nowait(ts + (uint32_t)(c0 / 2), pk);
                        if (c0 + 32 == C_FIRST || c0 + 32 == kTcKeys) {
                            tc_wait_st();
                            tc_fence_before();
                            mbar_arrive(&S.bp[x][c0 + 32 == kTcKeys]);
                        }
                    }
                    const float2 s2 = add2(ls[0], ls[1]);
                    l += s2.x + s2.y;
                }
                if constexpr (CL) {
                    if (ok) ok = __all_sync(0xffffffffu, waits(&S.bo[x], no++ & 1u));
                    cl_m = m2;
                    cl_l = l;
                    break;
                }
                // the rows' result or partial, once the last P V is done; what needs no wait first
                const bool result = whole && y.tile + count == y.tiles;
                const int tok = quotient(min(row, rows - 1), a.group);
                const bool mine = row < rows;
                const long long q_row = (long long)y.ch.row0 + y.tok + x * tx + tok;
                const int head = y.h * a.group + (row - tok * a.group);
                const long long at = (long long)(2 * cta + (whole ? 1 : 0)) * a.slot_rows + x * tx * a.group + row;
                const long long dst = !mine ? -1 : result ? q_row * a.ld_out + (long long)head * DH : at * DH;
                // rows leave through shared memory: 64 bytes of a row to four neighbouring lanes
                long long to4[4];  // of the rows 8 k + lane / 4
#pragma unroll
                for (int k = 0; k < 4; ++k) to4[k] = __shfl_sync(0xffffffffu, dst, 8 * k + lane / 4);
                if (left > count) next_item();
                if (ok) ok = __all_sync(0xffffffffu, waits(&S.bo[x], no++ & 1u));
                // (the products behind bo waited for every cleaned tile of the item: its flag is final from here on)
                const bool odd = S.odd_[it & 7] == it + 1;
                if (ok && warp_used) {
                    tc_fence_after();
                    float v[DH];
                    uint32_t *vi = reinterpret_cast<uint32_t *>(v);
#pragma unroll
                    for (int c0 = 0; c0 < DH; c0 += 32) tc_ld32_nowait(to + (uint32_t)c0, vi + c0);
#pragma unroll
                    for (int c0 = 0; c0 < DH; c0 += 32) tc_wait_ld32(vi + c0);
                    tc_fence_before();
                    if (odd && mine) {  // what is not finite reaches those who see it
                        const int my_pos = y.ch.base + y.tok + x * tx + tok;
                        for (int j = 0; j < count * kTcKeys; ++j) {
                            const int p = (y.kt0 + y.tile) * kTcKeys + j, p0 = p & ~(kTcKeys - 1);
                            if (p0 + kTcKeys - 1 <= first_pos && (a.window == 0 || p0 > (long long)last_pos - a.window)) continue;
                            if (p > my_pos || p < y.k.lo || (a.window > 0 && p <= (long long)my_pos - a.window)) continue;
                            const int page = a.kv.table[(long long)y.b * a.kv.max_pages + (p >> a.kv.ps_log2)];
                            if (page < 0 || page >= a.kv.n_pages) continue;
                            const T *src = static_cast<const T *>(a.kv.v) + page * a.kv.page_stride +
                                           ((((long long)y.h << a.kv.ps_log2) + (p & ((1 << a.kv.ps_log2) - 1))) * DH);
#pragma unroll
                            for (int i = 0; i < DH; ++i) {
                                const float f = (float)src[i];
                                if (!(fabsf(f) < INFINITY)) v[i] += f;
                            }
                        }
                    }
                    uint8_t *stage = t + L::OUT + (warp - 2) * 32 * L::OUT_ROW;
                    uint4 *own = reinterpret_cast<uint4 *>(stage + lane * L::OUT_ROW);
                    const uint4 *theirs = reinterpret_cast<const uint4 *>(stage + (lane / 4) * L::OUT_ROW + (lane & 3) * 16);
                    if (result) {
                        const float inv = inverse(l);
                        T *out = static_cast<T *>(a.out) + (lane & 3) * 8;
#pragma unroll
                        for (int c0 = 0; c0 < DH; c0 += 32) {
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const float *f = v + c0 + 8 * i;
                                own[i] = make_uint4(pack2<T>(f[0] * inv, f[1] * inv), pack2<T>(f[2] * inv, f[3] * inv),
                                                    pack2<T>(f[4] * inv, f[5] * inv), pack2<T>(f[6] * inv, f[7] * inv));
                            }
                            __syncwarp();
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                if (to4[k] >= 0) *reinterpret_cast<uint4 *>(out + to4[k] + c0) = theirs[k * 8 * L::OUT_ROW / 16];
                            __syncwarp();
                        }
                        if (mine && a.lse) a.lse[q_row * a.n_q + head] = m2 * 0.69314718055994530942f + logf(l);
                    } else {
                        const uint64_t keep = policy_evict_last();
                        float *out = a.part_o + (lane & 3) * 4;
#pragma unroll
                        for (int c0 = 0; c0 < DH; c0 += 16) {
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                own[i] = make_uint4(vi[c0 + 4 * i], vi[c0 + 4 * i + 1], vi[c0 + 4 * i + 2], vi[c0 + 4 * i + 3]);
                            __syncwarp();
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                if (to4[k] >= 0)
                                    st_hint(reinterpret_cast<float4 *>(out + to4[k] + c0),
                                            *reinterpret_cast<const float4 *>(theirs + k * 8 * L::OUT_ROW / 16), keep);
                            __syncwarp();
                        }
                        if (mine) a.part_ml[at] = make_float2(m2, l);
                    }
                }
            } else if (left > count) {  // (this warpgroup has no part in this item)
                next_item();
            }
            left -= count;
            at_tile += count;
            whole = true;
        }
    }
    if constexpr (CL) {
        // The CTAs' partials of the item: each softmax warp's rows belong to one CTA, which the others push theirs to
        // (where its operands lay: by the first barrier all products are done).
        __syncwarp();
        tc_fence_before();
        cluster_arrive();
        cluster_wait();
        tc_fence_after();
        const int wi = warp - 2, x = wi >> 2, quarter = warp & 3, row = 32 * quarter + lane;
        const int of = 8 / parts, block = 4 * x + quarter, owner = block / of;  // of: warps' rows of a CTA
        const ChunkWork &y = reinterpret_cast<const ChunkWork *>(t + L::WORK)[2 * (wi & 7)];
        const int rows = min(tx, y.toks - x * tx) * a.group;
        const bool used = wi >= 0 && 32 * quarter < rows, mine = row < rows;
        const uint32_t to = tmem + ((uint32_t)(32 * quarter) << 16) + C_O + (uint32_t)(x & 1) * 128;
        const bool odd = S.odd_[0] == 1;
        const int tok = used ? quotient(min(row, rows - 1), a.group) : 0;
        auto values = [&](int c0, float *v) {  // 32 dims of the row's unnormalised o here
            uint32_t *vi = reinterpret_cast<uint32_t *>(v);
            tc_ld32_nowait(to + (uint32_t)c0, vi);
            tc_wait_ld32(vi);
            if (odd && mine) {  // what is not finite reaches those who see it
                const int first_pos = y.ch.base + y.tok, last_pos = first_pos + y.toks - 1, my_pos = first_pos + x * tx + tok;
                for (int j = 0; j < n * kTcKeys; ++j) {
                    const int p = (y.kt0 + y.tile) * kTcKeys + j, p0 = p & ~(kTcKeys - 1);
                    if (p0 + kTcKeys - 1 <= first_pos && (a.window == 0 || p0 > (long long)last_pos - a.window)) continue;
                    if (p > my_pos || p < y.k.lo || (a.window > 0 && p <= (long long)my_pos - a.window)) continue;
                    const int page = a.kv.table[(long long)y.b * a.kv.max_pages + (p >> a.kv.ps_log2)];
                    if (page < 0 || page >= a.kv.n_pages) continue;
                    const T *src = static_cast<const T *>(a.kv.v) + page * a.kv.page_stride +
                                   ((((long long)y.h << a.kv.ps_log2) + (p & ((1 << a.kv.ps_log2) - 1))) * DH) + c0;
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        const float f = (float)src[i];
                        if (!(fabsf(f) < INFINITY)) v[i] += f;
                    }
                }
            }
        };
        // [other CTA][warp's rows][4 dims][row] and [other CTA][warp's rows][row]
        auto inbox = [&](int from, int to_cta) { return (from < to_cta ? from : from - 1) * of + block % of; };
        if (used && owner != rank) {
            const int slot = inbox(rank, owner);
            cluster_store(cluster_address(smem_u32(cum) + (uint32_t)(slot * 32 + lane) * 8, owner), make_float2(cl_m, cl_l));
            if (n > 0) {
                const uint32_t dst = cluster_address(smem_u32(t + L::Q) + (uint32_t)slot * DH * 128 + (uint32_t)lane * 16, owner);
#pragma unroll 1
                for (int c0 = 0; c0 < DH; c0 += 32) {
                    float v[32];
                    values(c0, v);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        cluster_store(dst + (uint32_t)(c0 / 4 + i) * 512, make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]));
                }
            }
        }
        __syncwarp();
        cluster_arrive();
        cluster_wait();
        if (used && owner == rank) {
            const float2 *stat = reinterpret_cast<const float2 *>(cum);
            float mx = cl_m;
            for (int k = 0; k < parts; ++k)
                if (k != rank) mx = fmaxf(mx, stat[inbox(k, rank) * 32 + lane].x);
            const float off = mx == -INFINITY ? 0.f : mx, f_own = ex2(cl_m - off);
            float sum = f_own * cl_l;
            for (int k = 0; k < parts; ++k)
                if (k != rank) {
                    const float2 z = stat[inbox(k, rank) * 32 + lane];
                    sum += ex2(z.x - off) * z.y;
                }
            const float inv = inverse(sum);
            const long long q_row = (long long)y.ch.row0 + y.tok + x * tx + tok;
            const int head = y.h * a.group + (row - tok * a.group);
            const long long dst = mine ? q_row * a.ld_out + (long long)head * DH : -1;
            long long to4[4];  // of the rows 8 k + lane / 4
#pragma unroll
            for (int k = 0; k < 4; ++k) to4[k] = __shfl_sync(0xffffffffu, dst, 8 * k + lane / 4);
            uint8_t *stage = t + L::OUT + wi * 32 * L::OUT_ROW;
            uint4 *own = reinterpret_cast<uint4 *>(stage + lane * L::OUT_ROW);
            const uint4 *theirs = reinterpret_cast<const uint4 *>(stage + (lane / 4) * L::OUT_ROW + (lane & 3) * 16);
            T *out = static_cast<T *>(a.out) + (lane & 3) * 8;
#pragma unroll 1
            for (int c0 = 0; c0 < DH; c0 += 32) {
                float v[32];
                if (n > 0) values(c0, v);
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] = n > 0 ? v[i] * f_own : 0.f;
                for (int k = 0; k < parts; ++k) {
                    if (k == rank) continue;
                    const int slot = inbox(k, rank);
                    const float z = stat[slot * 32 + lane].x;
                    if (__all_sync(0xffffffffu, z == -INFINITY)) continue;  // (a share without tiles leaves no o)
                    const float f = ex2(z - off);
                    const float4 *src = reinterpret_cast<const float4 *>(t + L::Q + slot * DH * 128 + lane * 16);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float4 q = src[(c0 / 4 + i) * 32];
                        v[4 * i] += f * q.x;
                        v[4 * i + 1] += f * q.y;
                        v[4 * i + 2] += f * q.z;
                        v[4 * i + 3] += f * q.w;
                    }
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float *f = v + 8 * i;
                    own[i] = make_uint4(pack2<T>(f[0] * inv, f[1] * inv), pack2<T>(f[2] * inv, f[3] * inv),
                                        pack2<T>(f[4] * inv, f[5] * inv), pack2<T>(f[6] * inv, f[7] * inv));
                }
                __syncwarp();
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (to4[k] >= 0) *reinterpret_cast<uint4 *>(out + to4[k] + c0) = theirs[k * 8 * L::OUT_ROW / 16];
                __syncwarp();
            }
            if (mine && a.lse) a.lse[q_row * a.n_q + head] = mx * 0.69314718055994530942f + logf(sum);
        }
    }
    tc_fence_before();
    __syncthreads();
    // After an error copies may be in flight, whichever warp gave up and whenever: they land (bounded) before the CTA ends.
    if (warp == 0 && lane == 0 && S.abort_) {
        const uint64_t dl = global_timer_ns() + 1000000000ull;
        while (!mbar_try_wait(&S.bk0, 0) && global_timer_ns() < dl) {
        }
        for (int x = 0; x < 2; ++x)
            while (loads[x] > 0 && !mbar_try_wait(&S.bq[x], (loads[x] - 1) & 1u) && global_timer_ns() < dl) {
            }
        for (int i = max(0, started - 2); i < started; ++i)
            while (!mbar_try_wait(&S.bl[i & 1], (i >> 1) & 1u) && global_timer_ns() < dl) {
            }
    }
    if (warp == 1) {
        if (lane == 0 && S.issued_) {  // the products may still run after an error: wait (bounded)
            const uint64_t dl = global_timer_ns() + 1000000000ull;
            while (!mbar_try_wait(&S.bdone, 0) && global_timer_ns() < dl) {
            }
        }
        __syncwarp();
        tc_fence_after();
        tc_dealloc(tmem, C_TMEM_COLS);
    }
}

// The queries as a 3-D tensor (dim, head, token), boxes of 64 dims x a group's heads x a row tile's tokens, swizzled.
bool query_map(CUtensorMap *map, const ChunkArgs &a, int dtype) {
    PagedEncode enc = paged_encoder();
    if (!enc) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)a.kv.head_dim, (cuuint64_t)a.n_q, (cuuint64_t)a.n_tokens};
    const cuuint64_t str[2] = {(cuuint64_t)a.kv.head_dim * 2, (cuuint64_t)a.ld_q * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)a.group, (cuuint32_t)(a.toks / 2)}, one[3] = {1, 1, 1};
    return enc(map, dtype == LF_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
               const_cast<void *>(a.q), dims, str, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, int DH>
lf_status launch_chunk_tc(const ChunkArgs &a, int dtype, int direct, cudaStream_t st) {
    constexpr int smem = CtSmem<DH>::BYTES;
    if (!set_smem_once<paged_chunk_tc_kernel<T, DH, false>>(smem) || !set_smem_once<paged_chunk_tc_kernel<T, DH, true>>(smem))
        return LF_ERR_CUDA;
    CUtensorMap mk, mv, mq;
    if (!cache_map(&mk, a.kv.k, a.kv, dtype) || !cache_map(&mv, a.kv.v, a.kv, dtype) || !query_map(&mq, a, dtype))
        return LF_ERR_CUDA;
    const bool ok = direct ? launch_pdl_cluster(paged_chunk_tc_kernel<T, DH, true>, (unsigned)direct,
                                                dim3((unsigned)(chunk_items(a) * direct)), C_THREADS, smem, st, mk, mv, mq, a)
                           : launch_pdl(paged_chunk_tc_kernel<T, DH, false>, a.grid, C_THREADS, smem, st, mk, mv, mq, a);
    return ok ? LF_OK : LF_ERR_CUDA;
}

}  // namespace

lf_status paged_chunk_tc(const ChunkArgs &a, int dtype, int direct, cudaStream_t st) {
    if (dtype == LF_F16)
        return a.kv.head_dim == 64 ? launch_chunk_tc<__half, 64>(a, dtype, direct, st) : launch_chunk_tc<__half, 128>(a, dtype, direct, st);
    return a.kv.head_dim == 64 ? launch_chunk_tc<__nv_bfloat16, 64>(a, dtype, direct, st)
                               : launch_chunk_tc<__nv_bfloat16, 128>(a, dtype, direct, st);
}

}  // namespace lf
