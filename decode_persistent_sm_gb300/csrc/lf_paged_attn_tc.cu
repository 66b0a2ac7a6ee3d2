// The common positions of lf_attn_paged_shared on the 5th-generation tensor
// cores, for batches whose rows (sequence, query head) of one KV head are many
// enough that warp-level MMAs would be the bound (tcgen05 + TMA + TMEM).
//
// An item is 256 rows of one KV head, two M = 128 tiles, against all common
// keys; the tiles of 128 keys of all items form one list, cut into equal
// shares, one per SM, and a CTA leaves one partial (unnormalised o, max, sum)
// per item it touches.  Per key tile and row tile x:
//   S = Q K^T into TMEM; the row tile's softmax warpgroup, a row per thread,
//   reads S, moves the row's running max (only when it grows by more than 2^8,
//   so P stays below 256), and writes P in the cache's type back over S;
//   O += P V with P as the A operand from TMEM.
// The two row tiles take turns: one's softmax runs under the other's products.
// K and V pages come by TMA (one box of min(page size, 128) positions x 64
// dims each), double-buffered; V is read as it lies, [key][dim], as an MN-major
// B operand, so no transposed copy of the cache is kept.  The common range is
// cut to whole pages here (what is left of the first and last page goes to the
// sequences' own items), and pages past its end are loaded from outside the
// tensor, which reads as zeros, so that no value that is not to be seen enters
// a product.
//
// Measured: 64 sequences x 8 heads per KV head (512 rows), 8 KV heads of 128, 16384
// common positions, BF16: 35 us, 980 TFLOP/s (51 % of the measured dense rate; the
// tensor pipe is active 41 % of the time).  The whole call 85 us: behind it the
// kernel of the sequences' own positions starts (6 to 8 us) and reads them (31 us,
// 135 MB); on warp-level MMAs alone 161.  A step
// (128 keys, both row tiles) takes 3700 cycles for 2048 of products.  Its chain is
// softmax (1400: load 100, max 200, exponentials 800, store and fence 160), then P V
// and Q K^T (512 each, and 340 until the result is seen).  Around the products the
// issuing thread's own instructions count, some 300 cycles for a wait even when it
// is over: so one wait for V and the next K, counters and descriptors in
// registers, no barrier that nobody waits for (-5 us).  Slower: a thread
// per half row (16 softmax warps, +8 %), an issuing warp per row tile (their products
// interleave and delay both, +2 %), tiles of 64 keys with two buffers of S (+30 %: twice
// as many waits).
//
// Every wait is bounded; a CTA that ran out of time flags it, lets its copies
// and products finish (bounded), frees its TMEM and exits.
#include "lf_paged_tc.cuh"

namespace lf {
namespace {

constexpr int T_THREADS = 320;            // copy warp, MMA warp, 2 x 4 softmax warps
constexpr uint32_t T_TMEM_COLS = 512;     // S / P of row tile x at 128 x, O at 256 + 128 x
constexpr uint32_t T_O = 256;
constexpr unsigned long long kTimeoutNs = 2000000000ull;

// Every barrier completes once per use of what it guards, and no waiter can
// fall two phases behind, so parity waits are unambiguous.
struct TcShared {
    uint64_t bq[2];   // Q of row tile x written (128 arrivals)
    uint64_t bk0;     // K of the first tile loaded
    uint64_t bl[2];   // V of tile p and K of tile p + 1 loaded (p = 0, 2, .. and 1, 3, ..)
    uint64_t bf[2];   // done: the S products of tile p and the P V products of tile p - 1 (p = 0, 2, .. and 1, 3, ..)
    uint64_t bs[2];   // row tile x: S of the next tile computed (and its earlier P V done)
    uint64_t bp[2];   // row tile x: P written to TMEM (128 arrivals)
    uint64_t bo[2];   // row tile x: the last P V of an item done
    uint64_t bdone;   // every product this CTA issued is done (one commit at the end)
    uint32_t tmem;
    volatile int abort_;
    volatile int issued_;  // 1 once any product was issued (then bdone gets its commit)
};

__device__ __forceinline__ bool await_phase(TcShared &S, uint64_t *bar, uint32_t parity, uint64_t deadline,
                                            uint32_t *err) {
    if (mbar_test_wait(bar, parity)) return true;
    while (!mbar_try_wait(bar, parity)) {
        if (S.abort_) return false;
        if (global_timer_ns() > deadline) {
            atomicExch(err, 2u);
            S.abort_ = 1;
            return false;
        }
    }
    return true;
}

template <int DH>
struct TcSmem {
    static constexpr int HALVES = DH / 64;
    static constexpr int TILE = HALVES * T_HALF;  // one row tile of Q, one buffer of K or V
    static constexpr int Q = 0, K = 2 * TILE, V = 4 * TILE, TILES = 6 * TILE;
    static constexpr int BYTES = TILES + 1024 + 256;
};

template <typename T, int DH>
__global__ void __launch_bounds__(T_THREADS, 1)
    paged_attn_tc_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                         const AttnArgs a) {
    using L = TcSmem<DH>;
    extern __shared__ __align__(1024) uint8_t tc_raw[];
    uint8_t *t = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(tc_raw) + 1023) & ~uintptr_t(1023));
    TcShared &S = *reinterpret_cast<TcShared *>(t + L::TILES);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    pdl_wait();
    pdl_trigger();
    const Common com(a, __reduce_max_sync(0xffffffffu, latest_start(a, lane)));
    const int keys = com.hi - com.lo, tiles = (keys + kTcKeys - 1) / kTcKeys, total = a.kv.n_kv * a.row_tiles * tiles;
    const Shares sh(total, gridDim.x);
    if ((int)blockIdx.x >= min(total, (int)gridDim.x)) return;
    const int u0 = sh.begin(blockIdx.x), n = sh.begin(blockIdx.x + 1) - u0;
    const int item0 = quotient(u0, tiles), tile0 = u0 - item0 * tiles;
    const int all_rows = a.kv.n_seqs * a.group;
    // row tiles in use of an item
    auto row_tiles_of = [&](int item) {
        return all_rows - (item % a.row_tiles) * kTcRows > 128 ? 2 : 1;
    };
    const uint64_t deadline = global_timer_ns() + kTimeoutNs;

    if (threadIdx.x == 0) {
        for (int b = 0; b < 2; ++b) {
            mbar_init(&S.bq[b], 128);
            mbar_init(&S.bl[b], 1);
            mbar_init(&S.bf[b], 1);
            mbar_init(&S.bs[b], 1);
            mbar_init(&S.bp[b], 128);
            mbar_init(&S.bo[b], 1);
        }
        mbar_init(&S.bk0, 1);
        mbar_init(&S.bdone, 1);
        S.abort_ = 0;
        S.issued_ = 0;
        fence_barrier_init();
        tma_prefetch_map(&tmK);
        tma_prefetch_map(&tmV);
    }
    if (warp == 1) tc_alloc(&S.tmem, T_TMEM_COLS);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = S.tmem;

    if (warp == 0) {
        // copies: lane i < pages looks up and loads the tile's i-th box
        const int box = min(1 << a.kv.ps_log2, kTcKeys), boxes = kTcKeys / box;
        struct Box {
            int h, page, row;
        };
        int tile = tile0, item = item0, started = 0;  // loads on bl so far
        auto next = [&] {  // this lane's box of the next tile of the list
            const int at = com.lo + tile * kTcKeys + lane * box;
            Box x;
            x.h = item / a.row_tiles;
            x.page = a.kv.n_pages;  // outside the tensor: zeros
            x.row = at & ((1 << a.kv.ps_log2) - 1);
            if (lane < boxes && at < com.hi) {
                const int p = a.kv.table[at >> a.kv.ps_log2];  // sequence 0's row of the table
                if (p >= 0 && p < a.kv.n_pages)
                    x.page = p;
                else
                    atomicExch(a.err, 1u);
            }
            if (++tile == tiles) {
                tile = 0;
                ++item;
            }
            return x;
        };
        auto load = [&](int tile_at, const CUtensorMap *map, const Box &x, uint64_t *bar) {
            if (lane < boxes)
                for (int i = 0; i < L::HALVES; ++i)
                    tma_load_4d(t + tile_at + lane * box * 128 + i * T_HALF, map, 64 * i, x.row, x.h, x.page, bar);
        };
        Box now = next(), then = now;
        if (lane == 0) mbar_arrive_expect_tx(&S.bk0, L::TILE);
        __syncwarp();
        load(L::K, &tmK, now, &S.bk0);
        bool ok = true;
        for (int j = 0; j < n; ++j) {  // V of tile j and K of the next
            if (j + 1 < n) then = next();
            // their buffers are free once the S products of tile j - 1 and the P V products of tile j - 2 are done
            if (j >= 1) ok = await_phase(S, &S.bf[(j - 1) & 1], ((j - 1) >> 1) & 1u, deadline, a.err);
            if (!__all_sync(0xffffffffu, ok)) break;
            uint64_t *bar = &S.bl[j & 1];
            if (lane == 0) mbar_arrive_expect_tx(bar, j + 1 < n ? 2 * L::TILE : L::TILE);
            __syncwarp();
            load(L::V + (j & 1) * L::TILE, &tmV, now, bar);
            if (j + 1 < n) load(L::K + ((j + 1) & 1) * L::TILE, &tmK, then, bar);
            ++started;
            now = then;
        }
        if (S.abort_ && lane == 0) {  // let the copies in flight land
            const uint64_t dl = global_timer_ns() + 1000000000ull;
            while (!mbar_try_wait(&S.bk0, 0) && global_timer_ns() < dl) {
            }
            for (int i = max(0, started - 2); i < started; ++i)
                while (!mbar_try_wait(&S.bl[i & 1], (i >> 1) & 1u) && global_timer_ns() < dl) {
                }
        }
    } else if (warp == 1) {
        if (lane == 0) {  // products, issued in order by this one thread
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
            };
            auto pv = [&](int x, int j, bool first) {
                const uint64_t v = on(v0, (uint32_t)(j & 1) * L::TILE);
#pragma unroll
                for (int kk = 0; kk < kTcKeys / 16; ++kk)
                    tc_mma_tmem_a(tmem + T_O + (uint32_t)x * 128, tmem + (uint32_t)x * kTcKeys + (uint32_t)kk * 8,
                                  on(v, (uint32_t)kk * 16 * 128), kIdescO, (!first || kk > 0) ? 1u : 0u);
            };
            int np[2] = {0, 0}, nq[2] = {0, 0};  // uses of bp and bq so far
            int tile = tile0, item = item0, nx = row_tiles_of(item0);
            bool first = true, ok = await_phase(S, &S.bk0, 0, deadline, a.err);
#pragma unroll
            for (int x = 0; x < 2; ++x) {  // (unrolled: the issuing thread's own instructions are on the critical path)
                if (!ok || x >= nx) break;
                ok = await_phase(S, &S.bq[x], nq[x]++ & 1u, deadline, a.err);
                if (!ok) break;
                tc_fence_after();
                qk(x, 0);
                S.issued_ = 1;
                tc_commit(&S.bs[x]);
            }
            if (ok) tc_commit(&S.bf[0]);
            for (int j = 0; ok && j < n; ++j) {
                const int b = j & 1, b1 = (j + 1) & 1;
                const bool ends = tile + 1 == tiles;  // the next tile belongs to another item
                ok = await_phase(S, &S.bl[b], (j >> 1) & 1u, deadline, a.err);
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    if (!ok || x >= nx) break;
                    ok = await_phase(S, &S.bp[x], np[x]++ & 1u, deadline, a.err);
                    if (!ok) break;
                    tc_fence_after();
                    pv(x, j, first);
                    if (ends || j + 1 == n) tc_commit(&S.bo[x]);
                    if (j + 1 < n && !ends) {  // after the P V that read P from the same columns
                        qk(x, j + 1);
                        tc_commit(&S.bs[x]);
                    }
                }
                if (!ok) break;
                first = false;
                if (ends) {
                    tile = 0;
                    ++item;
                    first = true;
                    if (j + 1 < n) {  // both row tiles are on their way out; the next item's Q follows
                        nx = row_tiles_of(item);
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            if (!ok || x >= nx) break;
                            ok = await_phase(S, &S.bq[x], nq[x]++ & 1u, deadline, a.err);
                            if (!ok) break;
                            tc_fence_after();
                            qk(x, j + 1);
                            tc_commit(&S.bs[x]);
                        }
                        if (!ok) break;
                    }
                } else {
                    ++tile;
                }
                tc_commit(&S.bf[b1]);
            }
            if (S.issued_) tc_commit(&S.bdone);  // tracks everything issued above
        }
    } else {  // softmax warpgroup x: warp w owns TMEM lanes (rows) 32 * (w % 4) .. + 31
        const int x = (warp - 2) >> 2, quarter = warp & 3, row = 32 * quarter + lane;
        const uint32_t trow = tmem + ((uint32_t)(32 * quarter) << 16);
        const uint32_t ts = trow + (uint32_t)x * kTcKeys, to = trow + T_O + (uint32_t)x * 128;
        const float sc2 = a.scale_log2;
        constexpr float kLazy = 8.f;  // log2 of the largest P before the max moves
        int item = item0, tile = tile0, left = n, ns = 0, no = 0;  // ns, no: uses of bs and bo so far
        bool ok = true;
        while (ok && left > 0) {
            const int count = min(left, tiles - tile);  // tiles of this item in this CTA
            if (x == 0 && row == 0) {  // for the join
                if (tile == 0) a.span[item].x = blockIdx.x;
                if (tile + count == tiles) a.span[item].y = blockIdx.x;
            }
            if (x < row_tiles_of(item)) {
                const int rt = item % a.row_tiles, h = item / a.row_tiles;
                const int at = rt * kTcRows + x * 128 + row;  // (sequence, head) row of the KV head
                {  // Q of this row into the swizzled tile; the item before is done with it (its last P V was awaited)
                    uint8_t *qs = t + L::Q + x * L::TILE;
                    const T *src = nullptr;
                    if (at < all_rows) {
                        const int b = at / a.group;
                        src = static_cast<const T *>(a.q) + (long long)b * a.ld_q +
                              (long long)(h * a.group + at - b * a.group) * DH;
                    }
                    uint4 v[DH / 8];  // (all loads before the first store)
#pragma unroll
                    for (int c = 0; c < DH / 8; ++c)
                        v[c] = src ? reinterpret_cast<const uint4 *>(src)[c] : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
                    for (int c = 0; c < DH / 8; ++c)
                        *reinterpret_cast<uint4 *>(qs + (c >> 3) * T_HALF + sw128_offset(row, (c & 7) * 8)) = v[c];
                    fence_proxy_async_shared();
                    mbar_arrive(&S.bq[x]);
                }
                float m2 = -INFINITY, l = 0.f;
                for (int j = 0; j < count; ++j, ++ns) {
                    const int valid = keys - (tile + j) * kTcKeys;  // keys of this tile (may exceed it)
                    ok = __all_sync(0xffffffffu, ok && await_phase(S, &S.bs[x], ns & 1u, deadline, a.err));
                    if (!ok) break;
                    tc_fence_after();
                    uint32_t r[kTcKeys];
#pragma unroll
                    for (int c0 = 0; c0 < kTcKeys; c0 += 32) tc_ld32_nowait(ts + (uint32_t)c0, r + c0);
#pragma unroll
                    for (int c0 = 0; c0 < kTcKeys; c0 += 32) tc_wait_ld32(r + c0);
                    if (valid < kTcKeys) {
#pragma unroll
                        for (int c = 0; c < kTcKeys; ++c) r[c] = c < valid ? r[c] : 0xff800000u;  // -inf
                    }
                    // the tile's max of the row in eight independent chains of three-input maxima
                    float mp[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) mp[i] = __uint_as_float(r[i]);
#pragma unroll
                    for (int c = 8; c < kTcKeys; c += 16)
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            mp[i] = c + 8 + i < kTcKeys
                                        ? max3(mp[i], __uint_as_float(r[c + i]), __uint_as_float(r[c + 8 + i]))
                                        : fmaxf(mp[i], __uint_as_float(r[c + i]));
                    const float mr = max3(max3(mp[0], mp[1], mp[2]), max3(mp[3], mp[4], mp[5]), fmaxf(mp[6], mp[7]));
                    float fac = 1.f;
                    if (mr != -INFINITY && mr * sc2 > m2 + kLazy) {
                        const float mn = mr * sc2;
                        fac = ex2(m2 - mn);  // 0 while the row had no key yet (O and l are 0 then)
                        l *= fac;
                        m2 = mn;
                    }
                    // P over the first 64 columns of S (S is in registers now)
                    const float neg_m2 = m2 == -INFINITY ? 0.f : -m2;
                    float ls[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int c0 = 0; c0 < kTcKeys; c0 += 32) {
                        uint32_t pk[16];
#pragma unroll
                        for (int i = 0; i < 32; i += 2) {
                            const float p0 = ex2(fmaf(__uint_as_float(r[c0 + i]), sc2, neg_m2));
                            const float p1 = ex2(fmaf(__uint_as_float(r[c0 + i + 1]), sc2, neg_m2));
                            ls[(i >> 1) & 3] += p0 + p1;
                            pk[i / 2] = pack2<T>(p0, p1);
                        }
                        tc_st16_nowait(ts + (uint32_t)(c0 / 2), pk);
                    }
                    l += (ls[0] + ls[1]) + (ls[2] + ls[3]);
                    tc_wait_st();
                    if (j > 0 && __any_sync(0xffffffffu, fac != 1.f)) {
                        // the commit that published S of this tile covers the row tile's
                        // previous P V, and this tile's waits for the arrival below: O is idle
#pragma unroll 1
                        for (int c0 = 0; c0 < DH; c0 += 16) {
                            float o[16];
                            tc_ld16(to + (uint32_t)c0, o);
                            uint32_t ob[16];
#pragma unroll
                            for (int i = 0; i < 16; ++i) ob[i] = __float_as_uint(o[i] * fac);
                            tc_st16_nowait(to + (uint32_t)c0, ob);
                        }
                        tc_wait_st();
                    }
                    tc_fence_before();
                    mbar_arrive(&S.bp[x]);
                }
                // the partial of this row, once the last P V is done
                if (ok) ok = __all_sync(0xffffffffu, await_phase(S, &S.bo[x], no++ & 1u, deadline, a.err));
                if (ok) {
                    tc_fence_after();
                    const long long slot = (long long)(item + blockIdx.x) * kTcRows + x * 128 + row;
                    float *dst = a.part_o + slot * DH;
                    const uint64_t keep = policy_evict_last();
#pragma unroll 1
                    for (int c0 = 0; c0 < DH; c0 += 32) {
                        float v[32];
                        tc_ld32(to + (uint32_t)c0, v);
                        if (at < all_rows) {
#pragma unroll
                            for (int i = 0; i < 32; i += 4)
                                st_hint(reinterpret_cast<float4 *>(dst + c0 + i), make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]), keep);
                        }
                    }
                    if (at < all_rows) a.part_ml[slot] = make_float2(m2, l);
                    tc_fence_before();
                }
            }
            left -= count;
            tile = 0;
            ++item;
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        if (lane == 0 && S.issued_) {  // the products may still run after an error: wait (bounded)
            const uint64_t dl = global_timer_ns() + 1000000000ull;
            while (!mbar_try_wait(&S.bdone, 0) && global_timer_ns() < dl) {
            }
        }
        __syncwarp();
        tc_fence_after();
        tc_dealloc(tmem, T_TMEM_COLS);
    }
}

template <typename T, int DH>
lf_status launch_tc(const AttnArgs &a, int dtype, cudaStream_t st) {
    constexpr int smem = TcSmem<DH>::BYTES;
    if (!set_smem_once<paged_attn_tc_kernel<T, DH>>(smem)) return LF_ERR_CUDA;
    CUtensorMap mk, mv;
    if (!cache_map(&mk, a.kv.k, a.kv, dtype) || !cache_map(&mv, a.kv.v, a.kv, dtype)) return LF_ERR_CUDA;
    return launch_pdl(paged_attn_tc_kernel<T, DH>, a.grid_c, T_THREADS, smem, st, mk, mv, a) ? LF_OK : LF_ERR_CUDA;
}

}  // namespace

lf_status paged_attn_tc(const AttnArgs &a, int dtype, cudaStream_t st) {
    if (dtype == LF_F16)
        return a.kv.head_dim == 64 ? launch_tc<__half, 64>(a, dtype, st) : launch_tc<__half, 128>(a, dtype, st);
    return a.kv.head_dim == 64 ? launch_tc<__nv_bfloat16, 64>(a, dtype, st)
                               : launch_tc<__nv_bfloat16, 128>(a, dtype, st);
}

}  // namespace lf
