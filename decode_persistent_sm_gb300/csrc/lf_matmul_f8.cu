// Product of 8-bit operands with a scale per row of each (sm_103a, tcgen05 + TMA):
//   C[m][n] = sa[m] sb[n] sum_k A[m][k] B[n][k],  A (M x K) and B (N x K) e4m3, row-major.
//
// A persistent CTA per SM walks 128 x BN tiles of C: a copy warp streams 128 x
// 128 and BN x 128 byte tiles of A and B into a shared-memory ring with TMA
// (128-byte swizzle; zeros past K, M and N), one thread issues tcgen05.mma
// (kind::f8f6f4, 32 values of K each, fp32 accumulators in one of two TMEM
// buffers), and four warps read a finished accumulator back, scale it and store
// it while the next tile's products run.
//
// What bounds it: with many rows no unit is full, 3584 x 8192 x 4096 in 90 us, 2660
// TFLOP/s (84 alone: tensor pipe 61 % active, shared memory's banks read and written
// 24 % of their peak each, issue slots 10 %, DRAM 9 %).  With few rows it is a CTA's
// walk along K, which nobody shares, and the weights' stream: 16 x 8192 x 4096 in 10.0
// us, but 16 x 1024, an eighth of the weights, from HBM in 4.2, 4.7, 9.4 and 14.5 with K
// 256 (the call), 1024, 4096 and 8192.  So BN is 256 where the tiles fill the SMs, and less
// where they do not or the stream has to be spread over them.
//
// With few rows a block of 128 along K is over in less time than a barrier's round
// trip: two blocks to a stage (KS) took 16 x 8192 x 4096 from 12.9 us to 10.1.  A stage
// that holds 32 rows of A instead of 128 (AR) leaves room for more of them:
// 14.2 us where 15.5 at 16 x 14336 x 4096.
//
// The accumulators are full fp32: a sum of 4096 products that spread over 2^30 in
// size comes out to 2^-23 of its terms' magnitude.
//
// Every wait is bounded (2 s without progress): on a timeout the CTA records an error,
// lets its copies and MMAs in flight finish (bounded), frees TMEM and exits.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>
#include <mutex>

#include "lf_paged.h"
#include "lf_tc.cuh"

namespace lf {
namespace {

constexpr int F8_BM = 128, F8_BK = 128;  // 128 values of K = 128 bytes = one swizzle row
constexpr int F8_THREADS = 192;          // warp 0 copies, warp 1 MMA + TMEM owner, warps 2-5 epilogue
constexpr int F8_GROUP_M = 32;           // M-tiles that take each B tile in turn
constexpr unsigned long long kF8TimeoutNs = 2000000000ull;

// AR: rows of A that a stage holds.  With fewer than 128 the products read on into what lies behind (the rows of
// their result that come of it are not stored), and more fits.  KS: blocks of 128 along K to a stage, i.e. to a wait.
template <int BN, int AR, int KS>
struct F8Tile {
    static constexpr int A = AR * F8_BK, B = BN * F8_BK, BLOCK = A + B, STAGE = KS * BLOCK;
    static constexpr int STAGES = 196608 / STAGE;  // 192 KB
    static constexpr uint32_t COLS = 2 * BN;       // two accumulators (a power of two, at least 32)
    static constexpr int SMEM = STAGES * STAGE + 1024 + 512 + (F8_BM - AR) * F8_BK;
};

template <int STAGES>
struct F8Shared {
    uint64_t full[STAGES], empty[STAGES];
    uint64_t acc_full[2], acc_empty[2];  // accumulator b computed / read back (128 arrivals)
    uint64_t done;                       // after an error: every product this CTA issued is done
    uint32_t tmem;
    volatile int abort_;
};

struct F8Args {
    const float *sa, *sb;
    void *c;
    int m, n, k, c_dtype, rows_a;  // rows_a: rows of A's box
    uint32_t *err;
    unsigned long long limit;  // of a wait, in ns
};

// The limit is a wait's, from its first failed try on (of up to 20 us, which costs most waits no look at the clock).
// `moves`: a barrier whose phases go by while what is waited for comes nearer (a whole tile's products may take longer than
// the limit): then the limit counts from its last change that was seen.
template <typename S>
__device__ __forceinline__ bool f8_wait(S &s, uint64_t *bar, uint32_t parity, const F8Args &a, uint64_t *moves = nullptr) {
    if (mbar_test_wait(bar, parity) || mbar_try_wait(bar, parity)) return true;
    uint64_t deadline = global_timer_ns() + a.limit;
    bool phase = moves && mbar_test_wait(moves, 0);
    while (!mbar_try_wait(bar, parity)) {
        if (s.abort_) return false;
        const uint64_t now = global_timer_ns();
        if (moves && mbar_test_wait(moves, 0) != phase) {
            phase = !phase;
            deadline = now + a.limit;
        } else if (now > deadline) {
            atomicExch(a.err, 2u);
            s.abort_ = 1;
            return false;
        }
    }
    return true;
}

__device__ __forceinline__ void tc_mma_f8(uint32_t tmem_d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem_d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ void f8_tile_of(int t, int mt, int nt, int &m, int &n) {
    const int per_group = F8_GROUP_M * nt, group = t / per_group, first = group * F8_GROUP_M;
    const int gm = min(F8_GROUP_M, mt - first), r = t - group * per_group;
    m = first + r % gm;
    n = r / gm;
}

template <typename T>
__device__ __forceinline__ T f8_round(float v) {
    if constexpr (sizeof(T) == 4)
        return v;
    else
        return (T)v;
}

// 32 columns of one row, from column `col` on.
template <typename T>
__device__ __forceinline__ void f8_store(T *dst, const float *v, int left) {
    __align__(16) T o[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) o[i] = f8_round<T>(v[i]);
    if (left >= 32 && (reinterpret_cast<uintptr_t>(dst) & 15) == 0) {
#pragma unroll
        for (int i = 0; i < 32 * (int)sizeof(T) / 16; ++i)
            reinterpret_cast<uint4 *>(dst)[i] = reinterpret_cast<const uint4 *>(o)[i];
    } else {
#pragma unroll
        for (int i = 0; i < 32; ++i)
            if (i < left) dst[i] = o[i];
    }
}

template <int BN, int AR, int KS>
__global__ void __launch_bounds__(F8_THREADS, 1)
    matmul_f8_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB, const F8Args a) {
    using L = F8Tile<BN, AR, KS>;
    constexpr int ST = L::STAGES;
    extern __shared__ __align__(1024) uint8_t f8_raw[];
    uint8_t *tiles = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(f8_raw) + 1023) & ~uintptr_t(1023));
    auto &S = *reinterpret_cast<F8Shared<ST> *>(tiles + ST * L::STAGE);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int mt = (a.m + F8_BM - 1) / F8_BM, nt = (a.n + BN - 1) / BN, ntiles = mt * nt;
    const int nk = (a.k + KS * F8_BK - 1) / (KS * F8_BK);  // stages of a tile

    if (threadIdx.x == 0) {
        for (int s = 0; s < ST; ++s) {
            mbar_init(&S.full[s], 1);
            mbar_init(&S.empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&S.acc_full[b], 1);
            mbar_init(&S.acc_empty[b], 128);
        }
        mbar_init(&S.done, 1);
        S.abort_ = 0;
        fence_barrier_init();
        tma_prefetch_map(&tmA);
        tma_prefetch_map(&tmB);
    }
    if (warp == 1) tc_alloc(&S.tmem, L::COLS);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = S.tmem;
    pdl_wait();
    pdl_trigger();
    int kbg = 0;          // the copying lane: stages filled so far (all tiles)
    bool issued = false;  // the lane that issues products has done so

    if (warp == 0) {
        if (lane == 0) {
            int s = 0;        // the next one's place
            uint32_t ph = 1;  // its parity while it is being emptied
            for (int t = blockIdx.x; t < ntiles && !S.abort_; t += gridDim.x) {
                int m, n;
                f8_tile_of(t, mt, nt, m, n);
                for (int kb = 0; kb < nk; ++kb, ++kbg) {
                    if (kbg >= ST && !f8_wait(S, &S.empty[s], ph, a)) break;
                    uint8_t *st = tiles + s * L::STAGE;
                    mbar_arrive_expect_tx(&S.full[s], KS * (a.rows_a * F8_BK + L::B));
#pragma unroll
                    for (int i = 0; i < KS; ++i) {  // (a block past K is zeros)
                        const int x = (kb * KS + i) * F8_BK;
                        tma_load_2d(st + i * L::BLOCK, &tmA, x, m * F8_BM, &S.full[s]);
                        tma_load_2d(st + i * L::BLOCK + L::A, &tmB, x, n * BN, &S.full[s]);
                    }
                    if (++s == ST) s = 0, ph ^= 1u;
                }
            }
        }
    } else if (warp == 1) {
        // The whole warp walks the loop and one lane issues: what the instructions take stays in uniform registers.  What
        // stands between two blocks' products counts (32 to 128 cycles each): one wait a stage, descriptors by addition.
        const bool leader = elect_one();
        // e4m3 operands (type 0), fp32 accumulators, both K-major
        constexpr uint32_t kIdesc = idesc_f16(F8_BM, BN);
        const uint64_t desc = smem_desc_sw128(smem_u32(tiles));
        auto on = [&](uint32_t bytes) { return (desc & 0xffffffff00000000ull) | (uint32_t)((uint32_t)desc + (bytes >> 4)); };
        int lt = 0, s = 0;
        uint32_t ph = 0;
        bool ok = true;
        for (int t = blockIdx.x; ok && t < ntiles; t += gridDim.x, ++lt) {
            const int b = lt & 1;
            const uint32_t acc = tmem + (uint32_t)b * BN;
            if (lt >= 2 && !__all_sync(0xffffffffu, f8_wait(S, &S.acc_empty[b], ((lt >> 1) - 1) & 1u, a))) break;
            for (int kb = 0; kb < nk; ++kb) {
                ok = __all_sync(0xffffffffu, f8_wait(S, &S.full[s], ph, a));
                if (!ok) break;
                tc_fence_after();
                if (leader) {
#pragma unroll
                    for (int kk = 0; kk < KS * F8_BK / 32; ++kk) {  // 32 values = 32 bytes along K per instruction
                        const uint32_t at = (uint32_t)(s * L::STAGE + kk / 4 * L::BLOCK + kk % 4 * 32);
                        tc_mma_f8(acc, on(at), on(at + L::A), kIdesc, (kb | kk) != 0);
                    }
                    tc_commit(&S.empty[s]);
                    issued = true;
                }
                __syncwarp();
                if (++s == ST) s = 0, ph ^= 1u;
            }
            if (ok && leader) tc_commit(&S.acc_full[b]);
            __syncwarp();
        }
    } else {  // warp w reads TMEM lanes 32 * (w % 4) .. + 31
        const int q = warp & 3;
        int lt = 0;
        for (int t = blockIdx.x; t < ntiles; t += gridDim.x, ++lt) {
            int m, n;
            f8_tile_of(t, mt, nt, m, n);
            const int b = lt & 1, row = m * F8_BM + 32 * q + lane;
            const float ra = row < a.m && a.sa ? a.sa[row] : 1.f;
            if (!__all_sync(0xffffffffu, f8_wait(S, &S.acc_full[b], (lt >> 1) & 1u, a, &S.empty[0]))) break;
            tc_fence_after();
            const uint32_t tacc = tmem + (uint32_t)b * BN + ((uint32_t)(32 * q) << 16);
#pragma unroll 1
            for (int c0 = 0; c0 < BN; c0 += 32) {
                const int col = n * BN + c0, left = a.n - col;
                if (left <= 0 || m * F8_BM + 32 * q >= a.m) break;  // (the whole warp)
                float v[32];
                tc_ld32(tacc + (uint32_t)c0, v);
                const float sc = a.sb && lane < left ? a.sb[col + lane] : 1.f;
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] = v[i] * ra * __shfl_sync(0xffffffffu, sc, i);
                if (row < a.m) {
                    const long long at = (long long)row * a.n + col;
                    if (a.c_dtype == LF_F32)
                        f8_store(static_cast<float *>(a.c) + at, v, left);
                    else if (a.c_dtype == LF_F16)
                        f8_store(static_cast<__half *>(a.c) + at, v, left);
                    else
                        f8_store(static_cast<__nv_bfloat16 *>(a.c) + at, v, left);
                }
                __syncwarp();
            }
            tc_fence_before();
            mbar_arrive(&S.acc_empty[b]);
        }
    }
    tc_fence_before();
    __syncthreads();
    // A CTA that gave up has copies and products under way, whichever of its warps gave up first, and in the middle of a tile
    // too: both end (bounded) before it does.
    if (warp == 0 && lane == 0 && S.abort_) {
        const uint64_t dl = global_timer_ns() + 1000000000ull;
        for (int k = kbg > ST ? kbg - ST : 0; k < kbg; ++k)
            while (!mbar_try_wait(&S.full[k % ST], (k / ST) & 1u) && global_timer_ns() < dl) {
            }
    }
    if (warp == 1) {
        if (issued && S.abort_) {
            tc_commit(&S.done);  // (without an error the accumulators' readers have waited for every product)
            const uint64_t dl = global_timer_ns() + 1000000000ull;
            while (!mbar_try_wait(&S.done, 0) && global_timer_ns() < dl) {
            }
        }
        __syncwarp();
        tc_fence_after();
        tc_dealloc(tmem, L::COLS);
    }
}

using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                 const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The limit of a wait.
std::atomic<unsigned long long> f8_limit{kF8TimeoutNs};

EncodeTiled encoder() {
    static EncodeTiled fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiled>(p);
    });
    return fn;
}

// Row-major [rows][k] bytes, boxes of box_rows x 128, 128-byte swizzle, zeros outside.
bool f8_map(CUtensorMap *map, const void *p, int rows, int k, int box_rows) {
    EncodeTiled enc = encoder();
    if (!enc) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)k, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)k};
    const cuuint32_t box[2] = {F8_BK, (cuuint32_t)box_rows}, one[2] = {1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(p), dims, strides, box, one,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int BN, int AR, int KS>
lf_status launch_f8(const void *A, const void *B, F8Args a, int n_sm, cudaStream_t st) {
    using L = F8Tile<BN, AR, KS>;
    a.rows_a = a.m >= AR ? AR : (a.m + 7) / 8 * 8;
    CUtensorMap ma, mb;
    if (!set_smem_once<matmul_f8_kernel<BN, AR, KS>>(L::SMEM) || !f8_map(&ma, A, a.m, a.k, a.rows_a) ||
        !f8_map(&mb, B, a.n, a.k, BN))
        return LF_ERR_CUDA;
    const long long tiles = (((long long)a.m + F8_BM - 1) / F8_BM) * (((long long)a.n + BN - 1) / BN);
    const unsigned grid = (unsigned)(tiles < n_sm ? tiles : n_sm);
    return launch_pdl(matmul_f8_kernel<BN, AR, KS>, grid, F8_THREADS, L::SMEM, st, ma, mb, a) ? LF_OK : LF_ERR_CUDA;
}

}  // namespace
}  // namespace lf

extern "C" lf_status lf_matmul_f8(const void *a_device, const float *a_scale_device, const void *b_device,
                                  const float *b_scale_device, void *c_device, int c_dtype, int m, int n, int k,
                                  uint32_t *err_device, void *cuda_stream) {
    const int bytes = lf::dtype_bytes(c_dtype);
    auto off = [](const void *p, int by) { return reinterpret_cast<uintptr_t>(p) % (unsigned)by != 0; };
    if (!bytes || m < 0 || n < 0 || k < 16 || k % 16 || !a_device || !b_device || !c_device || !err_device ||
        !lf::aligned16(a_device) || !lf::aligned16(b_device) || off(c_device, bytes) || off(a_scale_device, 4) ||
        off(b_scale_device, 4) || off(err_device, 4))
        return LF_ERR_INVALID_ARG;
    // coordinates and tile numbers are 32-bit (the narrowest tiles are 64 wide; the last stage's two blocks end up to 255
    // values behind K)
    if (m > INT32_MAX - 128 || n > INT32_MAX - 256 || k > INT32_MAX - 256 ||
        ((long long)m / 128 + 1) * ((long long)n / 64 + 1) + 4096 > INT32_MAX)
        return LF_ERR_UNSUPPORTED;
    if (m == 0 || n == 0) return LF_OK;
    int dev = 0, n_sm = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&n_sm, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n_sm < 1) {
        (void)cudaGetLastError();
        return LF_ERR_CUDA;
    }
    const lf::F8Args a = {a_scale_device, b_scale_device, c_device, m, n, k, c_dtype, 0, err_device,
                          lf::f8_limit.load(std::memory_order_relaxed)};
    cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
    // The width whose waves over the SMs take the least: a tile of 256, 128 and 64 columns takes as 12 : 7.2 : 5.
    // us by width 64 | 128 | 256, K 4096 (no other K was measured; no K is split):
    //   n  8192, m  128  10.4 | 12.4 | 17.6    200  15.0 | 12.6 | 17.6     384  20.6 | 19.5 | 17.8    1024  43.0 | 34.0 | 29.4
    //   n 14336, m   16  14.2 | 14.2 | 17.8    384  32.3 | 27.9 | 31.0     512  38.7 | 29.1 | 31.5    1024  72.6 | 52.0 | 44.5
    //   n  1024, m   16   8.1 |  8.9 | 13.2
    const long long mt = ((long long)m + 127) / 128;
    auto cost = [&](int bn, int weight) { return (mt * (((long long)n + bn - 1) / bn) + n_sm - 1) / n_sm * weight; };
    const long long c256 = cost(256, 120), c128 = cost(128, 72), c64 = cost(64, 50);
    if (c256 <= c128 && c256 <= c64) return lf::launch_f8<256, 128, 1>(a_device, b_device, a, n_sm, st);
    if (c128 <= c64) return lf::launch_f8<128, 128, 2>(a_device, b_device, a, n_sm, st);
    return m <= 32 ? lf::launch_f8<64, 32, 2>(a_device, b_device, a, n_sm, st) : lf::launch_f8<64, 128, 2>(a_device, b_device, a, n_sm, st);
}

extern "C" lf_status lf_debug_matmul_f8_wait(uint64_t limit_ns) {
    if (limit_ns > lf::kF8TimeoutNs) return LF_ERR_INVALID_ARG;
#ifdef LF_DEBUG
    lf::f8_limit.store(limit_ns, std::memory_order_relaxed);
    return LF_OK;
#else
    return LF_ERR_UNSUPPORTED;
#endif
}
