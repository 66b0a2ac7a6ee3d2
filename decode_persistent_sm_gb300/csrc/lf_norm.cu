// RMSNorm with the residual's addition, and an output in 16, 32 or 8 bits:
//   s = x + r,   y = g s / sqrt(mean(s^2) + eps),
// s rounded once to the residual's type, y to the output's; in 8 bits (e4m3)
// the row's scale max|y| / 448 goes beside it and y / scale is what is rounded.
//
// One pass: a row's values stay in registers (8 to a vector, up to four vectors a
// thread) between the sums and the stores.  max|y| is max|g s| times the row's
// 1 / rms, so the sum of squares and the maximum take one reduction, and y
// itself is computed once.  What bounds it is HBM: every value is read and
// written once.
//
// 3584 x 4096, fp32 and an fp32 residual to 8 bits: 191 MB in 31.6 us, 89 % of the
// rate of a plain copy; 8191 x 7168, all bf16: 470 MB in 79.3 us, 87 %.  16 rows:
// 5.0 us, which is the call.  Narrow rows leave lanes without a value: 100000 x 128,
// bf16, 2.5 TB/s (41 us), 20000 x 1024 6.0.  One vector a thread instead of two (more threads to a
// row, so more to reduce) took 172 us where two took 86; blocks of fewer registers
// (three an SM) 37 where these take 33; loads marked as read once 101 where plain
// ones took 86.
#include <cuda_fp8.h>

#include <algorithm>
#include <type_traits>

#include "lf_paged.h"
#include "lf_ptx.cuh"

namespace lf {
namespace {

constexpr int kNormMaxThreads = 1024, kNormMaxVecs = 4;  // so at most 32768 columns
constexpr int kNormWalkRows = 4;
constexpr float kE4m3Max = 448.f;

struct NormArgs {
    const void *x, *res, *gain;
    void *sum, *out;
    float *scale;
    long long ld_x, ld_res, ld_sum, ld_out;
    int gain_dtype, out_dtype, rows, cols;
    float eps;
    int tpr, rpb;  // threads of a row, rows of a block
};

template <typename T>
__device__ __forceinline__ float to_f(T v) {
    return static_cast<float>(v);
}

// Eight values from p, of which `n` exist (the others are 0), as they lie in memory:
// all loads of a row are on their way before the first value is used.  VEC: all
// eight exist, 16-byte aligned.
template <typename T, bool VEC>
struct Raw {
    __align__(16) T t[8];
    __device__ __forceinline__ void load(const T *p, int n) {
        if constexpr (VEC) {
#pragma unroll
            for (int i = 0; i < (int)sizeof(T) / 2; ++i)
                reinterpret_cast<uint4 *>(t)[i] = n > 0 ? reinterpret_cast<const uint4 *>(p)[i] : make_uint4(0u, 0u, 0u, 0u);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) t[i] = i < n ? p[i] : (T)0.f;
        }
    }
};
template <typename T, bool VEC>
__device__ __forceinline__ void store8(T *p, int n, const float *f) {
    __align__(16) T t[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if constexpr (sizeof(T) == 1)
            t[i] = T(f[i]);
        else if constexpr (sizeof(T) == 4)
            t[i] = f[i];
        else
            t[i] = (T)f[i];
    }
    if constexpr (VEC) {
        if constexpr (sizeof(T) == 1) {
            *reinterpret_cast<uint2 *>(p) = *reinterpret_cast<const uint2 *>(t);
        } else {
#pragma unroll
            for (int i = 0; i < (int)sizeof(T) / 2; ++i)
                reinterpret_cast<uint4 *>(p)[i] = reinterpret_cast<const uint4 *>(t)[i];
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) p[i] = t[i];
    }
}

// y of one vector of g s, in the output's type.
template <bool VEC>
__device__ __forceinline__ void put8(const NormArgs &a, long long at, int n, const float *s, float inv, float scale) {
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = s[i] * inv;
    if (a.out_dtype == LF_E4M3) {
        // one division a vector (eight took 33.4 us where this takes 31.5, 3584 x 4096): at most two more roundings in 24 bits
        // ahead of the one to 4 (the scale of a row of tiny values may have no reciprocal)
        if (scale >= 1e-30f) {
            const float per = 1.f / scale;
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] *= per;
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] /= scale;
        }
        store8<__nv_fp8_e4m3, VEC>(static_cast<__nv_fp8_e4m3 *>(a.out) + at, n, y);
    } else if (a.out_dtype == LF_F32) {
        store8<float, VEC>(static_cast<float *>(a.out) + at, n, y);
    } else if (a.out_dtype == LF_F16) {
        store8<__half, VEC>(static_cast<__half *>(a.out) + at, n, y);
    } else {
        store8<__nv_bfloat16, VEC>(static_cast<__nv_bfloat16 *>(a.out) + at, n, y);
    }
}

// The row's 1 / rms and 8-bit scale from its sum of squares and max |g s|.
__device__ __forceinline__ float2 row_scales(const NormArgs &a, float sq, float mx) {
    const float rms = sqrtf(sq / (float)a.cols + a.eps), inv = 1.f / rms;
    float scale = mx * inv / kE4m3Max;
    if (!(scale > 0.f && scale < INFINITY)) scale = 1.f;  // nothing but zeros, or a NaN or infinity somewhere
    return make_float2(inv, scale);
}

// A NaN among the values is the maximum.
__device__ __forceinline__ float max_nan(float a, float b) {
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}

template <typename TX, typename TR, int V, bool VEC>
__global__ void __launch_bounds__(kNormMaxThreads) add_rmsnorm_kernel(const NormArgs a) {
    __shared__ float2 part[kNormMaxThreads / 32];
    const int sub = threadIdx.x / a.tpr, t = threadIdx.x - sub * a.tpr;
    const long long row = (long long)blockIdx.x * a.rpb + sub;
    const bool live = row < a.rows;
    pdl_wait();
    pdl_trigger();
    const TX *x = static_cast<const TX *>(a.x) + row * a.ld_x;
    const TR *r = static_cast<const TR *>(a.res) + row * a.ld_res;
    auto left = [&](int v) { return live ? a.cols - 8 * (t + v * a.tpr) : 0; };  // values from this vector on
    Raw<TX, VEC> xs[V];
    Raw<TR, VEC> rs[V];
#pragma unroll
    for (int v = 0; v < V; ++v) xs[v].load(x + 8 * (t + v * a.tpr), left(v));
#pragma unroll
    for (int v = 0; v < V; ++v) rs[v].load(r + 8 * (t + v * a.tpr), a.res ? left(v) : 0);
    float s[V][8], sq = 0.f, mx = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            s[v][i] = a.res ? to_f(xs[v].t[i]) + to_f(rs[v].t[i]) : to_f(xs[v].t[i]);
            sq += s[v][i] * s[v][i];
        }
    if (a.sum) {
        TR *d = static_cast<TR *>(a.sum) + row * a.ld_sum;
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (left(v) > 0) store8<TR, VEC>(d + 8 * (t + v * a.tpr), left(v), s[v]);
    }
    // from here on s is g s
    if (a.gain) {
        auto apply = [&](auto *gain) {
            using TG = std::remove_cv_t<std::remove_pointer_t<decltype(gain)>>;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                Raw<TG, VEC> g;
                g.load(gain + 8 * (t + v * a.tpr), left(v));
#pragma unroll
                for (int i = 0; i < 8; ++i) s[v][i] *= to_f(g.t[i]);
            }
        };
        if (a.gain_dtype == LF_F32)
            apply(static_cast<const float *>(a.gain));
        else if (a.gain_dtype == LF_F16)
            apply(static_cast<const __half *>(a.gain));
        else
            apply(static_cast<const __nv_bfloat16 *>(a.gain));
    }
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
        for (int i = 0; i < 8; ++i) mx = max_nan(mx, fabsf(s[v][i]));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        sq += __shfl_xor_sync(0xffffffffu, sq, o);
        mx = max_nan(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    }
    if (a.tpr > 32) {  // a row's warps are neighbours
        const int warps = a.tpr >> 5, w0 = sub * warps;
        if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = make_float2(sq, mx);
        __syncthreads();
        sq = mx = 0.f;
        for (int w = 0; w < warps; ++w) {
            const float2 p = part[w0 + w];
            sq += p.x;
            mx = max_nan(mx, p.y);
        }
    }
    if (!live) return;
    const float2 by = row_scales(a, sq, mx);
    if (a.out_dtype == LF_E4M3 && t == 0) a.scale[row] = by.y;
#pragma unroll
    for (int v = 0; v < V; ++v)
        if (left(v) > 0) put8<VEC>(a, row * a.ld_out + 8 * (t + v * a.tpr), left(v), s[v], by.x, by.y);
}

// The same for many rows of whole vectors: a block walks its rows with the next one on
// its way (kNormStages - 1).  Each thread copies its own vectors into its own places of shared memory
// and reads them back, so that enough is in flight without registers and a
// row costs one barrier; the gain stays in registers.
constexpr int kNormStages = 2;
template <typename TX, typename TR, int V>
__global__ void __launch_bounds__(kNormMaxThreads) add_rmsnorm_rows_kernel(const NormArgs a) {
    constexpr int PX = sizeof(TX) / 2, PR = sizeof(TR) / 2, SLOT = V * (PX + PR);  // 16-byte pieces
    extern __shared__ __align__(16) uint4 norm_ring[];                            // [stage][SLOT][threads]
    __shared__ float2 part[2][kNormMaxThreads / 32];
    const int t = threadIdx.x, warps = a.tpr >> 5;
    pdl_wait();
    pdl_trigger();
    auto fetch = [&](long long row, int stage) {
        if (row < a.rows) {
            uint4 *to = norm_ring + (stage * SLOT) * a.tpr + t;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int at = 8 * (t + v * a.tpr);
                if (at >= a.cols) continue;
                const TX *x = static_cast<const TX *>(a.x) + row * a.ld_x + at;
                const TR *r = static_cast<const TR *>(a.res) + row * a.ld_res + at;
#pragma unroll
                for (int i = 0; i < PX; ++i) cp_async16(to + (v * (PX + PR) + i) * a.tpr, reinterpret_cast<const uint4 *>(x) + i);
                if (a.res) {
#pragma unroll
                    for (int i = 0; i < PR; ++i)
                        cp_async16(to + (v * (PX + PR) + PX + i) * a.tpr, reinterpret_cast<const uint4 *>(r) + i);
                }
            }
        }
        cp_async_commit();
    };
#pragma unroll
    for (int k = 0; k < kNormStages - 1; ++k) fetch(blockIdx.x + (long long)k * gridDim.x, k);
    float g[V][8];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int at = 8 * (t + v * a.tpr);
#pragma unroll
        for (int i = 0; i < 8; ++i) g[v][i] = 1.f;
        if (at >= a.cols || !a.gain) continue;
        auto take = [&](auto *p) {
#pragma unroll
            for (int i = 0; i < 8; ++i) g[v][i] = to_f(p[at + i]);
        };
        if (a.gain_dtype == LF_F32)
            take(static_cast<const float *>(a.gain));
        else if (a.gain_dtype == LF_F16)
            take(static_cast<const __half *>(a.gain));
        else
            take(static_cast<const __nv_bfloat16 *>(a.gain));
    }
    int stage = 0, turn = 0;
    for (long long row = blockIdx.x; row < a.rows; row += gridDim.x, turn ^= 1) {
        fetch(row + (long long)(kNormStages - 1) * gridDim.x, stage == 0 ? kNormStages - 1 : stage - 1);
        asm volatile("cp.async.wait_group %0;" ::"n"(kNormStages - 1) : "memory");
        const uint4 *from = norm_ring + (stage * SLOT) * a.tpr + t;
        stage = stage + 1 == kNormStages ? 0 : stage + 1;
        float s[V][8], sq = 0.f, mx = 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int at = 8 * (t + v * a.tpr);
            __align__(16) TX x[8];
            __align__(16) TR r[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) s[v][i] = 0.f;
            if (at >= a.cols) continue;
#pragma unroll
            for (int i = 0; i < PX; ++i) reinterpret_cast<uint4 *>(x)[i] = from[(v * (PX + PR) + i) * a.tpr];
#pragma unroll
            for (int i = 0; i < 8; ++i) s[v][i] = to_f(x[i]);
            if (a.res) {
#pragma unroll
                for (int i = 0; i < PR; ++i) reinterpret_cast<uint4 *>(r)[i] = from[(v * (PX + PR) + PX + i) * a.tpr];
#pragma unroll
                for (int i = 0; i < 8; ++i) s[v][i] += to_f(r[i]);
            }
            if (a.sum) store8<TR, true>(static_cast<TR *>(a.sum) + row * a.ld_sum + at, 8, s[v]);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                sq += s[v][i] * s[v][i];
                s[v][i] *= g[v][i];
                mx = max_nan(mx, fabsf(s[v][i]));
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            sq += __shfl_xor_sync(0xffffffffu, sq, o);
            mx = max_nan(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        }
        if ((t & 31) == 0) part[turn][t >> 5] = make_float2(sq, mx);
        __syncthreads();  // (the other half of `part` is free: whoever read it has passed this row's barrier's predecessor)
        sq = mx = 0.f;
        for (int w = 0; w < warps; ++w) {
            const float2 p = part[turn][w];
            sq += p.x;
            mx = max_nan(mx, p.y);
        }
        const float2 by = row_scales(a, sq, mx);
        if (a.out_dtype == LF_E4M3 && t == 0) a.scale[row] = by.y;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int at = 8 * (t + v * a.tpr);
            if (at < a.cols) put8<true>(a, row * a.ld_out + at, 8, s[v], by.x, by.y);
        }
    }
}

template <typename TX, typename TR, bool VEC>
bool launch_norm(NormArgs a, int n_sm, cudaStream_t st) {
    const int vecs = (a.cols + 7) / 8;
    // two vectors a thread, four where a block of 1024 threads needs them
    const int v = vecs > 2 * kNormMaxThreads ? 4 : 2;
    a.tpr = ((vecs + v - 1) / v + 31) / 32 * 32;
    a.rpb = std::max(1, 128 / a.tpr);
    if constexpr (VEC && sizeof(TX) == 2 && sizeof(TR) == 2) {
        // From kNormWalkRows rows an SM on, the walk that keeps rows on their way, for 16-bit rows that a block of 288 to 512
        // threads holds (256 where the output is 8 bits).  us, one block a row | walk, bf16 to bf16 and to 8 bits:
        //   4096 columns,  2432 rows  14.5 | -     15.1 | 14.3     8192 rows  45.0 | 48.2   44.7 | 40.6
        //   7168 columns,   608 rows   8.5 | 7.7    8.8 | 8.4      8192 rows  87.7 | 80.8   87.6 | 73.8
        //   8192 columns,  2432 rows  31.0 | 26.3   -   | -        8192 rows  93.3 | 92.8   90.9 | 78.4
        // fp32 rows fill the walk's memory with fewer rows on their way: 31.5 | 47.8 at 3584 x 4096.
        if (v == 2 && a.tpr <= 512 && (a.tpr > 256 || (a.tpr == 256 && a.out_dtype == LF_E4M3)) && a.rows >= kNormWalkRows * n_sm) {
            const int smem = kNormStages * a.tpr * 2 * 8 * (int)(sizeof(TX) + sizeof(TR));
            const int ctas = std::max(1, std::min(227 * 1024 / (smem + 2048), 1024 / a.tpr));
            return set_smem_once<add_rmsnorm_rows_kernel<TX, TR, 2>>(kNormStages * 512 * 2 * 8 * (int)(sizeof(TX) + sizeof(TR))) &&
                   launch_pdl(add_rmsnorm_rows_kernel<TX, TR, 2>, (unsigned)std::min<long long>(a.rows, (long long)ctas * n_sm),
                              (unsigned)a.tpr, (size_t)smem, st, a);
        }
    }
    const unsigned grid = (unsigned)(((long long)a.rows + a.rpb - 1) / a.rpb), threads = (unsigned)(a.tpr * a.rpb);
    return v == 2 ? launch_pdl(add_rmsnorm_kernel<TX, TR, 2, VEC>, grid, threads, 0, st, a)
                  : launch_pdl(add_rmsnorm_kernel<TX, TR, 4, VEC>, grid, threads, 0, st, a);
}

template <typename TX, typename TR>
bool launch_norm_vec(const NormArgs &a, bool vec, int n_sm, cudaStream_t st) {
    return vec ? launch_norm<TX, TR, true>(a, n_sm, st) : launch_norm<TX, TR, false>(a, n_sm, st);
}

template <typename TX>
bool launch_norm_res(const NormArgs &a, int res_dtype, bool vec, int n_sm, cudaStream_t st) {
    return res_dtype == LF_F32   ? launch_norm_vec<TX, float>(a, vec, n_sm, st)
           : res_dtype == LF_F16 ? launch_norm_vec<TX, __half>(a, vec, n_sm, st)
                                 : launch_norm_vec<TX, __nv_bfloat16>(a, vec, n_sm, st);
}

}  // namespace
}  // namespace lf

extern "C" lf_status lf_add_rmsnorm(const void *x_device, int x_dtype, int64_t ld_x, const void *residual_device,
                                    void *sum_device, int residual_dtype, int64_t ld_residual, int64_t ld_sum,
                                    const void *gain_device, int gain_dtype, int rows, int cols, float eps,
                                    void *out_device, int out_dtype, int64_t ld_out, float *scale_device,
                                    void *cuda_stream) {
    using lf::dtype_bytes;
    const int bx = dtype_bytes(x_dtype), br = residual_device || sum_device ? dtype_bytes(residual_dtype) : 4,
              bg = gain_device ? dtype_bytes(gain_dtype) : 4, bo = out_dtype == LF_E4M3 ? 1 : dtype_bytes(out_dtype);
    if (!bx || !br || !bg || !bo || rows < 0 || cols < 1 || !x_device || !out_device || ld_x < cols || ld_out < cols ||
        (residual_device && ld_residual < cols) || (sum_device && ld_sum < cols) || !(eps > 0.f && eps < INFINITY) ||
        (out_dtype == LF_E4M3 && !scale_device))
        return LF_ERR_INVALID_ARG;
    auto off = [](const void *p, int bytes) { return reinterpret_cast<uintptr_t>(p) % (unsigned)bytes != 0; };
    if (off(x_device, bx) || off(residual_device, br) || off(sum_device, br) || off(gain_device, bg) ||
        off(out_device, bo) || off(scale_device, 4))
        return LF_ERR_INVALID_ARG;
    // in place needs the same elements under the same threads
    if ((sum_device == x_device && (x_dtype != residual_dtype || ld_x != ld_sum)) ||
        (sum_device && sum_device == residual_device && ld_residual != ld_sum) || out_device == sum_device)
        return LF_ERR_INVALID_ARG;
    if (out_device == x_device && (x_dtype != out_dtype || ld_x != ld_out)) return LF_ERR_INVALID_ARG;
    if (out_device == residual_device && (residual_dtype != out_dtype || ld_residual != ld_out)) return LF_ERR_INVALID_ARG;
    if (cols > lf::kNormMaxThreads * lf::kNormMaxVecs * 8) return LF_ERR_UNSUPPORTED;
    if (rows == 0) return LF_OK;
    int dev = 0, n_sm = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&n_sm, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n_sm < 1) {
        (void)cudaGetLastError();
        return LF_ERR_CUDA;
    }
    lf::NormArgs a = {x_device, residual_device, gain_device, sum_device, out_device, scale_device, ld_x, ld_residual,
                      ld_sum,   ld_out,          gain_dtype,  out_dtype,  rows,       cols,         eps,  0, 0};
    // 16-byte accesses (8 bytes of an 8-bit output) where every row allows them
    auto fits = [&](const void *p, int64_t ld, int bytes) {
        return !p || (reinterpret_cast<uintptr_t>(p) % (bytes == 1 ? 8u : 16u) == 0 && ld % 8 == 0);
    };
    const bool vec = cols % 8 == 0 && fits(x_device, ld_x, bx) && fits(residual_device, ld_residual, br) &&
                     fits(sum_device, ld_sum, br) && fits(gain_device, 0, bg) && fits(out_device, ld_out, bo);
    cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
    const bool ok = x_dtype == LF_F32   ? lf::launch_norm_res<float>(a, residual_dtype, vec, n_sm, st)
                    : x_dtype == LF_F16 ? lf::launch_norm_res<__half>(a, residual_dtype, vec, n_sm, st)
                                        : lf::launch_norm_res<__nv_bfloat16>(a, residual_dtype, vec, n_sm, st);
    return ok ? LF_OK : LF_ERR_CUDA;
}
