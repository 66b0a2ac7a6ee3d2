// One draw per row of logits under temperature, top-k, top-p and min-p, from
// a given uniform number per row.
//
// With w_i = exp((z_i - max) / T), each filter is a lower bound on the logit:
//   top-k: the k-th largest value;
//   top-p: the largest t with mass{z >= t} >= top_p * mass (both within the
//          top-k set), mass{A} = sum of w over A;
//   min-p: max + T ln(min_p);
// the kept set is z >= the largest of the three, and the token is the first
// kept index whose running kept mass exceeds u times the kept mass.
//
// The answer is a whole number that sums decide, so the sums are exact: a
// weight is a 64-bit integer, 2^44 w rounded, from an exponential whose
// argument is carried as a pair of floats (error about 2^-40 of the weight:
// the fp32 exponential's 2^-22 would put one row in ten of a flat 131072-token
// row on the wrong side of some border).  Integer sums come out the same in
// any order, atomics included.
//
// A row belongs to a cluster of 1, 2, 4 or 8 CTAs, each with a contiguous
// range of the vocabulary in shared memory as fp32: the logits are read from
// HBM once.  A bound is found by a histogram over 1024 equal steps of the
// logit below the maximum (64-bit masses or counts as two 32-bit shared
// atomics, the second only on a carry), summed over the cluster through
// distributed shared memory; the step that holds the border is then refined
// on the float's bits, 10 bits a level, until one value is left (equal logits
// end at once).
#include <cooperative_groups.h>

#include <cfloat>
#include <climits>

#include "laneformer.h"
#include "lf_paged.h"

namespace cg = cooperative_groups;

namespace lf {
namespace {

constexpr int F_THREADS = 512, F_WARPS = F_THREADS / 32;
constexpr int F_BINS = 1024;
constexpr int F_MAX_CLUSTER = 8;
constexpr int F_MAX_VOCAB = 262144;
constexpr int F_FRAC = 44;          // weights are integers in units of 2^-44
constexpr float F_MAX_Y = 45.f;     // below 2^-45 a weight rounds to nothing

using u64 = unsigned long long;

// 2^62 * 2^(-f / 256), f = 0 .. 255 (Taylor series of the exponential).
struct Pow2Table {
    u64 v[256];
    constexpr Pow2Table() : v() {
        for (int f = 0; f < 256; ++f) {
            const double x = -0.69314718055994530942 * f / 256.0;
            double term = 1.0, sum = 1.0;
            for (int i = 1; i < 24; ++i) {
                term *= x / i;
                sum += term;
            }
            v[f] = (u64)(sum * 4611686018427387904.0 + 0.5);
        }
    }
};
__device__ constexpr Pow2Table kPow2;

struct FilterArgs {
    const void *logits;
    int rows, vocab, per;  // per: vocabulary entries of one CTA
    long long ld;
    const float *temperature;
    const int32_t *top_k;
    const float *top_p, *min_p, *u;
    int32_t *token;
    float *logprob;
};

struct Gather {  // one CTA's contribution to a cluster-wide exchange
    u64 a;
    uint32_t b, c;
};

struct FilterShared {
    u64 pow2[256];
    uint32_t lo[F_BINS], hi[F_BINS];
    Gather slot[2][F_MAX_CLUSTER];
    u64 wsum[F_WARPS];
    uint32_t wmin[F_WARPS], wmax[F_WARPS];
    uint32_t found_bin;
    u64 found_before;
    int found;
};

// Order-preserving bits of a float (no NaN; -0 was made +0).
__device__ __forceinline__ uint32_t key_of(float z) {
    const uint32_t b = __float_as_uint(z);
    return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }

// round(2^44 exp((z - max) / T)), (ch, cl) = log2(e) / T as a pair of floats.
// y = (max - z) log2(e) / T as a pair (error 2^-46 of it); y = j / 256 + r;
// 2^-y = 2^(-j / 256) (1 - q), q = 1 - e^(-r ln 2) with r ln 2 = th + tl < 0.0028:
// q = th + (tl - th^2 (1/2 - th / 6 + th^2 / 24)), its tail below 2^-42.
__device__ __forceinline__ u64 weight(float z, float mx, float ch, float cl, const u64 *pow2) {
    if (z == mx) return 1ull << F_FRAC;
    const float s = mx - z;
    const float yh = __fmul_rn(s, ch);
    if (!(yh < F_MAX_Y)) return 0;
    const float bb = __fsub_rn(s, mx);  // mx - z = s + e exactly
    const float e = __fsub_rn(__fsub_rn(mx, __fsub_rn(s, bb)), __fadd_rn(z, bb));
    const float yl = __fmaf_rn(s, ch, -yh) + __fmaf_rn(s, cl, e * ch);
    const int j = __float2int_rd(yh * 256.f);
    const float r = __fmaf_rn((float)j, -1.f / 256.f, yh);
    constexpr float kLn2 = 0.693147182464599609375f, kLn2Lo = -1.904654299957767878541e-9f;
    const float th = __fmul_rn(r, kLn2);
    const float tl = __fmaf_rn(r, kLn2, -th) + __fmaf_rn(r, kLn2Lo, yl * kLn2);
    const float poly = __fmaf_rn(th, __fmaf_rn(th, 1.f / 24.f, -1.f / 6.f), 0.5f);
    const float c = __fmaf_rn(-th * th, poly, tl);
    constexpr float kScale = 549755813888.f;  // 2^39
    const int q = __float2int_rn(th * kScale) + __float2int_rn(c * kScale);
    const u64 t = pow2[j & 255];
    const u64 w62 = t - (u64)(((long long)(t >> 31) * q) >> 8);
    const int sh = 62 - F_FRAC + (j >> 8);
    return (w62 + (1ull << (sh - 1))) >> sh;
}

// The step of a logit below the maximum, monotone in it.
__device__ __forceinline__ int step_of(float z, float mx, float c) {
    return z == mx ? 0 : (int)fminf((mx - z) * c, (float)(F_BINS - 1));
}

__device__ __forceinline__ void hist_add(FilterShared &S, int bin, u64 w) {
    const uint32_t wl = (uint32_t)w;
    uint32_t wh = (uint32_t)(w >> 32);
    const uint32_t old = atomicAdd(&S.lo[bin], wl);
    wh += (old + wl < old) ? 1u : 0u;
    if (wh) atomicAdd(&S.hi[bin], wh);
}

// Every CTA of the cluster gets every CTA's Gather.  `turn` alternates the
// buffers: a CTA can write the next but one exchange only after every CTA has
// passed the next, and so has read this one.
template <int C>
__device__ __forceinline__ const Gather *exchange(FilterShared &S, const Gather &g, int &turn) {
    Gather *mine = S.slot[turn & 1];
    ++turn;
    if constexpr (C == 1) {
        if (threadIdx.x == 0) mine[0] = g;
        __syncthreads();
    } else {
        cg::cluster_group cl = cg::this_cluster();
        if (threadIdx.x < C) cl.map_shared_rank(mine, threadIdx.x)[cl.block_rank()] = g;
        cl.sync();
    }
    return mine;
}

// Block-wide (min, max) of keys; every thread gets it.
__device__ __forceinline__ void block_minmax(FilterShared &S, uint32_t &mn, uint32_t &mx) {
    mn = __reduce_min_sync(0xffffffffu, mn);
    mx = __reduce_max_sync(0xffffffffu, mx);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) S.wmin[threadIdx.x >> 5] = mn, S.wmax[threadIdx.x >> 5] = mx;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < F_WARPS; ++w) {
        mn = min(mn, S.wmin[w]);
        mx = max(mx, S.wmax[w]);
    }
}

__device__ __forceinline__ u64 warp_sum(u64 v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Finds, in the cluster's summed histogram (bins in falling order of the
// logit), the bin where `above` + the running sum reaches the target, and
// `before`, above + the sum of the bins before it.  With frac >= 0 the target
// is first set to ceil(frac * total).
template <int C>
__device__ int find_bin(FilterShared &S, u64 above, u64 &target, double frac, int rank, int &turn, u64 &before) {
    constexpr int SL = F_BINS / C;                       // bins of this CTA's slice
    constexpr int PT = (SL + F_THREADS - 1) / F_THREADS;  // bins per thread (1 or 2)
    if constexpr (C == 1)
        __syncthreads();
    else
        cg::this_cluster().sync();  // every CTA's histogram is complete
    u64 v[PT], sum = 0;
    const int b0 = threadIdx.x * PT;
#pragma unroll
    for (int i = 0; i < PT; ++i) {
        v[i] = 0;
        if (b0 + i < SL) {
#pragma unroll
            for (int r = 0; r < C; ++r) {
                const uint32_t *lo = S.lo, *hi = S.hi;
                if constexpr (C > 1) {
                    lo = cg::this_cluster().map_shared_rank(S.lo, r);
                    hi = cg::this_cluster().map_shared_rank(S.hi, r);
                }
                v[i] += ((u64)hi[rank * SL + b0 + i] << 32) + lo[rank * SL + b0 + i];
            }
        }
        sum += v[i];
    }
    u64 inc = sum;  // inclusive scan over the slice
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const u64 y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
    }
    if (lane == 31) S.wsum[w] = inc;
    if (threadIdx.x == 0) S.found = 0;
    __syncthreads();
    u64 all = 0;
#pragma unroll
    for (int i = 0; i < F_WARPS; ++i) {
        if (i < w) inc += S.wsum[i];
        all += S.wsum[i];
    }
    const Gather *got = exchange<C>(S, Gather{all, 0u, 0u}, turn);
    u64 at = above + inc - sum, total = 0;
#pragma unroll
    for (int r = 0; r < C; ++r) {
        if (r < rank) at += got[r].a;
        total += got[r].a;
    }
    if (frac >= 0.0) target = max(1ull, (u64)ceil(frac * (double)total));
#pragma unroll
    for (int i = 0; i < PT; ++i) {
        if (at < target && target <= at + v[i]) {
            S.found = 1;
            S.found_bin = (uint32_t)(rank * SL + b0 + i);
            S.found_before = at;
        }
        at += v[i];
    }
    __syncthreads();
    got = exchange<C>(S, Gather{S.found_before, S.found_bin, (uint32_t)S.found}, turn);
    int bin = F_BINS - 1;
    before = above;
#pragma unroll
    for (int r = 0; r < C; ++r)
        if (got[r].c) {
            bin = (int)got[r].b;
            before = got[r].a;
        }
    return bin;
}

struct RowScale {
    float mx, ch, cl, step;  // the maximum, log2(e) / T as a pair, histogram steps per unit of logit
};

// The key of the largest value t for which A{z >= t} reaches its target, over
// the elements with z >= floor: A counts and the target is k, or (MASS) A is
// the mass and the target top_p of the whole.
template <int C, bool MASS>
__device__ uint32_t select_bound(FilterShared &S, const float *z, int n, const RowScale &rs, float floor, u64 k,
                                 double top_p, int rank, int &turn) {
    const int tid = threadIdx.x;
    for (int i = tid; i < F_BINS; i += F_THREADS) S.lo[i] = S.hi[i] = 0;
    __syncthreads();
    for (int i = tid; i < n; i += F_THREADS) {
        const float x = z[i];
        if (!(x >= floor)) continue;
        const u64 w = MASS ? weight(x, rs.mx, rs.ch, rs.cl, S.pow2) : 1ull;
        if (w) hist_add(S, step_of(x, rs.mx, rs.step), w);
    }
    u64 target = k, above = 0;
    const int step = find_bin<C>(S, 0, target, MASS ? top_p : -1.0, rank, turn, above);
    uint32_t kmin = 0xffffffffu, kmax = 0;  // the keys in that step
    for (int i = tid; i < n; i += F_THREADS) {
        const float x = z[i];
        if (x >= floor && step_of(x, rs.mx, rs.step) == step) {
            kmin = min(kmin, key_of(x));
            kmax = max(kmax, key_of(x));
        }
    }
    block_minmax(S, kmin, kmax);
    const Gather *got = exchange<C>(S, Gather{0ull, kmin, kmax}, turn);
#pragma unroll
    for (int r = 0; r < C; ++r) {
        kmin = min(kmin, got[r].b);
        kmax = max(kmax, got[r].c);
    }
    // refine: the keys of [kmin, kmax] in 1024 equal runs, until one key is
    // left (a run of keys holds no element of another step: steps are
    // monotone; 10 bits a level, so at most 4 levels)
    while (kmin < kmax) {
        int shift = 0;
        while (((kmax - kmin) >> shift) >= (uint32_t)F_BINS) ++shift;
        for (int i = tid; i < F_BINS; i += F_THREADS) S.lo[i] = S.hi[i] = 0;
        __syncthreads();
        for (int i = tid; i < n; i += F_THREADS) {
            const float x = z[i];
            const uint32_t key = key_of(x);
            if (key < kmin || key > kmax) continue;
            const u64 w = MASS ? weight(x, rs.mx, rs.ch, rs.cl, S.pow2) : 1ull;
            if (w) hist_add(S, (int)((kmax - key) >> shift), w);
        }
        u64 before = 0;
        const uint32_t bin = (uint32_t)find_bin<C>(S, above, target, -1.0, rank, turn, before);
        above = before;
        kmax -= min(bin << shift, kmax - kmin);
        kmin = max(kmin, kmax - min(kmax, (1u << shift) - 1u));
    }
    return kmax;
}

__device__ __forceinline__ float of_key(uint32_t k) {
    return __uint_as_float((k & 0x80000000u) ? k & 0x7fffffffu : ~k);
}

template <typename T, int C>
__global__ void __launch_bounds__(F_THREADS) sample_filtered_kernel(const FilterArgs a) {
    extern __shared__ float z[];  // this CTA's logits
    __shared__ FilterShared S;
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    const int row = blockIdx.x / C, rank = blockIdx.x % C;
    const int i0 = rank * a.per, n = max(0, min(a.per, a.vocab - i0));
    int turn = 0;
    const T *src = static_cast<const T *>(a.logits) + (long long)row * a.ld + i0;

    for (int i = tid; i < 256; i += F_THREADS) S.pow2[i] = kPow2.v[i];
    const float t = a.temperature ? a.temperature[row] : 1.f, top_p = a.top_p ? a.top_p[row] : 1.f;
    const float min_p = a.min_p ? a.min_p[row] : 0.f, u = a.u[row];
    const int top_k = a.top_k ? a.top_k[row] : 0;

    // load; the largest and smallest finite keys, and whether there is a NaN
    uint32_t kmax = 0, kmin = 0xffffffffu;
    bool nan = false;
    for (int i = tid; i < n; i += F_THREADS) {
        const float x = to_f32(src[i]) + 0.f;  // -0 becomes +0: one key per value
        z[i] = x;
        nan |= x != x;
        kmax = max(kmax, key_of(x));
        if (x > -INFINITY) kmin = min(kmin, key_of(x));
    }
    nan = __syncthreads_or(nan);
    block_minmax(S, kmin, kmax);
    const Gather *got = exchange<C>(S, Gather{nan ? 1ull : 0ull, kmin, kmax}, turn);
#pragma unroll
    for (int r = 0; r < C; ++r) {
        nan |= got[r].a != 0;
        kmin = min(kmin, got[r].b);
        kmax = max(kmax, got[r].c);
    }
    const float mx = of_key(kmax);
    const bool bad = nan || !(mx > -INFINITY) || !(t == 0.f || (t >= 1e-30f && t <= 1e30f)) || !(top_p > 0.f && top_p <= 1.f) ||
                     !(min_p >= 0.f && min_p <= 1.f) || !(u >= 0.f && u < 1.f);
    if (bad) {
        if (rank == 0 && tid == 0) {
            a.token[row] = -1;
            if (a.logprob) a.logprob[row] = __int_as_float(0x7fffffff);
        }
        return;
    }
    if (t == 0.f) {  // greedy
        uint32_t first = 0xffffffffu, unused = 0;
        for (int i = tid; i < n; i += F_THREADS)
            if (z[i] == mx) {
                first = (uint32_t)(i0 + i);
                break;
            }
        block_minmax(S, first, unused);
        got = exchange<C>(S, Gather{0ull, first, 0u}, turn);
#pragma unroll
        for (int r = 0; r < C; ++r) first = min(first, got[r].b);
        if (rank == 0 && tid == 0) {
            a.token[row] = (int)first;
            if (a.logprob) a.logprob[row] = 0.f;
        }
        return;
    }

    RowScale rs;
    const double cd = 1.4426950408889634074 / (double)t;
    rs.mx = mx;
    rs.ch = (float)cd;
    rs.cl = (float)(cd - (double)rs.ch);
    // 16 steps per factor of 2 in weight, finer where the whole row spans less
    rs.step = fmaxf(16.f * rs.ch, (float)(F_BINS - 1) / (mx - of_key(kmin)));

    float floor = -INFINITY;
    if (top_k > 0 && top_k < a.vocab)
        floor = of_key(select_bound<C, false>(S, z, n, rs, -INFINITY, (u64)top_k, 0.0, rank, turn));
    if (top_p < 1.f)
        floor = fmaxf(floor, of_key(select_bound<C, true>(S, z, n, rs, floor, 0ull, (double)top_p, rank, turn)));
    if (min_p > 0.f) floor = fmaxf(floor, __double2float_ru((double)mx + (double)t * log((double)min_p)));

    // the kept mass: each warp owns a contiguous range of the CTA's
    const int per_w = (n + F_WARPS - 1) / F_WARPS, r0 = min(n, w * per_w), r1 = min(n, r0 + per_w);
    u64 mine = 0;
    for (int i = r0 + lane; i < r1; i += 32)
        if (z[i] >= floor) mine += weight(z[i], mx, rs.ch, rs.cl, S.pow2);
    mine = warp_sum(mine);
    if (lane == 0) S.wsum[w] = mine;
    __syncthreads();
    u64 before = 0, all = 0;
#pragma unroll
    for (int i = 0; i < F_WARPS; ++i) {
        if (i < w) before += S.wsum[i];
        all += S.wsum[i];
    }
    got = exchange<C>(S, Gather{all, 0u, 0u}, turn);
    u64 total = 0;
#pragma unroll
    for (int r = 0; r < C; ++r) {
        if (r < rank) before += got[r].a;
        total += got[r].a;
    }
    const u64 goal = (u64)((double)u * (double)total);  // running > u * total <=> running > goal
    if (before > goal || goal >= before + mine) return;
    // this warp's range holds the crossing
    for (int c0 = r0; c0 < r1; c0 += 32) {
        const int i = c0 + lane;
        const float x = i < r1 ? z[i] : -INFINITY;
        const u64 wt = i < r1 && x >= floor ? weight(x, mx, rs.ch, rs.cl, S.pow2) : 0ull;
        u64 inc = wt;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const u64 y = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += y;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, before + inc > goal);
        if (hit) {
            if (lane == __ffs(hit) - 1) {
                a.token[row] = i0 + i;
                if (a.logprob) {  // from the logit, not from its rounded weight
                    const double d = x == mx ? 0.0 : ((double)x - (double)mx) / (double)t;
                    a.logprob[row] = (float)(d - log((double)total * 5.684341886080801e-14));  // 2^-44
                }
            }
            return;
        }
        before += __shfl_sync(0xffffffffu, inc, 31);
    }
}

constexpr int kMaxPer = 49152;  // logits of one CTA: 192 KB

template <typename T, int C>
lf_status launch_row(const FilterArgs &a, cudaStream_t st) {
    if (!set_smem_once<sample_filtered_kernel<T, C>>(kMaxPer * (int)sizeof(float))) return LF_ERR_CUDA;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.rows * C));
    cfg.blockDim = dim3(F_THREADS);
    cfg.dynamicSmemBytes = (size_t)a.per * sizeof(float);
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)C;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, sample_filtered_kernel<T, C>, a) != cudaSuccess) {
        (void)cudaGetLastError();
        return LF_ERR_CUDA;
    }
    return LF_OK;
}

template <int C>
lf_status launch_cluster(const FilterArgs &a, int dtype, cudaStream_t st) {
    return dtype == LF_F32   ? launch_row<float, C>(a, st)
           : dtype == LF_F16 ? launch_row<__half, C>(a, st)
                             : launch_row<__nv_bfloat16, C>(a, st);
}

lf_status launch_filtered(FilterArgs a, int dtype, cudaStream_t st) {
    int dev = 0, n_sm = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&n_sm, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
        (void)cudaGetLastError();
        return LF_ERR_CUDA;
    }
    int c = 1;
    while (c < F_MAX_CLUSTER && ((a.vocab + c - 1) / c > kMaxPer || (a.rows * c < n_sm && a.vocab / c > 2048))) c *= 2;
    a.per = ((a.vocab + c - 1) / c + 7) / 8 * 8;
    switch (c) {
        case 1: return launch_cluster<1>(a, dtype, st);
        case 2: return launch_cluster<2>(a, dtype, st);
        case 4: return launch_cluster<4>(a, dtype, st);
        default: return launch_cluster<8>(a, dtype, st);
    }
}

}  // namespace
}  // namespace lf

extern "C" lf_status lf_sample_filtered(const void *logits_device, int dtype, int rows, int vocab, int64_t ld,
                                        const float *temperature_device, const int32_t *top_k_device,
                                        const float *top_p_device, const float *min_p_device, const float *u_device,
                                        int32_t *token_device, float *logprob_device, void *cuda_stream) {
    const int bytes = lf::dtype_bytes(dtype);
    auto off = [](const void *p, int b) { return (reinterpret_cast<uintptr_t>(p) & (uintptr_t)(b - 1)) != 0; };
    if (!bytes || !logits_device || !u_device || !token_device || rows < 0 || vocab < 1 || ld < vocab ||
        off(logits_device, bytes) || off(temperature_device, 4) || off(top_k_device, 4) || off(top_p_device, 4) ||
        off(min_p_device, 4) || off(u_device, 4) || off(token_device, 4) || off(logprob_device, 4))
        return LF_ERR_INVALID_ARG;
    if (vocab > lf::F_MAX_VOCAB) return LF_ERR_UNSUPPORTED;
    if (rows > (1 << 24)) return LF_ERR_INVALID_ARG;
    if (rows == 0) return LF_OK;
    lf::FilterArgs a = {};
    a.logits = logits_device;
    a.rows = rows;
    a.vocab = vocab;
    a.ld = ld;
    a.temperature = temperature_device;
    a.top_k = top_k_device;
    a.top_p = top_p_device;
    a.min_p = min_p_device;
    a.u = u_device;
    a.token = token_device;
    a.logprob = logprob_device;
    return lf::launch_filtered(a, dtype, static_cast<cudaStream_t>(cuda_stream));
}
