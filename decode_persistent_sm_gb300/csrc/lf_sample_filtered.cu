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
// HBM once.  A bound is found in two stages.  First a histogram over 1024
// equal steps of the logit below the maximum, summed over the cluster through
// distributed shared memory, leaves few candidates:
//   top-k: the threads' own maxima are counted; k of them at or above a step
//          mean that the k-th largest logit is there too, so everything below
//          drops out (for k above half the threads: every logit is counted);
//   top-p: the masses of all logits (64 bits as two 32-bit shared atomics, the
//          second only on a carry) name the step that holds the border.
// The candidates' values are then gathered in every CTA and ranked against
// each other; a top-k set that was gathered serves top-p as well.  More
// candidates than the list holds (equal or close logits) are told apart on
// their float's bits, 10 a level.

#include <cooperative_groups.h>

#include <cfloat>
#include <climits>

#include "laneformer.h"
#include "lf_paged.h"

namespace cg = cooperative_groups;

namespace lf {
namespace {

constexpr int F_BINS = 1024;
constexpr int F_LIST = 320;  // candidates that are ranked pairwise: 320^2 comparisons take about 1 us of one SM
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
    int dtype, rows, vocab, per;  // per: vocabulary entries of one CTA
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

struct RowScale {
    float mx, ch, cl, step;  // the maximum, log2(e) / T as a pair, histogram steps per unit of logit
};

struct FilterShared {
    u64 pow2[256];
    uint32_t lo[F_BINS], hi[F_BINS];
    float cand[F_LIST];      // this CTA's candidates
    float all[F_LIST];       // the cluster's
    u64 mass[F_LIST];        // their weights
    Gather slot[2][F_MAX_CLUSTER];
    u64 wsum[32];
    uint32_t wmin[32], wmax[32];
    u64 found_before, target;
    double ln_min_p;         // T ln(min_p)
    float ch, cl, floor;
    uint32_t found_bin, key;
    int found, n_cand;
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

__device__ __forceinline__ u64 warp_sum(u64 v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

__device__ __forceinline__ float of_key(uint32_t k) {
    return __uint_as_float((k & 0x80000000u) ? k & 0x7fffffffu : ~k);
}

template <int NT, int C>
struct Row {
    static constexpr int NW = NT / 32;
    FilterShared &S;
    const float4 *z4;  // this CTA's logits, -inf past n up to a multiple of 4
    int n4, rank, tid, lane, w;
    int turn = 0;
    RowScale rs;

    __device__ Row(FilterShared &s, const float *z, int n, int r)
        : S(s), z4(reinterpret_cast<const float4 *>(z)), n4((n + 3) / 4), rank(r), tid(threadIdx.x),
          lane(threadIdx.x & 31), w(threadIdx.x >> 5) {}

    // f(value) for every logit of this CTA
    template <class F>
    __device__ __forceinline__ void each(F f) const {
#pragma unroll 2
        for (int i = tid; i < n4; i += NT) {
            const float4 x = z4[i];
            f(x.x);
            f(x.y);
            f(x.z);
            f(x.w);
        }
    }

    // Every CTA of the cluster gets every CTA's Gather.  `turn` alternates the
    // buffers: a CTA can write the next but one exchange only after every CTA
    // has passed the next, and so has read this one.
    __device__ __forceinline__ const Gather *exchange(const Gather &g) {
        Gather *mine = S.slot[turn & 1];
        ++turn;
        if constexpr (C == 1) {
            if (tid == 0) mine[0] = g;
            __syncthreads();
        } else {
            cg::cluster_group cl = cg::this_cluster();
            if (tid < C) cl.map_shared_rank(mine, tid)[rank] = g;
            cl.sync();
        }
        return mine;
    }
    __device__ __forceinline__ void sync() const {
        if constexpr (C == 1)
            __syncthreads();
        else
            cg::this_cluster().sync();
    }

    // Block-wide (min, max); every thread gets it.
    __device__ __forceinline__ void block_minmax(uint32_t &mn, uint32_t &mx) {
        mn = __reduce_min_sync(0xffffffffu, mn);
        mx = __reduce_max_sync(0xffffffffu, mx);
        __syncthreads();
        if (lane == 0) S.wmin[w] = mn, S.wmax[w] = mx;
        __syncthreads();
        mn = __reduce_min_sync(0xffffffffu, lane < NW ? S.wmin[lane] : 0xffffffffu);
        mx = __reduce_max_sync(0xffffffffu, lane < NW ? S.wmax[lane] : 0u);
    }

    __device__ __forceinline__ u64 weight_of(float x) const { return weight(x, rs.mx, rs.ch, rs.cl, S.pow2); }
    __device__ __forceinline__ int step(float x) const { return step_of(x, rs.mx, rs.step); }

    __device__ void clear_hist() {
        for (int i = tid; i < F_BINS; i += NT) S.lo[i] = S.hi[i] = 0;
        if (tid == 0) S.n_cand = 0;
        __syncthreads();
    }

    // Finds, in the cluster's summed histogram (bins in falling order of the
    // logit), the bin where `above` + the running sum reaches the target, and
    // `before`, above + the sum of the bins before it.  With frac >= 0 the
    // target is first set to ceil(frac * total).
    __device__ int find_bin(u64 above, u64 &target, float frac, u64 &before) {
        constexpr int SL = F_BINS / C;            // bins of this CTA's slice
        constexpr int PT = (SL + NT - 1) / NT;    // bins per thread (1 or 2)
        sync();  // every CTA's histogram is complete
        u64 v[PT], sum = 0;
        const int b0 = tid * PT;
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
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const u64 y = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += y;
        }
        if (lane == 31) S.wsum[w] = inc;
        if (tid == 0) S.found = 0;
        __syncthreads();
        const u64 ws = lane < NW ? S.wsum[lane] : 0;
        const u64 all = warp_sum(ws);
        inc += warp_sum(lane < w ? ws : 0ull);
        const Gather *got = exchange(Gather{all, 0u, 0u});
        u64 at = above + inc - sum, total = 0;
#pragma unroll
        for (int r = 0; r < C; ++r) {
            if (r < rank) at += got[r].a;
            total += got[r].a;
        }
        if (frac >= 0.f) {
            if (tid == 0) S.target = max(1ull, (u64)ceil((double)frac * (double)total));
            __syncthreads();
            target = S.target;
        }
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
        got = exchange(Gather{S.found_before, S.found_bin, (uint32_t)S.found});
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

    // Collects the logits for which take(value) holds: up to F_LIST of them in
    // S.all of every CTA.  Returns how many there are in the cluster (above
    // F_LIST: not collected) and their smallest and largest keys.
    template <class Take>
    __device__ int collect(Take take, uint32_t &kmin, uint32_t &kmax) {
        kmin = 0xffffffffu, kmax = 0;
        each([&](float x) {
            if (take(x)) {
                const uint32_t k = key_of(x);
                kmin = min(kmin, k);
                kmax = max(kmax, k);
                const int at = atomicAdd(&S.n_cand, 1);
                if (at < F_LIST) S.cand[at] = x;
            }
        });
        block_minmax(kmin, kmax);
        const int mine = S.n_cand;
        const Gather *got = exchange(Gather{(u64)mine, kmin, kmax});
        int total = 0, count[C], first[C];
#pragma unroll
        for (int r = 0; r < C; ++r) {
            kmin = min(kmin, got[r].b);
            kmax = max(kmax, got[r].c);
            first[r] = total;
            count[r] = (int)got[r].a;
            total += count[r];
        }
        if (total <= F_LIST) {
#pragma unroll
            for (int r = 0; r < C; ++r) {
                const float *src = S.cand;
                if constexpr (C > 1) src = cg::this_cluster().map_shared_rank(S.cand, r);
                for (int i = tid; i < count[r]; i += NT) S.all[first[r] + i] = src[i];
            }
            __syncthreads();
        }
        return total;
    }

    // Among the m gathered values: the key of the value at which the count of
    // values at or above it reaches k.
    __device__ uint32_t rank_count(int m, int k) {
        if (tid < m) {
            const float x = S.all[tid];
            int gt = 0, ge = 0;
            for (int j = 0; j < m; ++j) {
                const float y = S.all[j];
                gt += y > x ? 1 : 0;
                ge += y >= x ? 1 : 0;
            }
            if (gt < k && k <= ge) S.key = key_of(x);
        }
        __syncthreads();
        return S.key;
    }
    // The same by mass, over the values at or above `floor`: above + their
    // mass reaches the target (or, with frac >= 0, ceil(frac * their mass)).
    __device__ uint32_t rank_mass(int m, float floor, u64 above, u64 target, float frac) {
        u64 mine = 0;
        if (tid < m && S.all[tid] >= floor) mine = weight_of(S.all[tid]);
        if (tid < m) S.mass[tid] = mine;
        if (frac >= 0.f) {
            const u64 sum = warp_sum(mine);
            if (lane == 0) S.wsum[w] = sum;
            __syncthreads();
            if (w == 0) {
                const u64 all = warp_sum(lane < NW ? S.wsum[lane] : 0ull);
                if (lane == 0) S.target = max(1ull, (u64)ceil((double)frac * (double)all));
            }
        }
        __syncthreads();
        if (frac >= 0.f) target = S.target;
        if (mine) {
            const float x = S.all[tid];
            u64 gt = above, eq = 0;
            for (int j = 0; j < m; ++j) {
                const float y = S.all[j];
                const u64 wj = S.mass[j];
                gt += y > x ? wj : 0ull;
                eq += y == x ? wj : 0ull;
            }
            if (gt < target && target <= gt + eq) S.key = key_of(x);
        }
        __syncthreads();
        return S.key;
    }

    // The border among the keys of [kmin, kmax], which hold every candidate and
    // nothing else from `floor` on: 1024 equal runs of keys a level, until one
    // key is left.  (10 bits a level: at most 4 levels.)
    template <bool MASS>
    __device__ uint32_t refine(uint32_t kmin, uint32_t kmax, u64 above, u64 target) {
        while (kmin < kmax) {
            int shift = 0;
            while (((kmax - kmin) >> shift) >= (uint32_t)F_BINS) ++shift;
            clear_hist();
            each([&](float x) {
                const uint32_t key = key_of(x);
                if (key < kmin || key > kmax) return;
                const u64 wt = MASS ? weight_of(x) : 1ull;
                if (wt) hist_add(S, (int)((kmax - key) >> shift), wt);
            });
            u64 before = 0;
            const uint32_t bin = (uint32_t)find_bin(above, target, -1.f, before);
            above = before;
            kmax -= min(bin << shift, kmax - kmin);
            kmin = max(kmin, kmax - min(kmax, (1u << shift) - 1u));
        }
        return kmax;
    }

    // The key of the k-th largest logit, 0 < k < vocabulary.  `m` gets the
    // number of gathered values if they hold the whole top-k set, else 0.
    __device__ uint32_t top_k_key(int k, int vocab, float thread_max, int &m) {
        clear_hist();
        // (the padding behind the vocabulary is -inf, the same as a masked logit:
        // it lies below every logit or equals the smallest, so it changes no bound above -inf)
        if (2 * k <= NT * C) {
            hist_add(S, step(thread_max), 1ull);
        } else {
            each([&](float x) { hist_add(S, step(x), 1ull); });
        }
        u64 target = (u64)k, before = 0;
        const int last = find_bin(0ull, target, -1.f, before);
        uint32_t kmin, kmax;
        const int total = collect([&](float x) { return step(x) <= last; }, kmin, kmax);
        m = total <= F_LIST ? total : 0;
        if (m) return rank_count(m, k);
        return refine<false>(kmin, kmax, 0ull, (u64)k);
    }

    // The key of the nucleus border over the logits at or above `floor`.
    __device__ uint32_t top_p_key(float floor, float top_p) {
        clear_hist();
        each([&](float x) {
            if (!(x >= floor)) return;
            const u64 wt = weight_of(x);
            if (wt) hist_add(S, step(x), wt);
        });
        u64 target = 0, before = 0;
        const int border = find_bin(0ull, target, top_p, before);
        uint32_t kmin, kmax;
        const int total = collect([&](float x) { return x >= floor && step(x) == border; }, kmin, kmax);
        if (kmin == kmax) return kmax;
        if (total <= F_LIST) return rank_mass(total, floor, before, target, -1.f);
        return refine<true>(kmin, kmax, before, target);
    }
};

// Reads n logits as fp32 into shared memory (16-byte loads where the row is
// aligned for them); returns the thread's largest key, and through nan and kmin
// whether it saw a NaN and its smallest key above -inf.
template <typename T, int NT>
__device__ __forceinline__ uint32_t load_row(const T *src, int n, float *z, bool &nan, uint32_t &kmin) {
    constexpr int V = 16 / sizeof(T);
    uint32_t kmax = 0;
    auto take = [&](float x) {
        nan |= x != x;
        const uint32_t k = key_of(x);
        kmax = max(kmax, k);
        if (x > -INFINITY) kmin = min(kmin, k);
    };
    int done = 0;
    if ((reinterpret_cast<uintptr_t>(src) & 15u) == 0) {
        const int nv = n / V;
        done = nv * V;
#pragma unroll 4
        for (int i = threadIdx.x; i < nv; i += NT) {
            const uint4 raw = __ldg(reinterpret_cast<const uint4 *>(src) + i);
            const T *t = reinterpret_cast<const T *>(&raw);
            float x[V];
#pragma unroll
            for (int j = 0; j < V; ++j) {
                x[j] = to_f32(t[j]) + 0.f;  // -0 becomes +0: one key per value
                take(x[j]);
            }
#pragma unroll
            for (int j = 0; j < V; j += 4)
                reinterpret_cast<float4 *>(z)[(i * V + j) / 4] = make_float4(x[j], x[j + 1], x[j + 2], x[j + 3]);
        }
    }
#pragma unroll 4
    for (int i = done + threadIdx.x; i < n; i += NT) {
        const float x = to_f32(src[i]) + 0.f;
        z[i] = x;
        take(x);
    }
    if (threadIdx.x < ((4 - n % 4) & 3)) z[n + threadIdx.x] = -INFINITY;
    return kmax;
}

template <int NT, int C>
__global__ void __launch_bounds__(NT) sample_filtered_kernel(const FilterArgs a) {
    extern __shared__ __align__(16) float z[];  // this CTA's logits
    __shared__ FilterShared S;
    constexpr int NW = NT / 32;
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    const int row = blockIdx.x / C, rank = blockIdx.x % C;
    const int i0 = rank * a.per, n = max(0, min(a.per, a.vocab - i0));
    Row<NT, C> R(S, z, n, rank);
    for (int i = tid; i < 256; i += NT) S.pow2[i] = kPow2.v[i];
    pdl_wait();
    pdl_trigger();

    const float t = a.temperature ? a.temperature[row] : 1.f, top_p = a.top_p ? a.top_p[row] : 1.f;
    const float min_p = a.min_p ? a.min_p[row] : 0.f, u = a.u[row];
    const int top_k = a.top_k ? a.top_k[row] : 0;
    const bool fine = (t == 0.f || (t >= 1e-30f && t <= 1e30f)) && top_p > 0.f && top_p <= 1.f && min_p >= 0.f &&
                      min_p <= 1.f && u >= 0.f && u < 1.f;
    if (!fine) {  // every CTA of the row sees the same
        if (rank == 0 && tid == 0) {
            a.token[row] = -1;
            if (a.logprob) a.logprob[row] = __int_as_float(0x7fffffff);
        }
        return;
    }
    const long long at = (long long)row * a.ld + i0;
    uint32_t kmin = 0xffffffffu;
    bool nan = false;
    const uint32_t own = a.dtype == LF_F32 ? load_row<float, NT>(static_cast<const float *>(a.logits) + at, n, z, nan, kmin)
                         : a.dtype == LF_F16
                             ? load_row<__half, NT>(static_cast<const __half *>(a.logits) + at, n, z, nan, kmin)
                             : load_row<__nv_bfloat16, NT>(static_cast<const __nv_bfloat16 *>(a.logits) + at, n, z, nan, kmin);
    // 64-bit arithmetic is slow (and the same for every thread): one thread of
    // the last warp does the row's
    if (tid == NT - 32 && t > 0.f) {
        const double cd = 1.4426950408889634074 / (double)t;
        S.ch = (float)cd;
        S.cl = (float)(cd - (double)S.ch);
        if (min_p > 0.f) S.ln_min_p = (double)t * log((double)min_p);
    }
    uint32_t kmax = own;
    nan = __syncthreads_or(nan);
    R.block_minmax(kmin, kmax);
    const Gather *got = R.exchange(Gather{nan ? 1ull : 0ull, kmin, kmax});
#pragma unroll
    for (int r = 0; r < C; ++r) {
        nan |= got[r].a != 0;
        kmin = min(kmin, got[r].b);
        kmax = max(kmax, got[r].c);
    }
    const float mx = of_key(kmax);
    if (nan || !(mx > -INFINITY)) {
        if (rank == 0 && tid == 0) {
            a.token[row] = -1;
            if (a.logprob) a.logprob[row] = __int_as_float(0x7fffffff);
        }
        return;
    }
    if (t == 0.f) {  // greedy
        uint32_t first = 0xffffffffu, unused = 0;
        for (int i = tid; i < n; i += NT)
            if (z[i] == mx) {
                first = (uint32_t)(i0 + i);
                break;
            }
        R.block_minmax(first, unused);
        got = R.exchange(Gather{0ull, first, 0u});
#pragma unroll
        for (int r = 0; r < C; ++r) first = min(first, got[r].b);
        if (rank == 0 && tid == 0) {
            a.token[row] = (int)first;
            if (a.logprob) a.logprob[row] = 0.f;
        }
        return;
    }

    R.rs.mx = mx;
    R.rs.ch = S.ch;
    R.rs.cl = S.cl;
    // 16 steps per factor of 2 in weight, finer where the whole row spans less
    R.rs.step = fmaxf(16.f * S.ch, (float)(F_BINS - 1) / (mx - of_key(kmin)));

    float floor = -INFINITY;
    int m = 0;
    if (top_k > 0 && top_k < a.vocab)
        floor = of_key(R.top_k_key(top_k, a.vocab, own ? of_key(own) : -INFINITY, m));
    if (top_p < 1.f)
        floor = fmaxf(floor, of_key(m ? R.rank_mass(m, floor, 0ull, 0ull, top_p) : R.top_p_key(floor, top_p)));
    if (min_p > 0.f) {
        if (tid == 0) S.floor = __double2float_ru((double)mx + S.ln_min_p);
        __syncthreads();
        floor = fmaxf(floor, S.floor);
    }

    // the kept mass: each warp owns a contiguous range of the CTA's
    const int per_w = ((R.n4 + NW - 1) / NW), q0 = min(R.n4, w * per_w), q1 = min(R.n4, q0 + per_w);
    u64 mine = 0;
#pragma unroll 2
    for (int i = q0 + lane; i < q1; i += 32) {
        const float4 x = R.z4[i];
        if (x.x >= floor) mine += R.weight_of(x.x);
        if (x.y >= floor) mine += R.weight_of(x.y);
        if (x.z >= floor) mine += R.weight_of(x.z);
        if (x.w >= floor) mine += R.weight_of(x.w);
    }
    mine = warp_sum(mine);
    __syncthreads();
    if (lane == 0) S.wsum[w] = mine;
    __syncthreads();
    const u64 ws = lane < NW ? S.wsum[lane] : 0;
    u64 before = warp_sum(lane < w ? ws : 0ull);
    got = R.exchange(Gather{warp_sum(ws), 0u, 0u});
    u64 total = 0;
#pragma unroll
    for (int r = 0; r < C; ++r) {
        if (r < rank) before += got[r].a;
        total += got[r].a;
    }
    if (tid == 0) S.target = (u64)((double)u * (double)total);  // running > u * total <=> running > that
    __syncthreads();
    const u64 goal = S.target;
    if (before > goal || goal >= before + mine) return;
    // this warp's range holds the crossing
    for (int c0 = 4 * q0; c0 < 4 * q1; c0 += 32) {
        const int i = c0 + lane;
        const float x = i < 4 * q1 ? z[i] : -INFINITY;
        u64 inc = x >= floor ? R.weight_of(x) : 0ull;
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
constexpr int kWidePer = 26624;  // above it (one CTA per SM by its shared memory): 1024 threads, else 512

template <int NT, int C>
lf_status launch_row(const FilterArgs &a, cudaStream_t st) {
    if (!set_smem_once<sample_filtered_kernel<NT, C>>(kMaxPer * (int)sizeof(float))) return LF_ERR_CUDA;
    return launch_pdl_cluster(sample_filtered_kernel<NT, C>, C, dim3((unsigned)(a.rows * C)), NT,
                              (size_t)a.per * sizeof(float), st, a)
               ? LF_OK
               : LF_ERR_CUDA;
}

template <int C>
lf_status launch_cluster(const FilterArgs &a, cudaStream_t st) {
    return a.per > kWidePer ? launch_row<1024, C>(a, st) : launch_row<512, C>(a, st);
}

lf_status launch_filtered(FilterArgs a, cudaStream_t st) {
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
        case 1: return launch_cluster<1>(a, st);
        case 2: return launch_cluster<2>(a, st);
        case 4: return launch_cluster<4>(a, st);
        default: return launch_cluster<8>(a, st);
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
    a.dtype = dtype;
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
    return lf::launch_filtered(a, static_cast<cudaStream_t>(cuda_stream));
}
