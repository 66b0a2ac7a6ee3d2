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
// HBM once.  A bound is found in two stages.  First a cheap bound
// leaves few candidates (histograms: 2048 equal steps of the logit below the
// maximum, summed over the cluster through distributed shared memory):
//   top-k: of C CTAs, each takes the ceil(k / C)-th largest of its thread
//          groups' maxima; at least k logits reach the smallest of those, so
//          everything below drops out (for k above half the threads every
//          logit is counted in the histogram instead);
//   top-p: the masses of all logits (64 bits as two 32-bit shared atomics, the
//          second only on a carry) name the step that holds the border.
// The candidates' values (up to 1024) are then gathered in every CTA and told
// apart there, up to 256 by ranking them pairwise, more by their float's bits,
// 11 a level; a top-k set that was gathered serves top-p as well.  More
// candidates than the list holds (many equal logits) are told apart on their
// bits over all logits.
// No double precision on the way but for one sum per row (its rate here is 1/64
// of fp32's: a logarithm and a division cost 2 us): targets are exact integer
// products, log2(e) / T and ln(min_p) come as pairs of floats.
//
// Measured (us per call; rows of mixed filters, a fifth greedy; in brackets the
// bytes at the copy rate): 1 x 32000 fp32 5 - 11 (0.02), 16 x 32000 18 - 20 (0.3),
// 100 x 50257 39 (3), 256 x 131072 bf16 152 (10).  A single row is a chain of three
// to six exchanges between CTAs (about 1 us each) and passes over 4000 logits; many rows
// are bound by instructions: 76 per logit on average, two thirds of them the exact
// weights of the rows that need the mass of their whole vocabulary (no top-k).

#include <cooperative_groups.h>

#include <cfloat>
#include <climits>

#include "laneformer.h"
#include "lf_paged.h"
#include "lf_ptx.cuh"

namespace cg = cooperative_groups;

namespace lf {
namespace {

constexpr int F_BINS = 2048;
constexpr int F_LIST = 1024;  // candidates that every CTA of the row gathers
constexpr int F_RANK = 256;   // candidates that are ranked pairwise
constexpr int F_MAX_CLUSTER = 8;
constexpr int F_MAX_VOCAB = 262144;
constexpr int F_FRAC = 44;          // weights are integers in units of 2^-44
constexpr float F_MAX_Y = 45.f;     // below 2^-45 a weight rounds to nothing

using u64 = unsigned long long;

// 2^61 * 2^(-f / 256), f = 0 .. 255 (Taylor series of the exponential).
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
            v[f] = (u64)(sum * 2305843009213693952.0 + 0.5);
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

struct __align__(16) Gather {  // one CTA's contribution to a cluster-wide exchange
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
    u64 mass[F_RANK];        // weights of those ranked pairwise
    Gather slot[2][F_MAX_CLUSTER], said, heard[F_MAX_CLUSTER];
    uint64_t bar[2];
    u64 wsum[32];
    uint32_t wmin[32], wmax[32];
    u64 found_before;
    float floor;
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
// y = (max - z) log2(e) / T as a pair (error 2^-46 of it); y = j / 256 + r, |r| <= 1 / 512;
// 2^-y = 2^(-j / 256) (1 - q), q = 1 - e^(-t), t = r ln 2 = th + tl, |t| < 0.0014:
// q = th + (tl - th^2 (1/2 - th / 6)), the rest below 2^-42.  Sums of a large and a
// small integer are taken after their conversions (the small one by adding 1.5 * 2^23).
// mx is finite.
__device__ __forceinline__ u64 weight(float z, float mx, float ch, float cl, const u64 *pow2) {
    const float s = mx - z;
    const float yh = __fmul_rn(s, ch);
    constexpr float kRound = 12582912.f;  // 1.5 * 2^23: adding it leaves the integer part in the low mantissa bits
    constexpr int kRoundBits = 0x4B400000;
    const float bb = __fsub_rn(s, mx);  // mx - z = s + e exactly
    const float e = __fsub_rn(__fsub_rn(mx, __fsub_rn(s, bb)), __fadd_rn(z, bb));
    const float yl = __fmaf_rn(s, ch, -yh) + __fmaf_rn(s, cl, e * ch);
    const float tj = __fmaf_rn(yh, 256.f, kRound);
    const int j = __float_as_int(tj) - kRoundBits;
    const float r = __fmaf_rn(__fsub_rn(tj, kRound), -1.f / 256.f, yh);
    constexpr float kLn2 = 0.693147182464599609375f, kLn2Lo = -1.904654299957767878541e-9f;
    const float th = __fmul_rn(r, kLn2);
    const float tl = __fmaf_rn(r, kLn2, -th) + __fmaf_rn(r, kLn2Lo, yl * kLn2);
    const float c = __fmaf_rn(-th * th, __fmaf_rn(th, -1.f / 6.f, 0.5f), tl);
    constexpr float kScale = 549755813888.f;  // 2^39
    const int q = __float2int_rn(th * kScale) + (__float_as_int(__fmaf_rn(c, kScale, kRound)) - kRoundBits);
    const u64 t = pow2[j & 255];
    const u64 w61 = t - (u64)(((long long)(int)(t >> 31) * q) >> 8);
    const int sh = 61 - F_FRAC + (j >> 8);
    const u64 v = ((w61 >> ((sh - 1) & 63)) + 1) >> 1;
    return yh < F_MAX_Y ? v : 0ull;  // (a select: what was computed for a far or infinite z is dropped)
}

// The same as a call, for the places that are not loops over the row.
__device__ __noinline__ u64 weight_call(float z, float mx, float ch, float cl, const u64 *pow2) {
    return weight(z, mx, ch, cl, pow2);
}

// floor(f * s), or (up) its ceiling, exactly, for 0 <= f < 1.
__device__ __noinline__ u64 scaled(float f, u64 s, bool up) {
    const uint32_t bits = __float_as_uint(f) & 0x7fffffffu;  // (f may be -0)
    const int e = (int)(bits >> 23);
    const u64 m = e ? (bits & 0x7fffffu) | 0x800000u : bits;  // f = m 2^-k
    const int k = 150 - (e ? e : 1);                          // 24 ..
    const u64 lo = m * s, hi = __umul64hi(m, s);
    u64 v = 0;
    bool rest;
    if (k < 64) {
        v = (hi << (64 - k)) | (lo >> k);
        rest = (lo & ((1ull << k) - 1)) != 0;
    } else {
        const int d = k - 64;
        v = d < 64 ? hi >> d : 0;
        rest = lo != 0 || (d < 64 ? (hi & ((1ull << d) - 1)) != 0 : hi != 0);
    }
    return v + (up && rest ? 1 : 0);
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

// Phase wait whose acquire covers stores from other CTAs of the cluster.
__device__ __forceinline__ bool wait_cluster(uint64_t *bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity), "n"(kWaitHintNs)
        : "memory");
    return ok != 0;
}

__device__ __forceinline__ void no_draw(int32_t *token, float *logprob) {
    *token = -1;
    if (logprob) *logprob = __int_as_float(0x7fffffff);
}

template <int NT, int C>
struct Row {
    static constexpr int NW = NT / 32;
    static constexpr int RT = NT / F_RANK;  // threads to a candidate that is ranked pairwise
    FilterShared &S;
    const float4 *z4;  // this CTA's logits, -inf past n up to a multiple of 4
    int n4, rank, tid, lane, w;
    int turn = 0;
    int32_t *token;
    float *logprob;
    RowScale rs;

    __device__ Row(FilterShared &s, const float *z, int n, int r, int32_t *tok, float *lp)
        : S(s), z4(reinterpret_cast<const float4 *>(z)), n4((n + 3) / 4), rank(r), tid(threadIdx.x),
          lane(threadIdx.x & 31), w(threadIdx.x >> 5), token(tok), logprob(lp) {}

    // f(value) for every logit of this CTA
    template <class F>
    __device__ __forceinline__ void each(F f) const {
#pragma unroll 1
        for (int i = tid; i < n4; i += NT) {
            const float4 x = z4[i];
            f(x.x);
            f(x.y);
            f(x.z);
            f(x.w);
        }
    }

    // Every CTA of the cluster gets every CTA's Gather: one 16-byte store into
    // each CTA's shared memory, counted there on a barrier (about 1 us less than a
    // store and a cluster barrier).  g is the same in threads 0 .. C - 1; a
    // __syncthreads lies between two exchanges, so a CTA has read the buffer of
    // one before its message of the next lets anyone write the one after
    // (`turn` alternates two buffers).  The wait is bounded: a thread whose wait
    // runs out reports the row as one without a draw and ends.
    __device__ __forceinline__ const Gather *exchange(const Gather &g) {
        const int b = turn & 1, parity = (turn >> 1) & 1;
        Gather *mine = S.slot[b];
        ++turn;
        if constexpr (C == 1) {
            if (tid == 0) mine[0] = g;
            __syncthreads();
        } else {
            if (tid == 0) mbar_arrive_expect_tx(&S.bar[b], C * (uint32_t)sizeof(Gather));
            if (tid < C) {
                uint32_t dst, bar;
                asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(dst) : "r"(smem_u32(mine + rank)), "r"(tid));
                asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(bar) : "r"(smem_u32(&S.bar[b])), "r"(tid));
                asm volatile(
                    "st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(dst),
                    "r"((uint32_t)g.a), "r"((uint32_t)(g.a >> 32)), "r"(g.b), "r"(g.c), "r"(bar)
                    : "memory");
            }
            const uint64_t give_up = global_timer_ns() + 2000000000ull;
            while (!wait_cluster(&S.bar[b], parity))
                if (global_timer_ns() > give_up) {
                    no_draw(token, logprob);
                    asm volatile("exit;");
                }
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
    __device__ __forceinline__ u64 weight_cold(float x) const { return weight_call(x, rs.mx, rs.ch, rs.cl, S.pow2); }
    __device__ __forceinline__ int step(float x) const { return step_of(x, rs.mx, rs.step); }

    __device__ void clear_hist() {
        for (int i = tid; i < F_BINS; i += NT) S.lo[i] = S.hi[i] = 0;
        if (tid == 0) S.n_cand = 0;
        __syncthreads();
    }

    // Finds, in the summed histogram (bins in falling order of the logit), the
    // bin where `above` + the running sum reaches the target, and `before`,
    // above + the sum of the bins before it.  With frac >= 0 the target is first
    // set to frac of the total, rounded up.  G = C: the sum of the cluster's
    // histograms; G = 1: this CTA's alone.
    template <int G>
    __device__ int find_bin(u64 above, u64 &target, float frac, u64 &before) {
        constexpr int SL = F_BINS / G;            // bins of this CTA's slice
        constexpr int PT = (SL + NT - 1) / NT;    // bins per thread
        const int part = G == 1 ? 0 : rank;
        if constexpr (G > 1)
            sync();  // every CTA's histogram is complete
        else
            __syncthreads();
        u64 v[PT], sum = 0;
        const int b0 = tid * PT;
#pragma unroll
        for (int i = 0; i < PT; ++i) {
            v[i] = 0;
            if (b0 + i < SL) {
#pragma unroll
                for (int r = 0; r < G; ++r) {
                    const uint32_t *lo = S.lo, *hi = S.hi;
                    if constexpr (G > 1) {
                        lo = cg::this_cluster().map_shared_rank(S.lo, r);
                        hi = cg::this_cluster().map_shared_rank(S.hi, r);
                    }
                    v[i] += ((u64)hi[part * SL + b0 + i] << 32) + lo[part * SL + b0 + i];
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
        u64 ws = lane < NW ? S.wsum[lane] : 0, wi = ws;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const u64 y = __shfl_up_sync(0xffffffffu, wi, o);
            if (lane >= o) wi += y;
        }
        u64 total = __shfl_sync(0xffffffffu, wi, 31);
        u64 at = above + inc - sum + __shfl_sync(0xffffffffu, wi - ws, w);
        if constexpr (G > 1) {
            const Gather *got = exchange(Gather{total, 0u, 0u});
            total = 0;
#pragma unroll
            for (int r = 0; r < G; ++r) {
                if (r < rank) at += got[r].a;
                total += got[r].a;
            }
        }
        if (frac >= 0.f) target = max(1ull, scaled(frac, total, true));
#pragma unroll
        for (int i = 0; i < PT; ++i) {
            if (at < target && target <= at + v[i]) {
                S.found = 1;
                S.found_bin = (uint32_t)(part * SL + b0 + i);
                S.found_before = at;
            }
            at += v[i];
        }
        __syncthreads();
        int bin = F_BINS - 1;
        before = above;
        if constexpr (G > 1) {
            const Gather *got = exchange(Gather{S.found_before, S.found_bin, (uint32_t)S.found});
#pragma unroll
            for (int r = 0; r < G; ++r)
                if (got[r].c) {
                    bin = (int)got[r].b;
                    before = got[r].a;
                }
        } else if (S.found) {
            bin = (int)S.found_bin;
            before = S.found_before;
        }
        return bin;
    }

    // Collects the logits from `floor` on for which take(value) holds: up to F_LIST of them in
    // S.all of every CTA.  Returns how many there are in the cluster (above
    // F_LIST: not collected) and their smallest and largest keys.
    template <class Take>
    __device__ int collect(float floor, Take take, uint32_t &kmin, uint32_t &kmax) {
        kmin = 0xffffffffu, kmax = 0;
        auto one = [&](float x) {
            if (x >= floor && take(x)) {
                const uint32_t k = key_of(x);
                kmin = min(kmin, k);
                kmax = max(kmax, k);
                const int at = atomicAdd(&S.n_cand, 1);
                if (at < F_LIST) S.cand[at] = x;
            }
        };
        for (int i = tid; i < n4; i += NT) {
            const float4 x = z4[i];
            if (!(fmaxf(fmaxf(x.x, x.y), fmaxf(x.z, x.w)) >= floor)) continue;
            one(x.x);
            one(x.y);
            one(x.z);
            one(x.w);
        }
        block_minmax(kmin, kmax);
        // the lists and what each CTA says of its own are read from its shared memory
        if (tid == 0) S.said = Gather{(u64)S.n_cand, kmin, kmax};
        sync();
        const Gather *got = &S.said;
        if constexpr (C > 1) {
            if (tid < C) S.heard[tid] = *cg::this_cluster().map_shared_rank(&S.said, tid);
            __syncthreads();
            got = S.heard;
        }
        int total = 0, first[C];
#pragma unroll
        for (int r = 0; r < C; ++r) {
            kmin = min(kmin, got[r].b);
            kmax = max(kmax, got[r].c);
            first[r] = total;
            total += (int)got[r].a;
        }
        if (total <= F_LIST) {
            for (int i = tid; i < total; i += NT) {
                int r = 0, at = i;  // entry `at` of CTA r's list
#pragma unroll
                for (int x = 1; x < C; ++x)
                    if (i >= first[x]) r = x, at = i - first[x];
                const float *src = S.cand;
                if constexpr (C > 1) src = cg::this_cluster().map_shared_rank(S.cand, r);
                S.all[i] = src[at];
            }
            __syncthreads();
        }
        return total;
    }

    __device__ __forceinline__ u64 share(float x, bool mass) const { return mass ? weight_cold(x) : 1ull; }

    // The border among the keys of [kmin, kmax] over the row's logits (list:
    // over the m gathered ones, in this CTA alone), by mass or by count: 2048 equal
    // runs of keys a level, until one key is left.  (11 bits a level: at most 3.)
    __device__ uint32_t refine(bool mass, bool list, int m, uint32_t kmin, uint32_t kmax, u64 above, u64 target) {
        const float *src = list ? S.all : reinterpret_cast<const float *>(z4);
        const int n = list ? m : 4 * n4;
        while (kmin < kmax) {
            int shift = 0;
            while (((kmax - kmin) >> shift) >= (uint32_t)F_BINS) ++shift;
            clear_hist();
#pragma unroll 1
            for (int i = tid; i < n; i += NT) {
                const float x = src[i];
                const uint32_t key = key_of(x);
                if (key < kmin || key > kmax) continue;
                const u64 wt = share(x, mass);
                if (wt) hist_add(S, (int)((kmax - key) >> shift), wt);
            }
            u64 before = 0;
            const uint32_t bin = (uint32_t)(list ? find_bin<1>(above, target, -1.f, before)
                                                 : find_bin<C>(above, target, -1.f, before));
            above = before;
            kmax -= min(bin << shift, kmax - kmin);
            kmin = max(kmin, kmax - min(kmax, (1u << shift) - 1u));
        }
        return kmax;
    }

    // Among the m gathered values from `floor` on, all keys in [kmin, kmax]: the
    // key of the value at which above + the values at or above it, by their mass
    // or (MASS false: above 0, no floor) counted, reach the target; with frac >= 0
    // that is frac of them all.
    template <bool MASS>
    __device__ uint32_t border(int m, float floor, u64 above, u64 target, float frac, uint32_t kmin,
                                            uint32_t kmax) {
        if constexpr (!MASS) {
            if (m > F_RANK) return refine(false, true, m, kmin, kmax, above, target);
            const int i = tid / RT, k = (int)target;  // RT neighbouring threads share candidate i
            const float x = i < m ? S.all[i] : 0.f;
            int gt = 0, ge = 0;
            for (int j = tid % RT; j < m; j += RT) {
                const float y = S.all[j];
                gt += y > x ? 1 : 0;
                ge += y >= x ? 1 : 0;
            }
#pragma unroll
            for (int o = 1; o < RT; o <<= 1) {
                gt += __shfl_xor_sync(0xffffffffu, gt, o);
                ge += __shfl_xor_sync(0xffffffffu, ge, o);
            }
            if (i < m && gt < k && k <= ge) S.key = key_of(x);
            __syncthreads();
            return S.key;
        }
        u64 own = 0;
#pragma unroll 1
        for (int i = tid; i < m; i += NT) {
            const u64 v = S.all[i] >= floor ? weight_cold(S.all[i]) : 0ull;
            if (i < F_RANK) S.mass[i] = v;
            own += v;
        }
        if (frac >= 0.f) {
            own = warp_sum(own);
            if (lane == 0) S.wsum[w] = own;
            __syncthreads();
            target = max(1ull, scaled(frac, warp_sum(lane < NW ? S.wsum[lane] : 0ull), true));
        }
        if (m > F_RANK) return refine(true, true, m, max(kmin, key_of(floor)), kmax, above, target);
        __syncthreads();
        const int i = tid / RT;
        const float x = i < m ? S.all[i] : 0.f;
        u64 gt = 0, eq = 0;
#pragma unroll 1
        for (int j = tid % RT; j < m; j += RT) {
            const float y = S.all[j];
            const u64 wj = S.mass[j];
            gt += y > x ? wj : 0ull;
            eq += y == x ? wj : 0ull;
        }
#pragma unroll
        for (int o = 1; o < RT; o <<= 1) {
            gt += __shfl_xor_sync(0xffffffffu, gt, o);
            eq += __shfl_xor_sync(0xffffffffu, eq, o);
        }
        gt += above;
        if (i < m && gt < target && target <= gt + eq) S.key = key_of(x);
        __syncthreads();
        return S.key;
    }

    // A key that at least ceil(k / C) of this CTA's logits reach, so that k of
    // the row's reach the smallest of the CTAs' keys: the ceil(k / C)-th largest of
    // the maxima of groups of threads (32, 8 or 2 to 4 of them).  0 where 256 groups are too few for it (then the row's
    // histogram finds the bound).  `own` is the thread's largest key.
    __device__ uint32_t group_bound(uint32_t own, int k) {
        const int need = (k + C - 1) / C;
        // (at 4/5 of the groups, twice as many logits as wanted reach the bound)
        const int most = 5 * need / 4;
        const int size = most <= NT / 32 ? 32 : most <= NT / 8 ? 8 : most <= F_RANK ? RT : 0;
        if (size == 0) return 0;
        for (int o = 1; o < size; o <<= 1) own = max(own, __shfl_xor_sync(0xffffffffu, own, o));
        const int groups = NT / size;  // at most F_RANK
        if (tid % size == 0) S.lo[tid / size] = own;
        __syncthreads();
        const int i = tid / RT;  // RT neighbouring threads rank group i
        const uint32_t x = i < groups ? S.lo[i] : 0u;
        int gt = 0, ge = 0;
        for (int j = tid % RT; j < groups; j += RT) {
            const uint32_t y = S.lo[j];
            gt += y > x ? 1 : 0;
            ge += y >= x ? 1 : 0;
        }
#pragma unroll
        for (int o = 1; o < RT; o <<= 1) {
            gt += __shfl_xor_sync(0xffffffffu, gt, o);
            ge += __shfl_xor_sync(0xffffffffu, ge, o);
        }
        if (i < groups && gt < need && need <= ge) S.key = x;
        __syncthreads();
        return S.key;
    }

    // The lower bounds that top-k (off: k = 0) and top-p (off: 1) put on the
    // logit.  bound: a key that at least k logits, or all above -inf, reach, or 0.
    __device__ float bounds(int k, float top_p, uint32_t bound) {
        float floor = -INFINITY;
        uint32_t kmin, kmax;
        if (k == 1) {
            floor = rs.mx;
            top_p = 1.f;  // the maxima are the nucleus too
        } else if (k > 0) {
            clear_hist();
            // (the padding behind the vocabulary is -inf, the same as a masked logit:
            // it lies below every logit or equals the smallest, so it changes no bound above -inf)
            u64 target = (u64)k, before = 0;
            float least = -INFINITY;
            int last = F_BINS;
            if (bound) {
                least = of_key(bound);
            } else {
                each([&](float x) { hist_add(S, step(x), 1ull); });
                last = find_bin<C>(0ull, target, -1.f, before);
            }
            const int m = collect(least, [&](float x) { return last == F_BINS || step(x) <= last; }, kmin, kmax);
            if (m <= k)
                floor = of_key(kmin);  // (fewer: there are no more above -inf)
            else
                floor = of_key(m <= F_LIST ? border<false>(m, -INFINITY, 0ull, target, -1.f, kmin, kmax)
                                           : refine(false, false, 0, kmin, kmax, 0ull, target));
            if (m <= F_LIST) {  // the list holds the whole top-k set
                if (top_p < 1.f) floor = fmaxf(floor, of_key(border<true>(m, floor, 0ull, 0ull, top_p, kmin, kmax)));
                return floor;
            }
        }
        if (top_p < 1.f) {
            clear_hist();
            each([&](float x) {
                if (!(x >= floor)) return;
                const u64 wt = weight_of(x);
                if (wt) hist_add(S, step(x), wt);
            });
            u64 target = 0, before = 0;
            const int at = find_bin<C>(0ull, target, top_p, before);
            const int m = collect(floor, [&](float x) { return step(x) == at; }, kmin, kmax);
            uint32_t key = kmax;
            if (kmin != kmax)
                key = m <= F_LIST ? border<true>(m, floor, before, target, -1.f, kmin, kmax)
                                  : refine(true, false, 0, kmin, kmax, before, target);
            floor = fmaxf(floor, of_key(key));
        }
        return floor;
    }

    // The smallest float at or above max + T ln(p), by one thread: with p = m 2^e,
    // ln m = g + ln(m e^-g) for g near it, and m e^-g - 1 from the exact weight.
    __device__ float min_p_floor(float p, float t) const {
        int e;
        const float m = frexpf(p, &e), g = logf(m);
        const u64 we = weight_call(g, 0.f, 1.44269502162933349609375f, 1.92596299112661746887e-8f, S.pow2);
        const float rest = (float)((long long)((u64)(m * 16777216.f) << (F_FRAC - 24)) - (long long)we) / (float)we;
        return __double2float_ru((double)rs.mx + (double)t * ((double)e * 0.69314718055994530942 + (double)g + (double)rest));
    }
};

// The larger, NaN if either is.
__device__ __forceinline__ float max_or_nan(float a, float b) {
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}

// Reads n logits as fp32 into shared memory (16-byte loads where the row is
// aligned for them); returns the thread's largest (NaN if there is one, -inf if
// it read none), and through least its smallest above -inf.
template <typename T, int NT>
__device__ __forceinline__ float load_row(const T *src, int n, float *z, float &least) {
    constexpr int V = 16 / sizeof(T);
    float most = -INFINITY;
    auto take = [&](float x) {
        most = max_or_nan(most, x);
        if (x > -INFINITY) least = fminf(least, x);
    };
    int done = 0;
    if ((reinterpret_cast<uintptr_t>(src) & 15u) == 0) {
        const int nv = n / V;
        done = nv * V;
#pragma unroll 4
        for (int i = threadIdx.x; i < nv; i += NT) {
            const uint4 raw = reinterpret_cast<const uint4 *>(src)[i];
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
    return most;
}

template <int NT, int C>
__global__ void __launch_bounds__(NT, 1024 / NT) sample_filtered_kernel(const FilterArgs a) {
    extern __shared__ __align__(16) float z[];  // this CTA's logits
    __shared__ FilterShared S;
    constexpr int NW = NT / 32;
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    const int row = blockIdx.x / C, rank = blockIdx.x % C;
    const int i0 = rank * a.per, n = max(0, min(a.per, a.vocab - i0));
    float *logprob = a.logprob ? a.logprob + row : nullptr;
    Row<NT, C> R(S, z, n, rank, a.token + row, logprob);
    for (int i = tid; i < 256; i += NT) S.pow2[i] = kPow2.v[i];
    if constexpr (C > 1) {
        if (tid == 0) {
            mbar_init(&S.bar[0], 1);
            mbar_init(&S.bar[1], 1);
            fence_barrier_init();
        }
        R.sync();  // no message comes before the barriers are there
    }
    pdl_wait();
    pdl_trigger();

    const float t = a.temperature ? a.temperature[row] : 1.f, top_p = a.top_p ? a.top_p[row] : 1.f;
    const float min_p = a.min_p ? a.min_p[row] : 0.f, u = a.u[row];
    const int top_k = a.top_k ? a.top_k[row] : 0;
    const bool fine = (t == 0.f || (t >= 1e-30f && t <= 1e30f)) && top_p > 0.f && top_p <= 1.f && min_p >= 0.f &&
                      min_p <= 1.f && u >= 0.f && u < 1.f;
    if (!fine) {  // every CTA of the row sees the same
        if (rank == 0 && tid == 0) no_draw(a.token + row, logprob);
        return;
    }
    const long long at = (long long)row * a.ld + i0;
    float least = INFINITY;
    const float most = a.dtype == LF_F32   ? load_row<float, NT>(static_cast<const float *>(a.logits) + at, n, z, least)
                       : a.dtype == LF_F16 ? load_row<__half, NT>(static_cast<const __half *>(a.logits) + at, n, z, least)
                                           : load_row<__nv_bfloat16, NT>(static_cast<const __nv_bfloat16 *>(a.logits) + at, n, z, least);
    bool nan = __syncthreads_or(most != most);
    const uint32_t own = key_of(most);
    uint32_t kmax = own, kmin = key_of(least);  // (least +inf: no logit above -inf, or only infinite ones)
    const int k = top_k > 0 && top_k < a.vocab ? top_k : 0;
    R.block_minmax(kmin, kmax);
    uint32_t bound = k > 1 && t > 0.f ? R.group_bound(own, k) : 0u;
    const Gather *got = R.exchange(Gather{(u64)bound << 32 | (nan ? 1u : 0u), kmin, kmax});
#pragma unroll
    for (int r = 0; r < C; ++r) {
        nan |= (got[r].a & 1) != 0;
        bound = min(bound, (uint32_t)(got[r].a >> 32));
        kmin = min(kmin, got[r].b);
        kmax = max(kmax, got[r].c);
    }
    if (bound && bound <= key_of(-INFINITY)) bound = kmin;  // a CTA with few logits above -inf: then all of those
    float mx = of_key(kmax);
    if (nan || !(mx > -INFINITY)) {
        if (rank == 0 && tid == 0) no_draw(a.token + row, logprob);
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
            if (logprob) *logprob = 0.f;
        }
        return;
    }

    const bool infinite = mx == INFINITY;
    if (infinite) {  // the infinite logits hold all the mass, equally, under any filter: 0 there and -inf elsewhere
        for (int i = tid; i < 4 * R.n4; i += NT) z[i] = z[i] == INFINITY ? 0.f : -INFINITY;
        mx = 0.f;
        kmin = key_of(0.f);
        __syncthreads();
    }

    // log2(e) / T as a pair: the quotient and what its product with T leaves
    constexpr float kLog2eHi = 1.44269502162933349609375f, kLog2eLo = 1.92596299112661746887e-8f;
    R.rs.mx = mx;
    R.rs.ch = __fdiv_rn(kLog2eHi, t);
    R.rs.cl = __fdiv_rn(__fmaf_rn(-R.rs.ch, t, kLog2eHi) + kLog2eLo, t);
    // 32 steps per factor of 2 in weight, finer where the whole row spans less
    R.rs.step = fmaxf(32.f * R.rs.ch, (float)(F_BINS - 1) / (mx - of_key(kmin)));

    float floor = infinite ? 0.f : R.bounds(k, top_p, bound);
    if (min_p > 0.f && !infinite) {
        if (tid == 0) S.floor = R.min_p_floor(min_p, t);
        __syncthreads();
        floor = fmaxf(floor, fminf(S.floor, mx));  // (min_p 1: the maxima stay whatever the last bit of the sum)
    }

    // the kept mass: each warp owns a contiguous range of the CTA's
    const int per_w = ((R.n4 + NW - 1) / NW), q0 = min(R.n4, w * per_w), q1 = min(R.n4, q0 + per_w);
    u64 mine = 0;
#pragma unroll 1
    for (int i = q0 + lane; i < q1; i += 32) {
        const float4 x = R.z4[i];
        if (!(fmaxf(fmaxf(x.x, x.y), fmaxf(x.z, x.w)) >= floor)) continue;
        const u64 wx = R.weight_of(x.x), wy = R.weight_of(x.y), wz = R.weight_of(x.z), ww = R.weight_of(x.w);
        mine += (x.x >= floor ? wx : 0ull) + (x.y >= floor ? wy : 0ull) + (x.z >= floor ? wz : 0ull) +
                (x.w >= floor ? ww : 0ull);
    }
    mine = warp_sum(mine);
    __syncthreads();
    if (lane == 0) S.wsum[w] = mine;
    __syncthreads();
    const u64 ws = lane < NW ? S.wsum[lane] : 0;
    u64 wi = ws;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const u64 y = __shfl_up_sync(0xffffffffu, wi, o);
        if (lane >= o) wi += y;
    }
    u64 before = __shfl_sync(0xffffffffu, wi - ws, w);
    got = R.exchange(Gather{__shfl_sync(0xffffffffu, wi, 31), 0u, 0u});
    u64 total = 0;
#pragma unroll
    for (int r = 0; r < C; ++r) {
        if (r < rank) before += got[r].a;
        total += got[r].a;
    }
    const u64 goal = scaled(u, total, false);  // running > u * total <=> running > that
    if (before > goal || goal >= before + mine) return;
    // this warp's range holds the crossing
    for (int c0 = 4 * q0; c0 < 4 * q1; c0 += 32) {
        const int i = c0 + lane;
        const float x = i < 4 * q1 ? z[i] : -INFINITY;
        u64 inc = x >= floor ? R.weight_cold(x) : 0ull;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const u64 y = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += y;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, before + inc > goal);
        if (hit) {
            if (lane == __ffs(hit) - 1) {
                a.token[row] = i0 + i;
                // from the logit, not from its rounded weight; the mass is 1 + something (the maximum is kept)
                if (logprob) {
                    const float more = (float)(total - (1ull << F_FRAC)) * 5.684341886080801e-14f;  // 2^-44
                    *logprob = (x == mx ? 0.f : (x - mx) / t) - log1pf(more);
                }
            }
            return;
        }
        before += __shfl_sync(0xffffffffu, inc, 31);
    }
}

constexpr int kMaxPer = 49152;   // logits of one CTA: 192 KB
constexpr int kPairPer = 20480;  // up to here two CTAs fit an SM's shared memory

template <int NT, int C>
lf_status launch_row(const FilterArgs &a, cudaStream_t st) {
    if (!set_smem_once<sample_filtered_kernel<NT, C>>(kMaxPer * (int)sizeof(float))) return LF_ERR_CUDA;
    return launch_pdl_cluster(sample_filtered_kernel<NT, C>, C, dim3((unsigned)(a.rows * C)), NT,
                              (size_t)a.per * sizeof(float), st, a)
               ? LF_OK
               : LF_ERR_CUDA;
}

template <int C>
lf_status launch_cluster(const FilterArgs &a, int n_sm, cudaStream_t st) {
    // 1024 threads where a CTA has its SM to itself, or nearly all do: 512, two CTAs
    // to an SM, win with more of them or few logits (us, 512 | 1024 threads; CTAs x logits
    // of one: 160 x 10000 30.6 | 24.6, 200 x 10000 30.2 | 26.5, 200 x 4000 21.6 | 20.8,
    // 300 x 10000 31.7 | 35.4, 200 x 37 10.6 | 12.9)
    const int wide = a.per > 2048 ? n_sm + n_sm / 3 : n_sm;
    return a.per > kPairPer || a.rows <= wide / C ? launch_row<1024, C>(a, st) : launch_row<512, C>(a, st);
}

lf_status launch_filtered(FilterArgs a, cudaStream_t st) {
    int dev = 0, n_sm = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&n_sm, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
        (void)cudaGetLastError();
        return LF_ERR_CUDA;
    }
    // CTAs per row: what the shared memory asks for, and more while a CTA has at least
    // 4096 logits and the grid fits the SMs, or overflows them by a third at 12000 logits
    // and more.  Measured (us, c = 1 | 2 | 4 | 8): 1 x 32000 17.1 | 12.9 | 10.1 | 9.4,
    // 16 x 32000 38 | 26 | 20 | 19, 40 x 32000 37 | 27 | 23 | 38, 70 x 32000 37 | 28 | 33 | 59,
    // 100 x 32000 39 | 33 | 43 | 79, 100 x 10000 20 | 30 | 42 | 86, 150 x 10000 21 | 40 | 59 |
    // 132, 256 x 32000 57 | 65 | 94 | 185, 1 x 4000 7.3 | 7.6 | 8.0 | 8.9.
    int c = 1;
    auto more = [&] {
        const int per = a.vocab / c, room = per > 12000 ? n_sm + n_sm / 3 : n_sm;
        return (a.vocab + c - 1) / c > kMaxPer || (per > 4096 && a.rows <= room / (2 * c));
    };
    while (c < F_MAX_CLUSTER && more()) c *= 2;
    a.per = ((a.vocab + c - 1) / c + 7) / 8 * 8;
    switch (c) {
        case 1: return launch_cluster<1>(a, n_sm, st);
        case 2: return launch_cluster<2>(a, n_sm, st);
        case 4: return launch_cluster<4>(a, n_sm, st);
        default: return launch_cluster<8>(a, n_sm, st);
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
