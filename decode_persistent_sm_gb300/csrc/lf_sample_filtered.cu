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
// The answer is a whole number that sums decide, so the sums are integers: a
// weight is 2^58 w rounded up, from an exponential whose argument is carried as a
// pair of floats (error about 2^-40 of the weight: the fp32 exponential's 2^-22
// would put one row in ten of a flat 131072-token row on the wrong side of some
// border).  The largest weight is 1 and a row has at most 2^18 logits, so all
// that is rounded up is below 2^-40 of the mass (units of 2^-44 would lose 2^-27 in
// a long tail of equal weights).  Rounded up and not to nearest: a weight that 64
// bits can hold counts, if only by a unit, and u = 0 draws the first kept
// index.  A thread's sum fits 64 bits (at most 48 logits), what is summed further
// has 128.  Integer sums come out the same in any order, atomics included.
//
// A row belongs to a cluster of 1, 2, 4 or 8 CTAs, each with a contiguous
// range of the vocabulary in shared memory as fp32: the logits are read from
// HBM once.  A bound is found in two stages.  First a cheap bound
// leaves few candidates (histograms: 2048 equal steps of the logit below the
// maximum, summed over the cluster through distributed shared memory):
//   top-k: of C CTAs, each takes the ceil(k / C)-th largest of its thread
//          groups' maxima; at least k logits reach the smallest of those, so
//          everything below drops out (for k above 204 C every logit is counted
//          in the histogram instead);
//   top-p: the masses of all logits (64 bits as two 32-bit shared atomics, the
//          second where the high word changes) name the step that holds the border.
//          A step's unit is 2^-44 of the largest weight that can lie in it, down to
//          2^-58: a sum of 2^18 weights of one step fits 64 bits at full precision.
// The candidates' values (up to 1024) are then gathered in every CTA and told
// apart there, up to 256 by ranking them pairwise, more by their float's bits,
// 11 a level; a top-k set that was gathered serves top-p as well.  More
// candidates than the list holds (many equal logits) are told apart on their
// bits over all logits.
// No double precision on the way but for one sum per row (its rate here is 1/64
// of fp32's: a logarithm and a division cost 2 us): targets are exact integer
// products, log2(e) / T and ln(min_p) come as pairs of floats.
//
// Measured (us per call; in brackets the bytes at the copy rate): 1 x 32000 fp32 6.5
// without a filter, 14 under top-p, 10 under top-k 50, 15 under both, 3 greedy (0.02);
// rows of mixed filters, a fifth greedy: 16 x 32000 20 (0.3), 100 x 50257 42 - 47 (3), 256
// x 131072 bf16 151 - 156 (10).  A single row is a chain of two to six exchanges
// between CTAs (about 1 us each) and passes over 4000 logits; many rows are bound by
// instructions: 73 per logit on average, two thirds of them the exact weights of the
// rows that need the mass of their whole vocabulary (no top-k).

#include <cooperative_groups.h>

#include <atomic>
#include <cfloat>
#include <climits>

#include "laneformer.h"
#include "lf_paged.h"
#include "lf_ptx.cuh"
#include "lf_sample.h"

namespace cg = cooperative_groups;

namespace lf {
namespace {

constexpr int F_BINS = 2048;
constexpr int F_LIST = 1024;  // candidates that every CTA of the row gathers
constexpr int F_RANK = 256;   // candidates that are ranked pairwise
constexpr int F_MAX_CLUSTER = 8;
constexpr int F_MAX_VOCAB = 262144;
constexpr int F_FRAC = 58;          // weights are integers in units of 2^-58: 48 of them fit 64 bits
constexpr int F_STEP_FRAC = 44;     // in a step of the histogram: 2^-44 of its largest weight, at least 2^-58
constexpr int F_LIST_FRAC = 53;     // among the candidates of a list: F_LIST of them fit 64 bits
constexpr float F_ZERO_Y = 1075.f;  // a weight below 2^-1075 is zero, as in 64-bit arithmetic
constexpr long long F_WAIT_CYCLES = 4000000000ll;  // 2 s

using u64 = unsigned long long;
using u128 = unsigned __int128;

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
    uint32_t *err;           // nullable: 2 when a wait ran out
    long long wait_cycles;   // limit of a wait between CTAs
#ifdef LF_DEBUG
    int lose_rank, lose_wait;  // the CTA of this rank (-1: each) gives up in its lose_wait-th wait (0: none)
#endif
};

struct __align__(16) Gather {  // one CTA's contribution to a cluster-wide exchange
    u64 a;
    uint32_t b, c;
};

struct RowScale {
    float mx, ch, cl, step;  // the maximum, log2(e) / T as a pair, histogram steps per unit of logit
    int oct;                 // log2 of the steps to a factor of 2 in weight
};

struct FilterShared {
    u64 pow2[256];
    uint32_t lo[F_BINS], hi[F_BINS];
    float cand[F_LIST];      // this CTA's candidates
    float all[F_LIST];       // the cluster's
    u64 mass[F_RANK];        // weights of those ranked pairwise
    Gather slot[2][F_MAX_CLUSTER], said, heard[F_MAX_CLUSTER];
    uint64_t bar[2], ready;
    u128 wsum[32], found_before;
    // what warp 0 makes of an exchange
    u128 base, target, before, total, left;
    uint32_t kmin, kmax, bound, first, bin;
    int nan, winner, lost;
    uint32_t wmin[32], wmax[32];
    float floor;
    uint32_t found_bin, key;  // found_bin: the step and 1, 0 for none
    int n_cand;
};

// Order-preserving bits of a float (no NaN; -0 was made +0).
__device__ __forceinline__ uint32_t key_of(float z) {
    const uint32_t b = __float_as_uint(z);
    return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }

// ceil(2^frac exp((z - max) / T)), (ch, cl) = log2(e) / T as a pair of floats.
// y = (max - z) log2(e) / T as a pair (error 2^-46 of it); y = j / 256 + r, |r| <= 1 / 512;
// 2^-y = 2^(-j / 256) (1 - q), q = 1 - e^(-t), t = r ln 2 = th + tl, |t| < 0.0014:
// q = th + (tl - th^2 (1/2 - th / 6)), the rest below 2^-42.  Sums of a large and a
// small integer are taken after their conversions (the small one by adding 1.5 * 2^23).
// From `far` <= frac on (in y) the weight is one unit, from F_ZERO_Y on 0 (a masked
// logit's).  mx is finite.
__device__ __forceinline__ u64 weight(float z, float mx, float ch, float cl, const u64 *pow2, int frac, float far) {
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
    const u64 v = ((w61 - 1) >> ((61 - frac + (j >> 8)) & 63)) + 1;
    return yh < far ? v : (yh < F_ZERO_Y ? 1ull : 0ull);  // (selects: what was computed for a far or infinite z is dropped)
}

// The same as a call, for the places that are not loops over the row.
__device__ __noinline__ u64 weight_call(float z, float mx, float ch, float cl, const u64 *pow2, int frac) {
    return weight(z, mx, ch, cl, pow2, frac, (float)frac);
}

// floor(f * s), or (up) its ceiling, exactly, for 0 <= f < 1 and s < 2^104.
__device__ __noinline__ u128 scaled(float f, u128 s, bool up) {
    const uint32_t bits = __float_as_uint(f) & 0x7fffffffu;  // (f may be -0)
    const int e = (int)(bits >> 23);
    const u128 p = s * (e ? (bits & 0x7fffffu) | 0x800000u : bits);  // f = m 2^-k
    const int k = 150 - (e ? e : 1);                                 // 24 ..
    const u128 v = k < 128 ? p >> k : 0;
    const bool rest = k < 128 ? (v << k) != p : p != 0;
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

// The warp's sum, in pieces of 22 bits.
__device__ __forceinline__ u128 warp_sum(u64 v) {
    const uint32_t a = __reduce_add_sync(0xffffffffu, (uint32_t)v & 0x3fffffu),
                   b = __reduce_add_sync(0xffffffffu, (uint32_t)(v >> 22) & 0x3fffffu),
                   c = __reduce_add_sync(0xffffffffu, (uint32_t)(v >> 44));
    return ((u128)c << 44) + ((u64)b << 22) + a;
}

__device__ __forceinline__ u64 shfl(u64 v, int lane) { return __shfl_sync(0xffffffffu, v, lane); }
__device__ __forceinline__ u128 shfl(u128 v, int lane) {
    return (u128)shfl((u64)(v >> 64), lane) << 64 | shfl((u64)v, lane);
}
// Inclusive sum over the lanes.
__device__ __forceinline__ u64 warp_scan(u64 v, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const u64 y = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += y;
    }
    return v;
}
__device__ __forceinline__ u128 warp_scan(u128 v, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const u64 lo = __shfl_up_sync(0xffffffffu, (u64)v, o), hi = __shfl_up_sync(0xffffffffu, (u64)(v >> 64), o);
        if (lane >= o) v += (u128)hi << 64 | lo;
    }
    return v;
}
// A sum of a Gather's a (low 64 bits) and b (the rest).
__device__ __forceinline__ u128 wide(const Gather &g) { return (u128)g.b << 64 | g.a; }

__device__ __forceinline__ float of_key(uint32_t k) {
    return __uint_as_float((k & 0x80000000u) ? k & 0x7fffffffu : ~k);
}

// Phase wait, suspended for kWaitHintNs at most, whose acquire covers stores from
// other CTAs of the cluster.
__device__ __forceinline__ bool try_cluster(uint64_t *bar, uint32_t parity) {
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

// A warp's wait for a phase, of about `cycles` at most; the same answer in every
// lane.  (The lanes stay together: after a loop of one lane the warp goes on in two
// parts, and every shuffle costs a hundred cycles: 3 us for the sums of an exchange.)
__device__ __forceinline__ bool wait_cluster(uint64_t *bar, uint32_t parity, long long cycles) {
    const long long since = clock64();
    while (!__all_sync(0xffffffffu, try_cluster(bar, parity)))
        if (__any_sync(0xffffffffu, clock64() - since > cycles)) return false;
    return true;
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
    int turn = 0, published = 0;
    bool lost = false;  // a wait of this CTA ran out: the same in all its threads
    bool met = false;   // past meet()
    const FilterArgs &a;
    RowScale rs;
#ifdef LF_DEBUG
    int waits = 0;
#endif

    __device__ Row(FilterShared &s, const float *z, int n, int r, const FilterArgs &args)
        : S(s), z4(reinterpret_cast<const float4 *>(z)), n4((n + 3) / 4), rank(r), tid(threadIdx.x),
          lane(threadIdx.x & 31), w(threadIdx.x >> 5), a(args) {}

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

    // Warp 0's bounded wait for a phase; its answer holds for the CTA.
    __device__ __forceinline__ bool await(uint64_t *bar, uint32_t parity) {
#ifdef LF_DEBUG
        if (++waits == a.lose_wait && (a.lose_rank < 0 || a.lose_rank == rank)) return false;
#endif
        __syncwarp();
        return wait_cluster(bar, parity, a.wait_cycles);
    }

    // A Gather from each of G CTAs (all of the cluster, or 1: this one alone) to all
    // of them: one 16-byte store into each CTA's shared memory, counted there on a
    // barrier (about 1 us less than a store and a cluster barrier).  g counts in
    // warp 0, which passes what arrived to digest(lane r: the Gather of CTA r) and
    // leaves what that makes of it in shared memory for the others.  A CTA has
    // digested one exchange before its message of the next lets anyone write the
    // one after (`turn` alternates two buffers).
    // The wait is bounded.  A CTA whose wait ran out takes part in nothing more but
    // leave(), so the row's other CTAs run out of theirs; nobody goes on with numbers
    // that did not arrive.
    template <int G, class D>
    __device__ __forceinline__ void exchange(const Gather &g, D digest) {
        if (lost) return;
        if constexpr (G == 1) {
            if (w == 0) digest(g);
            __syncthreads();
        } else {
            const int b = turn & 1, parity = (turn >> 1) & 1;
            ++turn;
            if (w == 0) {
                if (tid == 0) mbar_arrive_expect_tx(&S.bar[b], G * (uint32_t)sizeof(Gather));
                if (tid < G) {
                    uint32_t dst, bar;
                    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                                 : "=r"(dst)
                                 : "r"(smem_u32(&S.slot[b][rank])), "r"(tid));
                    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(bar) : "r"(smem_u32(&S.bar[b])), "r"(tid));
                    asm volatile(
                        "st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(dst),
                        "r"((uint32_t)g.a), "r"((uint32_t)(g.a >> 32)), "r"(g.b), "r"(g.c), "r"(bar)
                        : "memory");
                }
                if (await(&S.bar[b], parity))
                    digest(S.slot[b][lane % G]);
                else if (lane == 0)
                    S.lost = 1;
            }
            __syncthreads();
            lost = S.lost != 0;
        }
    }

    // The row's last exchange.  Who has its messages needs nothing more of the
    // others, nor they of it.  A CTA whose wait ran out looks again when all others
    // have ended or given up: either every CTA had sent its message, then it goes
    // on; or one had given up before, then no CTA of the row has them all and
    // none writes a token.
    template <class D>
    __device__ __forceinline__ void last_exchange(const Gather &g, D digest) {
        exchange<C>(g, digest);
        if constexpr (C > 1) {
            if (lost) {
                meet();
                if (w == 0 && landed(turn - 1)) {
                    digest(S.slot[(turn - 1) & 1][lane % C]);
                    if (lane == 0) S.lost = 0;
                }
                __syncthreads();
                lost = S.lost != 0;
            }
        }
    }

    // Every CTA's shared memory as it was at this call may be read by the others
    // behind it.  (Not a cluster barrier: a CTA that gave up has to leave those
    // that wait here waiting, not let them pass.)
    __device__ __forceinline__ void publish() {
        __syncthreads();
        if constexpr (C > 1) {
            if (lost) return;
            const int parity = published++ & 1;
            if (w == 0) {
                if (tid < C) {
                    uint32_t bar;
                    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(bar) : "r"(smem_u32(&S.ready)), "r"(tid));
                    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
                }
                if (!await(&S.ready, parity) && lane == 0) S.lost = 1;
            }
            __syncthreads();
            lost = S.lost != 0;
        }
    }

    // The messages of exchange i, waited for about a millisecond (warp 0).
    __device__ bool landed(int i) { return wait_cluster(&S.bar[i & 1], (i >> 1) & 1, 2000000); }
    // Where CTAs that gave up wait until the row's others are here or have ended (an
    // exited thread counts as arrived).  All waits being bounded, they do.
    __device__ __forceinline__ void meet() {
        __syncwarp();
        cg::this_cluster().sync();
        met = true;
    }

    // The end of a row that exchanged anything: no CTA ends while another may still
    // read or write its shared memory.  A CTA that received all it waited for may
    // end: the others sent it nothing else, and what they read of it they
    // had read before they sent the last message.  One that gave up waits for the
    // others and (a millisecond) for what they sent to it, its last exchange's
    // messages and those of CTAs one exchange further, and reports the row.
    __device__ __forceinline__ void leave(int row) {
        if constexpr (C > 1) {
            if (!lost) return;
            if (!met) meet();
            if (w == 0) {
                if (turn > 0) (void)landed(turn - 1);
                if (lane == 0) mbar_arrive_expect_tx(&S.bar[turn & 1], C * (uint32_t)sizeof(Gather));
                (void)landed(turn);
                if (lane == 0) {
                    no_draw(a.token + row, a.logprob ? a.logprob + row : nullptr);
                    if (a.err) atomicCAS(a.err, 0u, 2u);
                }
            }
        }
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

    __device__ __forceinline__ u64 weight_of(float x) const {
        return weight(x, rs.mx, rs.ch, rs.cl, S.pow2, F_FRAC, (float)F_FRAC);
    }
    // in units of x's step (where the unit is above 2^-58, y stays far below 58)
    __device__ __forceinline__ u64 weight_in_step(float x, int step) const {
        return weight(x, rs.mx, rs.ch, rs.cl, S.pow2, step_frac(step), (float)F_FRAC);
    }
    __device__ __forceinline__ u64 weight_cold(float x, int frac) const {
        return weight_call(x, rs.mx, rs.ch, rs.cl, S.pow2, frac);
    }
    __device__ __forceinline__ int step(float x) const { return step_of(x, rs.mx, rs.step); }
    // weights of step s are at most 2^-(s >> oct)
    __device__ __forceinline__ int step_frac(int s) const { return min(F_STEP_FRAC + (s >> rs.oct), F_FRAC); }

    __device__ void clear_hist() {
        for (int i = tid; i < F_BINS; i += NT) S.lo[i] = S.hi[i] = 0;
        if (tid == 0) S.n_cand = 0;
        __syncthreads();
    }

    // Finds, in the summed histogram (bins in falling order of the logit), the
    // bin where `above` + the running sum reaches the target, and `before`,
    // above + the sum of the bins before it.  With frac >= 0 the target is first
    // set to frac of the total, rounded up.  G = C: the sum of the cluster's
    // histograms; G = 1: this CTA's alone.  Sum u128: bins hold masses in their
    // steps' units, the sums are in units of 2^-58.
    template <int G, typename Sum>
    __device__ int find_bin(Sum above, Sum &target, float frac, Sum &before) {
        constexpr bool MASS = sizeof(Sum) > sizeof(u64);
        constexpr int SL = F_BINS / G;            // bins of this CTA's slice
        constexpr int PT = (SL + NT - 1) / NT;    // bins per thread
        const int part = G == 1 ? 0 : rank;
        if constexpr (G > 1)
            publish();  // every CTA's histogram is complete
        else
            __syncthreads();
        if (lost) return F_BINS - 1;
        Sum v[PT], sum = 0;
        const int b0 = tid * PT;
#pragma unroll
        for (int i = 0; i < PT; ++i) {
            v[i] = 0;
            if (b0 + i < SL) {
                u64 in_bin = 0;
#pragma unroll
                for (int r = 0; r < G; ++r) {
                    const uint32_t *lo = S.lo, *hi = S.hi;
                    if constexpr (G > 1) {
                        lo = cg::this_cluster().map_shared_rank(S.lo, r);
                        hi = cg::this_cluster().map_shared_rank(S.hi, r);
                    }
                    in_bin += ((u64)hi[part * SL + b0 + i] << 32) + lo[part * SL + b0 + i];
                }
                v[i] = in_bin;
                if constexpr (MASS) v[i] <<= F_FRAC - step_frac(part * SL + b0 + i);
            }
            sum += v[i];
        }
        const Sum inc = warp_scan(sum, lane);  // inclusive over the slice
        if (lane == 31) S.wsum[w] = inc;
        if (tid == 0) S.found_bin = 0;
        __syncthreads();
        Sum total = 0;
        if (w == 0) {  // what lies before each warp's bins
            const Sum ws = lane < NW ? (Sum)S.wsum[lane] : 0, wi = warp_scan(ws, lane);
            if (lane < NW) S.wsum[lane] = wi - ws;
            total = shfl(wi, 31);
        }
        exchange<G>(Gather{(u64)total, (uint32_t)((u128)total >> 64), 0u}, [&](const Gather &got) {
            const Sum x = lane < G ? (Sum)wide(got) : 0, xi = warp_scan(x, lane);
            const Sum base = shfl(xi - x, part), all = shfl(xi, 31);
            if (lane == 0) {
                S.base = base;
                if (frac >= 0.f) {
                    const Sum want = (Sum)scaled(frac, all, true);
                    S.target = want == 0 ? 1 : want;
                }
            }
        });
        if (lost) return F_BINS - 1;
        if (frac >= 0.f) target = (Sum)S.target;
        Sum at = above + (Sum)S.base + (Sum)S.wsum[w] + inc - sum;
#pragma unroll
        for (int i = 0; i < PT; ++i) {
            if (at < target && target <= at + v[i]) {
                S.found_bin = (uint32_t)(part * SL + b0 + i) + 1;
                S.found_before = at;
            }
            at += v[i];
        }
        __syncthreads();
        if constexpr (G > 1) {
            exchange<G>(Gather{(u64)S.found_before, (uint32_t)(S.found_before >> 64), S.found_bin}, [&](const Gather &got) {
                const unsigned in = __ballot_sync(0xffffffffu, lane < G && got.c != 0);
                if (lane == (in ? __ffs(in) - 1 : 0)) {
                    S.bin = got.c;
                    S.before = wide(got);
                }
            });
            if (lost) return F_BINS - 1;
        }
        const uint32_t bin = G > 1 ? S.bin : S.found_bin;
        before = bin ? (Sum)(G > 1 ? S.before : S.found_before) : above;
        return bin ? (int)bin - 1 : F_BINS - 1;
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
        publish();
        if (lost) return 0;
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

    // The border among the keys of [kmin, kmax] over the row's logits (list:
    // over the m gathered ones, in this CTA alone), by mass in units of 2^-frac or
    // (frac 0) by count: 2048 equal runs of keys a level, until one key is left.
    // (11 bits a level: at most 3.)
    __device__ uint32_t refine(int frac, bool list, int m, uint32_t kmin, uint32_t kmax, u64 target) {
        const float *src = list ? S.all : reinterpret_cast<const float *>(z4);
        const int n = list ? m : 4 * n4;
        u64 above = 0;
        while (kmin < kmax && !lost) {
            int shift = 0;
            while (((kmax - kmin) >> shift) >= (uint32_t)F_BINS) ++shift;
            clear_hist();
#pragma unroll 1
            for (int i = tid; i < n; i += NT) {
                const float x = src[i];
                const uint32_t key = key_of(x);
                if (key < kmin || key > kmax) continue;
                const u64 wt = frac ? weight_cold(x, frac) : 1ull;
                if (wt) hist_add(S, (int)((kmax - key) >> shift), wt);
            }
            u64 before = 0;
            const uint32_t bin = (uint32_t)(list ? find_bin<1, u64>(above, target, -1.f, before)
                                                 : find_bin<C, u64>(above, target, -1.f, before));
            above = before;
            kmax -= min(bin << shift, kmax - kmin);
            kmin = max(kmin, kmax - min(kmax, (1u << shift) - 1u));
        }
        return kmax;
    }

    // Among the m gathered values from `floor` on, all keys in [kmin, kmax]: the
    // key of the value at which the values at or above it, by their mass in units
    // of 2^-units or (MASS false: no floor) counted, reach the target; with
    // part >= 0 that is this part of them all.
    template <bool MASS>
    __device__ uint32_t border(int m, float floor, int units, u64 target, float part, uint32_t kmin, uint32_t kmax) {
        if constexpr (!MASS) {
            if (m > F_RANK) return refine(0, true, m, kmin, kmax, target);
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
            const u64 v = S.all[i] >= floor ? weight_cold(S.all[i], units) : 0ull;
            if (i < F_RANK) S.mass[i] = v;
            own += v;
        }
        if (part >= 0.f) {
            const u128 all = warp_sum(own);
            if (lane == 0) S.wsum[w] = all;
            __syncthreads();
            target = max((u64)1, (u64)scaled(part, warp_sum(lane < NW ? (u64)S.wsum[lane] : 0ull), true));
        }
        if (m > F_RANK) return refine(units, true, m, max(kmin, key_of(floor)), kmax, target);
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
                last = find_bin<C, u64>(0ull, target, -1.f, before);
                if (lost) return floor;
            }
            const int m = collect(least, [&](float x) { return last == F_BINS || step(x) <= last; }, kmin, kmax);
            if (lost) return floor;
            if (m <= k)
                floor = of_key(kmin);  // (fewer: there are no more above -inf)
            else
                floor = of_key(m <= F_LIST ? border<false>(m, -INFINITY, 0, target, -1.f, kmin, kmax)
                                           : refine(0, false, 0, kmin, kmax, target));
            if (m <= F_LIST) {  // the list holds the whole top-k set
                if (top_p < 1.f)
                    floor = fmaxf(floor, of_key(border<true>(m, floor, F_LIST_FRAC, 0ull, top_p, kmin, kmax)));
                return floor;
            }
        }
        if (top_p < 1.f) {
            clear_hist();
            each([&](float x) {
                if (!(x >= floor)) return;
                const int s = step(x);
                const u64 wt = weight_in_step(x, s);
                if (wt) hist_add(S, s, wt);
            });
            u128 target = 0, before = 0;
            const int at = find_bin<C, u128>(0, target, top_p, before), units = step_frac(at);
            if (lost) return floor;
            // what is wanted of the step, in its units, rounded up
            const u64 rest = (u64)((target - before + (1ull << (F_FRAC - units)) - 1) >> (F_FRAC - units));
            const int m = collect(floor, [&](float x) { return step(x) == at; }, kmin, kmax);
            if (lost) return floor;
            uint32_t key = kmax;
            if (kmin != kmax)
                key = m <= F_LIST ? border<true>(m, floor, units, rest, -1.f, kmin, kmax)
                                  : refine(units, false, 0, kmin, kmax, rest);
            floor = fmaxf(floor, of_key(key));
        }
        return floor;
    }

    // The smallest float at or above max + T ln(p), by one thread: with p = m 2^e,
    // ln m = g + ln(m e^-g) for g near it, and m e^-g - 1 from the exact weight.
    __device__ float min_p_floor(float p, float t) const {
        int e;
        const float m = frexpf(p, &e), g = logf(m);
        const u64 we = weight_call(g, 0.f, 1.44269502162933349609375f, 1.92596299112661746887e-8f, S.pow2, F_FRAC);
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

// The row's draw, by all threads of its CTAs.  false: nothing was exchanged.
template <int NT, int C>
__device__ __forceinline__ bool draw_row(const FilterArgs &a, Row<NT, C> &R, FilterShared &S, float *z, int row, int i0,
                                         int n) {
    constexpr int NW = NT / 32;
    const int tid = R.tid, lane = R.lane, w = R.w, rank = R.rank;
    float *logprob = a.logprob ? a.logprob + row : nullptr;
    const float t = a.temperature ? a.temperature[row] : 1.f, top_p = a.top_p ? a.top_p[row] : 1.f;
    const float min_p = a.min_p ? a.min_p[row] : 0.f, u = a.u[row];
    const int top_k = a.top_k ? a.top_k[row] : 0;
    const bool fine = (t == 0.f || (t >= 1e-30f && t <= 1e30f)) && top_p > 0.f && top_p <= 1.f && min_p >= 0.f &&
                      min_p <= 1.f && u >= 0.f && u < 1.f;
    if (!fine) {  // every CTA of the row sees the same
        if (rank == 0 && tid == 0) no_draw(a.token + row, logprob);
        return false;
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
    R.template exchange<C>(Gather{(u64)bound << 32 | (nan ? 1u : 0u), kmin, kmax}, [&](const Gather &got) {
        const uint32_t lo = __reduce_min_sync(0xffffffffu, got.b), hi = __reduce_max_sync(0xffffffffu, got.c),
                       bd = __reduce_min_sync(0xffffffffu, (uint32_t)(got.a >> 32));
        const int bad = __any_sync(0xffffffffu, (got.a & 1) != 0);
        if (lane == 0) S.kmin = lo, S.kmax = hi, S.bound = bd, S.nan = bad;
    });
    if (R.lost) return true;
    kmin = S.kmin, kmax = S.kmax, bound = S.bound, nan = S.nan != 0;
    if (bound && bound <= key_of(-INFINITY)) bound = kmin;  // a CTA with few logits above -inf: then all of those
    float mx = of_key(kmax);
    if (nan || !(mx > -INFINITY)) {
        if (rank == 0 && tid == 0) no_draw(a.token + row, logprob);
        return true;
    }
    if (t == 0.f) {  // greedy
        uint32_t first = 0xffffffffu, unused = 0;
        for (int i = tid; i < n; i += NT)
            if (z[i] == mx) {
                first = (uint32_t)(i0 + i);
                break;
            }
        R.block_minmax(first, unused);
        R.last_exchange(Gather{0ull, first, 0u}, [&](const Gather &got) {
            const uint32_t least_index = __reduce_min_sync(0xffffffffu, got.b);
            if (lane == 0) S.first = least_index;
        });
        if (rank == 0 && tid == 0 && !R.lost) {
            a.token[row] = (int)S.first;
            if (logprob) *logprob = 0.f;
        }
        return true;
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
    // 32 steps per factor of 2 in weight, more (a power of two) where the whole row spans less
    const float fit = (float)(F_BINS - 1) / ((mx - of_key(kmin)) * R.rs.ch);
    R.rs.oct = fit >= 64.f ? min((int)(__float_as_uint(fit) >> 23) - 127, 30) : 5;
    R.rs.step = R.rs.ch * (float)(1 << R.rs.oct);

    float floor = infinite ? 0.f : R.bounds(k, top_p, bound);
    if (R.lost) return true;
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
    const u128 own_mass = warp_sum(mine);
    __syncthreads();
    if (lane == 0) S.wsum[w] = own_mass;
    __syncthreads();
    // warp 0 finds the warp, if it is one of this CTA, whose range holds the crossing
    u128 ws = 0, wi = 0, all = 0;
    if (w == 0) {
        ws = lane < NW ? S.wsum[lane] : 0;
        wi = warp_scan(ws, lane);
        all = shfl(wi, 31);
    }
    R.last_exchange(Gather{(u64)all, (uint32_t)(all >> 64), 0u}, [&](const Gather &got) {
        const u128 x = lane < C ? wide(got) : 0, xi = warp_scan(x, lane), total = shfl(xi, 31);
        const u128 before = shfl(xi - x, rank) + wi - ws, goal = scaled(u, total, false);  // running > u * total <=> running > that
        const bool mine_is_it = before <= goal && goal - before < ws;
        const unsigned in = __ballot_sync(0xffffffffu, mine_is_it);
        if (lane == 0) S.winner = in ? __ffs(in) - 1 : -1;
        if (mine_is_it) {
            S.left = goal - before;
            S.total = total;
        }
    });
    if (R.lost || w != S.winner) return true;
    const u128 total = S.total;
    u128 left = S.left;
    for (int c0 = 4 * q0; c0 < 4 * q1; c0 += 32) {
        const int i = c0 + lane;
        const float x = i < 4 * q1 ? z[i] : -INFINITY;
        const u64 inc = warp_scan(x >= floor ? R.weight_cold(x, F_FRAC) : 0ull, lane);  // (32 of them fit 64 bits)
        const unsigned hit = __ballot_sync(0xffffffffu, inc > left);
        if (hit) {
            if (lane == __ffs(hit) - 1) {
                a.token[row] = i0 + i;
                // from the logit, not from its rounded weight; the mass is 1 + something (the maximum is kept)
                if (logprob) {
                    const u128 rest = total - ((u128)1 << F_FRAC);
                    const float more = (rest >> 64) == 0 ? (float)(u64)rest * 0x1p-58f : (float)(u64)(rest >> 20) * 0x1p-38f;
                    *logprob = (x == mx ? 0.f : (x - mx) / t) - log1pf(more);
                }
            }
            break;
        }
        left -= shfl(inc, 31);
    }
    return true;
}

template <int NT, int C>
__global__ void __launch_bounds__(NT, 1024 / NT) sample_filtered_kernel(const FilterArgs a) {
    extern __shared__ __align__(16) float z[];  // this CTA's logits
    __shared__ FilterShared S;
    const int row = blockIdx.x / C, rank = blockIdx.x % C;
    const int i0 = rank * a.per, n = max(0, min(a.per, a.vocab - i0));
    Row<NT, C> R(S, z, n, rank, a);
    for (int i = threadIdx.x; i < 256; i += NT) S.pow2[i] = kPow2.v[i];
    if constexpr (C > 1) {
        if (threadIdx.x == 0) {
            mbar_init(&S.bar[0], 1);
            mbar_init(&S.bar[1], 1);
            mbar_init(&S.ready, C);
            S.lost = 0;
            fence_barrier_init();
        }
        cg::this_cluster().sync();  // no message comes before the barriers are there
    }
    pdl_wait();
    pdl_trigger();
    if (draw_row(a, R, S, z, row, i0, n)) R.leave(row);
}

constexpr int kMaxPer = 49152;   // logits of one CTA: 192 KB
constexpr int kPairPer = 20480;  // up to here two CTAs fit an SM's shared memory
// a lane's weights (rounded up, so at most 2^58 each) in the kept mass fit 64 bits
static_assert((kMaxPer / 4 / 32 + 31) / 32 * 4 < 64 && (kPairPer / 4 / 16 + 31) / 32 * 4 < 64, "sums of a lane");

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
    // of one: 160 x 10000 31.1 | 24.9, 200 x 10000 31.1 | 27.4, 240 x 10000 32.2 | 31.7, 300 x
    // 10000 32.4 | 35.9, 200 x 4000 22.7 | 21.1, 260 x 4000 23.0 | 23.9, 200 x 37 10.6 | 13.0;
    // it takes the slower one, 1024, at 120 x 37: 8.8 | 9.8)
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
    // and more.  Measured (us, c = 1 | 2 | 4 | 8): 1 x 32000 17.0 | 12.1 | 9.1 | 7.4,
    // 16 x 32000 42 | 27 | 20 | 18, 40 x 32000 40 | 27 | 23 | 31, 70 x 32000 41 | 28 | 32 | 40,
    // 100 x 32000 42 | 33 | 36 | 51, 100 x 10000 23 | 26 | 29 | 46, 150 x 20000 29 | 34 | 41 | 64,
    // 256 x 32000 58 | 58 | 72 | 109, 1 x 4000 5.9 | 6.4 | 6.1 | 6.4.  Not the best choice at 32 x
    // 131072, where 4 take 43.6 and 8 would 40.0, and at 20 x 20000 (4: 20.6, 8: 19.5).
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

#ifdef LF_DEBUG
std::atomic<long long> g_wait_cycles{F_WAIT_CYCLES};
std::atomic<int> g_lose_rank{-1}, g_lose_wait{0};
#endif

}  // namespace

lf_status launch_sample_filtered(const void *logits, int dtype, int rows, int vocab, int64_t ld, const float *temperature,
                                 const int32_t *top_k, const float *top_p, const float *min_p, const float *u,
                                 int32_t *token, float *logprob, uint32_t *err, cudaStream_t stream) {
    const int bytes = dtype_bytes(dtype);
    auto off = [](const void *p, int b) { return (reinterpret_cast<uintptr_t>(p) & (uintptr_t)(b - 1)) != 0; };
    if (!bytes || !logits || !u || !token || rows < 0 || vocab < 1 || ld < vocab || off(logits, bytes) ||
        off(temperature, 4) || off(top_k, 4) || off(top_p, 4) || off(min_p, 4) || off(u, 4) || off(token, 4) ||
        off(logprob, 4))
        return LF_ERR_INVALID_ARG;
    if (vocab > F_MAX_VOCAB) return LF_ERR_UNSUPPORTED;
    if (rows > (1 << 24)) return LF_ERR_INVALID_ARG;
    if (rows == 0) return LF_OK;
    FilterArgs a = {};
    a.logits = logits;
    a.dtype = dtype;
    a.rows = rows;
    a.vocab = vocab;
    a.ld = ld;
    a.temperature = temperature;
    a.top_k = top_k;
    a.top_p = top_p;
    a.min_p = min_p;
    a.u = u;
    a.token = token;
    a.logprob = logprob;
    a.err = err;
    a.wait_cycles = F_WAIT_CYCLES;
#ifdef LF_DEBUG
    a.wait_cycles = g_wait_cycles;
    a.lose_rank = g_lose_rank;
    a.lose_wait = g_lose_wait;
#endif
    return launch_filtered(a, stream);
}

}  // namespace lf

extern "C" lf_status lf_sample_filtered(const void *logits_device, int dtype, int rows, int vocab, int64_t ld,
                                        const float *temperature_device, const int32_t *top_k_device,
                                        const float *top_p_device, const float *min_p_device, const float *u_device,
                                        int32_t *token_device, float *logprob_device, void *cuda_stream) {
    return lf::launch_sample_filtered(logits_device, dtype, rows, vocab, ld, temperature_device, top_k_device, top_p_device,
                                      min_p_device, u_device, token_device, logprob_device, nullptr,
                                      static_cast<cudaStream_t>(cuda_stream));
}

extern "C" lf_status lf_debug_sample_wait(uint64_t limit_ns, int rank, int nth) {
    if (limit_ns > 2000000000ull || rank < -1 || nth < 0) return LF_ERR_INVALID_ARG;
#ifdef LF_DEBUG
    lf::g_wait_cycles = (long long)limit_ns * 2;
    lf::g_lose_rank = rank;
    lf::g_lose_wait = nth;
    return LF_OK;
#else
    return LF_ERR_UNSUPPORTED;
#endif
}
