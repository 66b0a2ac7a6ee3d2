// Log probabilities of given tokens, with the distribution's entropy, the token's
// rank and the most probable tokens, in one pass over the logits.
//
// With a_i = (z_i - m) / T, m the maximum, S = sum e^a and E = sum a e^a:
//   ln p_t = a_t - ln S,   entropy = ln S - E / S.
// Each thread keeps its own running (m, S, E); when its maximum moves by d (in
// units of 1 / T, d <= 0) the sums follow as E' = e^d (E + d S), S' = e^d S, and
// the same joins the threads, warps and CTAs of a row.  The rank counts what comes
// before the token, whose logit is read first.
//
// The most probable tokens: the top_n-th largest of the threads' maxima is a
// lower bound of the top_n-th largest logit, and only threads whose maximum
// reaches it hold candidates (as many as tokens are wanted, unless there are ties),
// so a second look is at a few hundredths of the row, from L2.  Candidates are
// ordered pairwise.  Where there are more candidates than the list holds (rows of
// many equal logits) the tokens are found one at a time instead.
//
// Each thread has its next LP_STAGES - 1 batches of LP_U 16-byte pieces on their
// way into its own places of shared memory (no barrier), and the maximum lags: it
// moves only when a logit's exponential lies over 2^3 above it, so that most batches
// take an exponential and two multiply-adds a logit and little else.  Logits of
// -inf (a masked vocabulary) take a way of their own.
//
// What bounds it: HBM for many rows of fp32, the call and the second look for few
// (300 x 50257, two thirds masked, in 19.9 us, of which 9 are the bytes; 1 x 32000 with
// five of the most probable tokens in 6.5, 4.3 without), the instructions of a logit for 16
// bits (2048 x 131072 bf16 in 105.9 us, 75 % of the copy rate; 74 % of the issue
// slots are taken).  Batches of two pieces took 110.6 us there; one stage more or
// batches of four pieces took no less.
#include <cooperative_groups.h>

#include <algorithm>
#include <type_traits>

#include "lf_paged.h"
#include "lf_ptx.cuh"

namespace cg = cooperative_groups;

namespace lf {
namespace {

constexpr int LP_THREADS = 256, LP_WARPS = LP_THREADS / 32, LP_TOP = 32, LP_LIST = 512, LP_PARTS = 8;
constexpr int LP_U = 3, LP_STAGES = 3;  // 16-byte pieces of a thread's batch, batches on their way
constexpr int LP_RING = LP_STAGES * LP_U * LP_THREADS * 16;
constexpr int LP_MAX_VOCAB = 1 << 18;
constexpr float kLog2E = 1.4426950408889634f, kLn2 = 0.69314718055994530942f;

struct LpArgs {
    const void *z;
    long long ld;
    int rows, vocab, top, parts;
    const float *temperature;
    const int32_t *token;
    float *logprob, *entropy, *top_logprob;
    int32_t *rank, *top_token;
};

__device__ __forceinline__ float lp_ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// A running maximum with the sums below it, in units of log2: s = sum 2^d, e = sum d 2^d, d = (z - m) c.
struct Sums {
    float m, s, e;
    // The sums as of another maximum, at least as large.
    __device__ __forceinline__ void move(float to, float c) {
        if (m == to) return;
        if (m == -INFINITY) {
            s = e = 0.f;
        } else {
            const float d = fmaxf((m - to) * c, -1e30f), f = lp_ex2(d);
            e = f * fmaf(d, s, e);
            s *= f;
        }
        m = to;
    }
    __device__ __forceinline__ void join(Sums o, float c) {
        const float to = fmaxf(m, o.m);
        if (to == INFINITY) {  // (no sums are kept then)
            m = to;
            return;
        }
        move(to, c);
        o.move(to, c);
        s += o.s;
        e += o.e;
    }
};

// What a CTA of a row tells the row's first.
struct LpPart {
    Sums sums;
    int before, bad, infs;  // logits before the token; a NaN; logits of +inf
    int n;                  // candidates of this part, in order
    float top[LP_TOP];
    int at[LP_TOP];
};

struct LpShared {
    LpPart part, all[LP_PARTS];  // all: of the CTAs of the row, in its first
    Sums warp_sums[LP_WARPS];
    int warp_count[LP_WARPS][3];
    float best[LP_WARPS][LP_TOP];  // each warp's maxima in descending order
    float bound;
    int n_list, n_hold;
    int hold[LP_THREADS];  // threads that hold candidates; in the end the places of the parts' candidates among all
    float list_z[LP_LIST];
    int list_at[LP_LIST];
    float pick_z[LP_WARPS];
    int pick_at[LP_WARPS];
    float row_m, row_norm;
    int row_ok;
};

// Comes before in the order of the most probable: the larger logit, the lower index among equal ones.
__device__ __forceinline__ bool precedes(float z, int at, float y, int other) { return z > y || (z == y && at < other); }

template <typename T>
struct Vec {
    static constexpr int N = 16 / (int)sizeof(T);
};
template <typename T>
__device__ __forceinline__ void unpack(const uint4 &q, float *f) {
    if constexpr (sizeof(T) == 4) {
        f[0] = __uint_as_float(q.x), f[1] = __uint_as_float(q.y), f[2] = __uint_as_float(q.z), f[3] = __uint_as_float(q.w);
    } else {
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float2 y;
            if constexpr (std::is_same<T, __half>::value)
                y = __half22float2(*reinterpret_cast<const __half2 *>(w + i));
            else  // (a bf16 is an fp32's upper half)
                y = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
            f[2 * i] = y.x, f[2 * i + 1] = y.y;
        }
    }
}

// A row's share of one CTA: whole 16-byte pieces [v0, v1) from `body` on, and in the
// first and last share the few logits before and behind them.
template <typename T>
struct Share {
    const T *row, *body;
    int head, v0, v1;  // logits before body
    int extra0, extras;  // first of them; how many single logits this share has
    int tail_at;         // index of the first single logit behind the pieces
    __device__ Share(const LpArgs &a, long long r, int part) {
        row = static_cast<const T *>(a.z) + r * a.ld;
        const int lead = (int)(((16u - (uint32_t)(reinterpret_cast<uintptr_t>(row) & 15u)) & 15u) / sizeof(T));
        head = min(lead, a.vocab);
        body = row + head;
        const int pieces = (a.vocab - head) / Vec<T>::N;
        v0 = (int)((long long)pieces * part / a.parts);
        v1 = (int)((long long)pieces * (part + 1) / a.parts);
        tail_at = head + pieces * Vec<T>::N;
        extra0 = part == 0 ? 0 : head;
        extras = (part == 0 ? head : 0) + (part == a.parts - 1 ? a.vocab - tail_at : 0);
    }
    // index of this share's i-th single logit
    __device__ int extra(int i) const { return extra0 + i < head ? extra0 + i : tail_at + (extra0 + i - head); }
    __device__ int index(int piece) const { return head + piece * Vec<T>::N; }
};

// The next value of the type above z, for which y > z says y >= it; a NaN (never
// reached) above +inf and for a NaN.
__device__ __forceinline__ float next_above(float z) {
    if (!(z < INFINITY)) return NAN;
    const int i = __float_as_int(z + 0.f);  // (no -0)
    return i == 0x80000000 || i == 0 ? __int_as_float(1) : __int_as_float(i + (i > 0 ? 1 : -1));
}
template <typename T>
__device__ __forceinline__ T next_above16(T z) {  // the same for 16 bits
    uint16_t i = *reinterpret_cast<const uint16_t *>(&z);
    if (!((float)z < INFINITY))
        i = 0x7fff;
    else if ((i & 0x7fff) == 0)
        i = 1;
    else
        i += i & 0x8000 ? -1 : 1;
    return *reinterpret_cast<const T *>(&i);
}

// Two values to an instruction.
__device__ __forceinline__ float2 lp_fma2(float2 x, float2 y, float2 z) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(r)
        : "l"(*reinterpret_cast<const uint64_t *>(&x)), "l"(*reinterpret_cast<const uint64_t *>(&y)),
          "l"(*reinterpret_cast<const uint64_t *>(&z)));
    return *reinterpret_cast<float2 *>(&r);
}
__device__ __forceinline__ float2 lp_add2(float2 x, float2 y) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;"
        : "=l"(r)
        : "l"(*reinterpret_cast<const uint64_t *>(&x)), "l"(*reinterpret_cast<const uint64_t *>(&y)));
    return *reinterpret_cast<float2 *>(&r);
}
__device__ __forceinline__ float2 lp_mul2(float2 x, float2 y) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;"
        : "=l"(r)
        : "l"(*reinterpret_cast<const uint64_t *>(&x)), "l"(*reinterpret_cast<const uint64_t *>(&y)));
    return *reinterpret_cast<float2 *>(&r);
}

// What a token's logit is compared with: pieces before its own count equal logits too.
template <typename T>
struct Before {
    float z, above;
    uint32_t z2, above2;  // both halves, 16-bit types
    int token, piece;     // its piece (below all, above all: in the single logits)
    int own;              // its index from the first piece on
    __device__ Before(float zt, int tok, const Share<T> &sh) {
        z = tok < 0 ? NAN : zt;
        above = next_above(z);
        token = tok;
        own = tok - sh.head;
        piece = tok < sh.head ? -1 : tok >= sh.tail_at ? INT32_MAX : (tok - sh.head) / Vec<T>::N;
        z2 = above2 = 0;
        if constexpr (sizeof(T) == 2) {
            const T t = (T)z, u = next_above16<T>(t);
            z2 = *reinterpret_cast<const uint16_t *>(&t) * 0x10001u;
            above2 = *reinterpret_cast<const uint16_t *>(&u) * 0x10001u;
        }
    }
};

// One thread's walk over its pieces.
template <typename T>
struct Walk {
    static constexpr int N = Vec<T>::N;
    using T2 = std::conditional_t<std::is_same<T, __half>::value, __half2, __nv_bfloat162>;
    // The sums are taken below m, which moves when a larger logit lies over 2^kLag above it: they stay as exact, and few
    // threads ever move.
    static constexpr float kLag = 3.f;
    float m, limit, c;  // limit: what a logit must pass for m to move
    float2 s, e;        // (in two halves)
    float best;
    uint32_t before, masks;  // masks: of 16-bit comparisons, L of lower and H of upper halves as 65536 (L - H) - L
    int bad, infs;
    bool masked;

    __device__ __forceinline__ Walk(float c_) : c(c_), masked(false) {
        m = limit = best = -INFINITY;
        s = e = make_float2(0.f, 0.f);
        before = masks = 0;
        bad = infs = 0;
    }
    __device__ __forceinline__ Sums sums() const { return Sums{m, s.x + s.y, e.x + e.y}; }
    __device__ __forceinline__ int count() const {
        const int low = (int)((0u - masks) & 0xffffu);  // L
        return (int)before + low + (low - (int16_t)((masks + (uint32_t)low) >> 16));
    }
    __device__ __forceinline__ void move(float to) {
        Sums t = sums();
        t.move(to, c);
        m = to;
        limit = to + kLag / c;
        s = make_float2(t.s, 0.f), e = make_float2(t.e, 0.f);
    }

    template <int U>
    __device__ __forceinline__ void add(const uint4 *q, int v, const Before<T> &b) {  // pieces v, v + LP_THREADS, ..
        const float lm = largest<U>(q);
        best = fmaxf(best, lm);
        if (lm > limit) move(lm);
        if (!masked) {
            const float2 was_s = s, was_e = e;
            terms<U, false>(q);
            // a masked logit (0 times an infinite d is none), or one that is not finite: from here on the other way
            if (!(fabsf(e.x + e.y) < INFINITY)) masked = true, s = was_s, e = was_e;
        }
        if (masked) {
            uint4 again[U];  // (unpacked anew: kept values would cost the common way its registers)
#pragma unroll
            for (int u = 0; u < U; ++u) {
                again[u] = q[u];
                asm volatile("" : "+r"(again[u].x), "+r"(again[u].y), "+r"(again[u].z), "+r"(again[u].w));
            }
            bad |= lm != lm;
            if (fabsf(m) < INFINITY) terms<U, true>(again);  // (no sums without a finite maximum)
            if (lm == INFINITY) {
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    float f[N];
                    unpack<T>(again[u], f);
#pragma unroll
                    for (int i = 0; i < N; ++i) infs += f[i] == INFINITY;
                }
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int at = v + u * LP_THREADS;
            if constexpr (sizeof(T) == 4) {
                float f[N];
                unpack<T>(q[u], f);
                const float to = at < b.piece ? b.z : b.above;
#pragma unroll
                for (int i = 0; i < N; ++i) before += f[i] >= to;
            } else {
                const uint32_t to = at < b.piece ? b.z2 : b.above2, *w = reinterpret_cast<const uint32_t *>(&q[u]);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    masks += __hge2_mask(*reinterpret_cast<const T2 *>(w + i), *reinterpret_cast<const T2 *>(&to));
            }
            if (at == b.piece) {  // equal logits before the token in its own piece
                uint4 own = q[u];
                asm volatile("" : "+r"(own.x), "+r"(own.y), "+r"(own.z), "+r"(own.w));
                float f[N];
                unpack<T>(own, f);
#pragma unroll
                for (int i = 0; i < N; ++i) before += at * N + i < b.own && f[i] == b.z;
            }
        }
    }
    // The largest of the pieces' values; a NaN if there is one.
    template <int U>
    __device__ __forceinline__ float largest(const uint4 *q) {
        const uint32_t *w = reinterpret_cast<const uint32_t *>(q);
        if constexpr (sizeof(T) == 4) {
            float y = __uint_as_float(w[0]);
            asm("max.NaN.f32 %0, %0, %1;" : "+f"(y) : "f"(__uint_as_float(w[1])));
#pragma unroll
            for (int i = 2; i < 4 * U; i += 2)
                asm("max.NaN.f32 %0, %0, %1, %2;" : "+f"(y) : "f"(__uint_as_float(w[i])), "f"(__uint_as_float(w[i + 1])));
            return y;
        } else {
            T2 y = *reinterpret_cast<const T2 *>(w);
#pragma unroll
            for (int i = 1; i < 4 * U; ++i) y = __hmax2_nan(y, *reinterpret_cast<const T2 *>(w + i));
            float z;
            asm("max.NaN.f32 %0, %1, %2;" : "=f"(z) : "f"((float)y.x), "f"((float)y.y));
            return z;
        }
    }
    // Adds the pieces' terms below m.  CLAMP: a term of an infinite distance adds nothing (a NaN stays one).
    template <int U, bool CLAMP>
    __device__ __forceinline__ void terms(const uint4 *q) {
        const float2 m2 = make_float2(-m, -m), c2 = make_float2(c, c);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float2 f[N / 2];
            unpack<T>(q[u], reinterpret_cast<float *>(f));
#pragma unroll
            for (int i = 0; i < N / 2; ++i) {
                float2 d = lp_mul2(lp_add2(f[i], m2), c2);
                if (CLAMP) {
                    asm("max.NaN.f32 %0, %0, %1;" : "+f"(d.x) : "f"(-1e30f));
                    asm("max.NaN.f32 %0, %0, %1;" : "+f"(d.y) : "f"(-1e30f));
                }
                const float2 p = make_float2(lp_ex2(d.x), lp_ex2(d.y));
                s = lp_add2(s, p);
                e = lp_fma2(d, p, e);
            }
        }
    }
    __device__ __forceinline__ void add_one(float f, int at, const Before<T> &b) {
        best = fmaxf(best, f);
        bad |= f != f;
        infs += f == INFINITY;
        if (f > limit) move(f);
        if (fabsf(m) < INFINITY) {
            const float d = fmaxf((f - m) * c, -1e30f), p = lp_ex2(d);
            s.x += p;
            e.x = fmaf(d, p, e.x);
        }
        before += precedes(f, at, b.z, b.token);
    }
};

// The CTA's most probable tokens one at a time: for rows whose candidates are too
// many for the list.
template <typename T>
__device__ void pick_slowly(const LpArgs &a, const Share<T> &sh, LpShared &S) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    float last_z = INFINITY;
    int last_at = -1, n = 0;
    for (; n < a.top; ++n) {
        float z = -INFINITY;
        int at = INT32_MAX;
        auto look = [&](float y, int i) {
            if (precedes(last_z, last_at, y, i) && precedes(y, i, z, at)) z = y, at = i;
        };
        for (int v = sh.v0 + tid; v < sh.v1; v += LP_THREADS) {
            float f[Vec<T>::N];
            unpack<T>(reinterpret_cast<const uint4 *>(sh.body)[v], f);
#pragma unroll
            for (int i = 0; i < Vec<T>::N; ++i) look(f[i], sh.index(v) + i);
        }
        for (int i = tid; i < sh.extras; i += LP_THREADS) look((float)sh.row[sh.extra(i)], sh.extra(i));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const float y = __shfl_xor_sync(0xffffffffu, z, o);
            const int i = __shfl_xor_sync(0xffffffffu, at, o);
            if (precedes(y, i, z, at)) z = y, at = i;
        }
        if (lane == 0) S.pick_z[warp] = z, S.pick_at[warp] = at;
        __syncthreads();
        z = S.pick_z[0], at = S.pick_at[0];
        for (int w = 1; w < LP_WARPS; ++w)
            if (precedes(S.pick_z[w], S.pick_at[w], z, at)) z = S.pick_z[w], at = S.pick_at[w];
        if (z == -INFINITY) break;  // (the same in all threads)
        if (tid == 0) S.part.top[n] = z, S.part.at[n] = at;
        last_z = z, last_at = at;
        __syncthreads();
    }
    if (tid == 0) S.part.n = n;
}

// 32 values of a warp in descending order.
__device__ __forceinline__ float sort_desc(float x, int lane) {
#pragma unroll
    for (int k = 2; k <= 32; k <<= 1)
#pragma unroll
        for (int j = k >> 1; j > 0; j >>= 1) {
            const float y = __shfl_xor_sync(0xffffffffu, x, j);
            const bool up = (lane & k) != 0, low = (lane & j) == 0;  // ascending runs; the lower of the pair
            x = low != up ? fmaxf(x, y) : fminf(x, y);
        }
    return x;
}
// The 32 largest of two descending lists of 32, in descending order.
__device__ __forceinline__ float merge_desc(float a, float b_reversed, int lane) {
    float x = fmaxf(a, b_reversed);
#pragma unroll
    for (int j = 16; j > 0; j >>= 1) {
        const float y = __shfl_xor_sync(0xffffffffu, x, j);
        x = (lane & j) == 0 ? fmaxf(x, y) : fminf(x, y);
    }
    return x;
}

// The places of the parts' candidates among all, by the warps behind the first (the sums of the row take that one as long):
// eight lanes to four candidates of a list, a list to a lane.  A thread to a candidate took 8.0 us for 1 x 32000 and five
// tokens where this takes 6.5.
__device__ __forceinline__ void places(const LpPart *all, int *place, int parts, int top) {
    constexpr int kC = 4;
    const int lane = threadIdx.x & 31, o = threadIdx.x % LP_PARTS;
    const int per = (top + kC - 1) / kC, n = o < parts ? all[o].n : 0;
    for (int y = ((int)threadIdx.x - 32) / LP_PARTS; y < parts * per; y += (LP_THREADS - 32) / LP_PARTS) {
        const int k = y / per, i = (y - k * per) * kC;
        float z[kC];
        int at[kC], ahead[kC] = {};
#pragma unroll
        for (int e = 0; e < kC; ++e) z[e] = all[k].top[i + e], at[e] = all[k].at[i + e];
#pragma unroll 2
        for (int x = 0; x < n; ++x) {
            const float lz = all[o].top[x];
            const int lat = all[o].at[x];
#pragma unroll
            for (int e = 0; e < kC; ++e) ahead[e] += precedes(lz, lat, z[e], at[e]);
        }
#pragma unroll
        for (int e = 0; e < kC; ++e) {
#pragma unroll
            for (int d = LP_PARTS / 2; d > 0; d /= 2) ahead[e] += __shfl_xor_sync(0xffu << (lane & 24), ahead[e], d);
            if (o == e) place[k * LP_TOP + i + e] = ahead[e];
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(LP_THREADS, 4) token_logprobs_kernel(const LpArgs a) {
    __shared__ LpShared S;
    constexpr int N = Vec<T>::N, U = LP_U;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const long long r = blockIdx.x / (unsigned)a.parts;
    const int part = (int)(blockIdx.x - r * a.parts);
    cg::cluster_group cl = cg::this_cluster();
    pdl_wait();
    pdl_trigger();
    if (a.parts > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;");  // (every CTA of the row has begun: below)
    const Share<T> sh(a, r, part);
    // Each thread copies its own pieces, a batch of U at a time, into its own places of a ring and reads them back:
    // enough on their way for HBM without holding registers, and no barrier.
    const uint4 *body = reinterpret_cast<const uint4 *>(sh.body);
    extern __shared__ __align__(16) uint4 ring[];  // [LP_STAGES][U][LP_THREADS]
    const int pieces = sh.v1 - sh.v0 - tid, batches = pieces <= 0 ? 0 : (pieces + LP_THREADS - 1) / LP_THREADS / U;
    const uint4 *from = body + sh.v0 + tid;
    uint4 *const mine = ring + tid;
    int in = 0;  // copies: the stage they go to
    auto fetch = [&](int k) {
        if (k < batches) {
#pragma unroll
            for (int u = 0; u < U; ++u) cp_async16(mine + in + u * LP_THREADS, from + u * LP_THREADS);
            from += U * LP_THREADS;
            in = in + U * LP_THREADS == LP_STAGES * U * LP_THREADS ? 0 : in + U * LP_THREADS;
        }
        cp_async_commit();
    };
#pragma unroll
    for (int k = 0; k < LP_STAGES - 1; ++k) fetch(k);
    const float temp = a.temperature ? a.temperature[r] : 1.f;
    const int token = a.token ? a.token[r] : -1;
    const bool asked = token >= 0 && token < a.vocab;
    const float zt = asked ? (float)sh.row[token] : NAN;
    const bool warm = temp >= 1e-30f && temp <= 1e30f;
    const float c = warm ? kLog2E / temp : 1.f;
    const Before<T> b(zt, asked ? token : -1, sh);
    Walk<T> w(c);
    int v = sh.v0 + tid;
    for (int k = 0, out = 0; k < batches; ++k, v += U * LP_THREADS) {
        fetch(k + LP_STAGES - 1);
        asm volatile("cp.async.wait_group %0;" ::"n"(LP_STAGES - 1) : "memory");
        uint4 q[U];
#pragma unroll
        for (int u = 0; u < U; ++u) q[u] = mine[out + u * LP_THREADS];
        out = out + U * LP_THREADS == LP_STAGES * U * LP_THREADS ? 0 : out + U * LP_THREADS;
        w.template add<U>(q, v, b);
    }
#pragma unroll
    for (int u = 0; u < U - 1; ++u, v += LP_THREADS)  // less than a batch is left
        if (v < sh.v1) {
            const uint4 q = body[v];
            w.template add<1>(&q, v, b);
        }
    if (tid < sh.extras) w.add_one((float)sh.row[sh.extra(tid)], sh.extra(tid), b);
    // the CTA's sums, below its maximum
    float m = w.best;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const int n_bad = __reduce_or_sync(0xffffffffu, w.bad), n_inf = __reduce_add_sync(0xffffffffu, w.infs),
              n_before = __reduce_add_sync(0xffffffffu, w.count());
    Sums t0 = w.sums();
    t0.move(m, c);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        t0.s += __shfl_xor_sync(0xffffffffu, t0.s, o);
        t0.e += __shfl_xor_sync(0xffffffffu, t0.e, o);
    }
    if (lane == 0) {
        S.warp_sums[warp] = t0;
        S.warp_count[warp][0] = n_before, S.warp_count[warp][1] = n_bad, S.warp_count[warp][2] = n_inf;
    }
    float x = 0.f;
    if (a.top > 0) S.best[warp][lane] = x = sort_desc(w.best, lane);
    if (tid == 0) S.n_list = S.n_hold = 0;
    __syncthreads();
    if (tid == 0) {
        Sums t = S.warp_sums[0];
        int before = S.warp_count[0][0], bad = S.warp_count[0][1], infs = S.warp_count[0][2];
#pragma unroll
        for (int k = 1; k < LP_WARPS; ++k) {
            t.join(S.warp_sums[k], c);
            before += S.warp_count[k][0], bad |= S.warp_count[k][1], infs += S.warp_count[k][2];
        }
        S.part.sums = t;
        S.part.before = before, S.part.bad = bad, S.part.infs = infs, S.part.n = 0;
    }
    if (a.top > 0) {
        // the top_n-th largest of the threads' maxima: the warps' lists in pairs (the last warps, beside the sums)
#pragma unroll
        for (int half = LP_WARPS / 2; half > 0; half /= 2) {
            if (warp >= LP_WARPS - half) {
                x = merge_desc(x, S.best[warp - half][31 - lane], lane);
                if (half > 1) S.best[warp][lane] = x;
                if (half == 1 && lane == a.top - 1) S.bound = x;
            }
            __syncthreads();
        }
        const float bound = S.bound;
        if (w.best >= bound && w.best > -INFINITY) S.hold[atomicAdd(&S.n_hold, 1)] = tid;
        __syncthreads();
        // every piece of the threads that hold candidates, spread over the CTA
        const int hold = S.n_hold, steps = (sh.v1 - sh.v0 + LP_THREADS - 1) / LP_THREADS;
        auto keep = [&](float z, int at) {
            if (z >= bound && z > -INFINITY) {
                const int i = atomicAdd(&S.n_list, 1);
                if (i < LP_LIST) S.list_z[i] = z, S.list_at[i] = at;
            }
        };
        for (int y = tid; y < hold * steps; y += LP_THREADS) {
            const int p = sh.v0 + y / hold * LP_THREADS + S.hold[y % hold];
            if (p >= sh.v1) continue;
            float f[N];
            unpack<T>(body[p], f);
#pragma unroll
            for (int i = 0; i < N; ++i) keep(f[i], sh.index(p) + i);
        }
        if (tid < sh.extras) keep((float)sh.row[sh.extra(tid)], sh.extra(tid));
        __syncthreads();
        const int n = S.n_list;
        if (n > LP_LIST) {
            pick_slowly<T>(a, sh, S);
        } else if (n <= 64) {  // (nearly always) a lane holds two candidates, a warp counts those before one
            const float z0 = lane < n ? S.list_z[lane] : -INFINITY, z1 = lane + 32 < n ? S.list_z[lane + 32] : -INFINITY;
            const int at0 = lane < n ? S.list_at[lane] : INT32_MAX, at1 = lane + 32 < n ? S.list_at[lane + 32] : INT32_MAX;
            for (int y = warp; y < n; y += LP_WARPS) {
                const float z = S.list_z[y];
                const int at = S.list_at[y];
                const int ahead = __popc(__ballot_sync(0xffffffffu, precedes(z0, at0, z, at))) +
                                  __popc(__ballot_sync(0xffffffffu, precedes(z1, at1, z, at)));
                if (lane == 0 && ahead < a.top) S.part.top[ahead] = z, S.part.at[ahead] = at;
            }
            if (tid == 0) S.part.n = min(n, a.top);
        } else {
            for (int y = tid; y < n; y += LP_THREADS) {
                const float z = S.list_z[y];
                const int at = S.list_at[y];
                int ahead = 0;
                for (int o = 0; o < n; ++o) ahead += precedes(S.list_z[o], S.list_at[o], z, at);
                if (ahead < a.top) S.part.top[ahead] = z, S.part.at[ahead] = at;
            }
            if (tid == 0) S.part.n = min(n, a.top);
        }
    }
    __syncthreads();
    // every CTA's part into the shared memory of the row's first
    if (a.parts > 1) {
        asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
        const uint32_t *src = reinterpret_cast<const uint32_t *>(&S.part);
        uint32_t *dst = reinterpret_cast<uint32_t *>(cl.map_shared_rank(&S.all[part], 0));
        if (tid < (int)(sizeof(LpPart) / 4)) dst[tid] = src[tid];
        cl.sync();
        if (part > 0) return;
    }
    const LpPart *all = a.parts > 1 ? S.all : &S.part;
    if (warp == 0) {
        Sums t = {-INFINITY, 0.f, 0.f};
        int before = 0, bad = 0, infs = 0;
        if (lane < a.parts) {
            t = all[lane].sums;
            before = all[lane].before, bad = all[lane].bad, infs = all[lane].infs;
        }
#pragma unroll
        for (int o = LP_PARTS / 2; o > 0; o >>= 1) {
            Sums y;
            y.m = __shfl_xor_sync(0xffffffffu, t.m, o);
            y.s = __shfl_xor_sync(0xffffffffu, t.s, o);
            y.e = __shfl_xor_sync(0xffffffffu, t.e, o);
            t.join(y, c);
            before += __shfl_xor_sync(0xffffffffu, before, o);
            bad |= __shfl_xor_sync(0xffffffffu, bad, o);
            infs += __shfl_xor_sync(0xffffffffu, infs, o);
        }
        if (lane == 0) {
            const bool ok = warm && !bad && t.m > -INFINITY;
            const bool inf = t.m == INFINITY;
            const float norm = logf(inf ? (float)infs : t.s);
            if (a.entropy) a.entropy[r] = !ok ? NAN : inf ? norm : norm - kLn2 * t.e / t.s;
            if (a.logprob)
                a.logprob[r] = !ok || !asked ? NAN : inf ? (zt == INFINITY ? -norm : -INFINITY) : (zt - t.m) / temp - norm;
            if (a.rank) a.rank[r] = !ok || !asked ? -1 : before;
            S.row_m = t.m, S.row_norm = norm, S.row_ok = ok;
        }
    }
    if (a.top == 0) return;
    if (a.parts > 1 && warp > 0) places(all, S.hold, a.parts, a.top);
    __syncthreads();
    const int k = tid / LP_TOP, i = tid % LP_TOP;
    const float norm = S.row_norm, row_m = S.row_m;
    auto put = [&](int place, int at, float lp) {
        if (a.top_token) a.top_token[r * a.top + place] = at;
        if (a.top_logprob) a.top_logprob[r * a.top + place] = lp;
    };
    if (!S.row_ok) {
        if (tid < a.top) put(tid, -1, NAN);
        return;
    }
    int total = 0;
    for (int o = 0; o < a.parts; ++o) total += all[o].n;
    if (k < a.parts && i < all[k].n) {
        const float z = all[k].top[i];
        const int at = all[k].at[i];
        const int ahead = a.parts > 1 ? S.hold[tid] : i;
        if (ahead < a.top)
            put(ahead, at, row_m == INFINITY ? (z == INFINITY ? -norm : -INFINITY) : (z - row_m) / temp - norm);
    }
    if (tid < a.top && tid >= total) put(tid, -1, -INFINITY);
}

// CTAs to a row (a cluster, joined through distributed shared memory): with few rows as many as there are SMs for, each of
// 4000 logits at least; two CTAs an SM still pay for two to a row.  us by 1 | 2 | 4 | 8 CTAs to a row:
//   fp32, 131072 logits:  1 row 22.8 | 15.5 | 11.6 | 10.1   38 rows 24.2 | 16.8 | 14.0 | 15.3   76 rows 24.5 | 17.3 | 19.8 | 22.6
//                         152 rows 25.2 | 20.8 | 27.9 | 33.3   304 rows 32.8 | 34.0 | 43.3 | 55.1
//   fp32, 32000 logits:   38 rows 10.5 | 9.2 | 8.8 | 10.6   152 rows 12.2 | 11.2 | 17.8 | 23.4   304 rows 14.2 | 15.3 | 26.8 | 39.6
//   bf16, 131072 logits:  38 rows 16.1 | 12.3 | 10.9 | 13.0   152 rows 17.6 | 16.2 | 21.9 | 30.1
int parts_of(int rows, int vocab, int n_sm) {
    int parts = 1;
    while (parts < LP_PARTS && (long long)rows * parts * 2 <= (parts == 1 ? 2 * n_sm : n_sm + n_sm / 16) && vocab / (parts * 2) >= 4000)
        parts *= 2;
    return parts;
}

template <typename T>
bool launch_logprobs(const LpArgs &a, cudaStream_t st) {
    return set_smem_once<token_logprobs_kernel<T>>(LP_RING) &&
           launch_pdl_cluster(token_logprobs_kernel<T>, (unsigned)a.parts, dim3((unsigned)a.rows * (unsigned)a.parts),
                              LP_THREADS, LP_RING, st, a);
}

}  // namespace
}  // namespace lf

extern "C" lf_status lf_token_logprobs(const void *logits_device, int dtype, int rows, int vocab, int64_t ld,
                                       const float *temperature_device, const int32_t *token_device, int top_n,
                                       float *logprob_device, int32_t *rank_device, float *entropy_device,
                                       int32_t *top_token_device, float *top_logprob_device, void *cuda_stream) {
    const int bytes = lf::dtype_bytes(dtype);
    auto off = [](const void *p, int by) { return reinterpret_cast<uintptr_t>(p) % (unsigned)by != 0; };
    if (!bytes || rows < 0 || vocab < 1 || ld < vocab || !logits_device || off(logits_device, bytes) ||
        off(temperature_device, 4) || off(token_device, 4) || off(logprob_device, 4) || off(rank_device, 4) ||
        off(entropy_device, 4) || off(top_token_device, 4) || off(top_logprob_device, 4) || top_n < 0 ||
        top_n > lf::LP_TOP || top_n > vocab || (!token_device && (logprob_device || rank_device)))
        return LF_ERR_INVALID_ARG;
    if (vocab > lf::LP_MAX_VOCAB) return LF_ERR_UNSUPPORTED;
    if (rows == 0) return LF_OK;
    int dev = 0, n_sm = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&n_sm, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n_sm < 1) {
        (void)cudaGetLastError();
        return LF_ERR_CUDA;
    }
    const bool top = top_token_device || top_logprob_device;
    const lf::LpArgs a = {logits_device,  ld,           rows,           vocab,          top ? top_n : 0,    lf::parts_of(rows, vocab, n_sm),
                          temperature_device, token_device, logprob_device, entropy_device, top_logprob_device, rank_device,
                          top_token_device};
    cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
    const bool ok = dtype == LF_F32   ? lf::launch_logprobs<float>(a, st)
                    : dtype == LF_F16 ? lf::launch_logprobs<__half>(a, st)
                                      : lf::launch_logprobs<__nv_bfloat16>(a, st);
    return ok ? LF_OK : LF_ERR_CUDA;
}
