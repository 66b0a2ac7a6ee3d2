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
// What bounds it is HBM, each logit read once.  Few rows are spread over clusters
// of up to 8 CTAs a row, joined through distributed shared memory.
#include <cooperative_groups.h>

#include <algorithm>

#include "lf_paged.h"
#include "lf_ptx.cuh"

namespace cg = cooperative_groups;

namespace lf {
namespace {

constexpr int LP_THREADS = 256, LP_WARPS = LP_THREADS / 32, LP_TOP = 32, LP_LIST = 512, LP_PARTS = 8;
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
__device__ __forceinline__ float lp_max_nan(float a, float b) {
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
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
    LpPart part;
    Sums warp_sums[LP_WARPS];
    int warp_count[LP_WARPS][3];
    float best[LP_WARPS][LP_TOP];  // each warp's maxima in descending order
    float bound;
    int n_list, n_hold;
    int hold[LP_THREADS];          // threads that hold candidates
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
        const T *t = reinterpret_cast<const T *>(&q);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = (float)t[i];
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

// One thread's walk over its pieces.
template <typename T>
struct Walk {
    Sums t;
    int before, bad, infs;
    template <int N>
    __device__ __forceinline__ void add(const float *f, const int *at, float c, float zt, int token) {
        float lm = f[0];
#pragma unroll
        for (int i = 1; i < N; ++i) lm = lp_max_nan(lm, f[i]);
        bad |= lm != lm;
        if (lm > t.m) t.move(lm, c);
        if (t.m > -INFINITY && t.m < INFINITY) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const float d = fmaxf((f[i] - t.m) * c, -1e30f), p = lp_ex2(d);  // (0 times an infinite d is none)
                t.s += p;
                t.e = fmaf(d, p, t.e);
            }
        }
        if (lm == INFINITY) {
#pragma unroll
            for (int i = 0; i < N; ++i) infs += f[i] == INFINITY;
        }
#pragma unroll
        for (int i = 0; i < N; ++i) before += precedes(f[i], at[i], zt, token);
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

template <typename T>
__global__ void __launch_bounds__(LP_THREADS) token_logprobs_kernel(const LpArgs a) {
    __shared__ LpShared S;
    constexpr int N = Vec<T>::N, U = 4;  // pieces in flight
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const long long r = blockIdx.x / (unsigned)a.parts;
    const int part = (int)(blockIdx.x - r * a.parts);
    pdl_wait();
    pdl_trigger();
    const Share<T> sh(a, r, part);
    const float temp = a.temperature ? a.temperature[r] : 1.f;
    const int token = a.token ? a.token[r] : -1;
    const bool asked = token >= 0 && token < a.vocab;
    const float zt = asked ? (float)sh.row[token] : INFINITY;  // (nothing comes before an infinity that is not there)
    const int tok = asked ? token : -1;
    const bool warm = temp >= 1e-30f && temp <= 1e30f;
    const float c = warm ? kLog2E / temp : 1.f;

    Walk<T> w;
    w.t = Sums{-INFINITY, 0.f, 0.f};
    w.before = w.bad = w.infs = 0;
    for (int v = sh.v0 + tid; v < sh.v1; v += U * LP_THREADS) {
        uint4 q[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (v + u * LP_THREADS < sh.v1) q[u] = reinterpret_cast<const uint4 *>(sh.body)[v + u * LP_THREADS];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (v + u * LP_THREADS < sh.v1) {
                float f[N];
                int at[N];
                unpack<T>(q[u], f);
#pragma unroll
                for (int i = 0; i < N; ++i) at[i] = sh.index(v + u * LP_THREADS) + i;
                w.template add<N>(f, at, c, zt, tok);
            }
    }
    for (int i = tid; i < sh.extras; i += LP_THREADS) {
        const int at = sh.extra(i);
        const float f = (float)sh.row[at];
        w.template add<1>(&f, &at, c, zt, tok);
    }
    // the CTA's sums
    const float mine = w.t.m;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        Sums y;
        y.m = __shfl_xor_sync(0xffffffffu, w.t.m, o);
        y.s = __shfl_xor_sync(0xffffffffu, w.t.s, o);
        y.e = __shfl_xor_sync(0xffffffffu, w.t.e, o);
        w.t.join(y, c);
    }
    w.before = __reduce_add_sync(0xffffffffu, w.before);
    w.bad = __reduce_or_sync(0xffffffffu, w.bad);
    w.infs = __reduce_add_sync(0xffffffffu, w.infs);
    if (lane == 0) {
        S.warp_sums[warp] = w.t;
        S.warp_count[warp][0] = w.before, S.warp_count[warp][1] = w.bad, S.warp_count[warp][2] = w.infs;
    }
    if (a.top > 0) S.best[warp][lane] = sort_desc(mine, lane);
    if (tid == 0) S.n_list = S.n_hold = 0;
    __syncthreads();
    if (tid == 0) {
        Sums t = S.warp_sums[0];
        int before = S.warp_count[0][0], bad = S.warp_count[0][1], infs = S.warp_count[0][2];
        for (int k = 1; k < LP_WARPS; ++k) {
            t.join(S.warp_sums[k], c);
            before += S.warp_count[k][0], bad |= S.warp_count[k][1], infs += S.warp_count[k][2];
        }
        S.part.sums = t;
        S.part.before = before, S.part.bad = bad, S.part.infs = infs, S.part.n = 0;
    }
    if (a.top > 0) {
        if (warp == LP_WARPS - 1) {  // the top_n-th largest of the threads' maxima
            float x = S.best[0][lane];
#pragma unroll
            for (int k = 1; k < LP_WARPS; ++k) x = merge_desc(x, S.best[k][31 - lane], lane);
            if (lane == a.top - 1) S.bound = x;
        }
        __syncthreads();
        const float bound = S.bound;
        if (mine >= bound && mine > -INFINITY) S.hold[atomicAdd(&S.n_hold, 1)] = tid;
        __syncthreads();
        // every piece of the threads that hold candidates, spread over the CTA
        const int hold = S.n_hold, steps = (sh.v1 - sh.v0 + LP_THREADS - 1) / LP_THREADS;
        auto keep = [&](float z, int at) {
            if (z >= bound && z > -INFINITY) {
                const int i = atomicAdd(&S.n_list, 1);
                if (i < LP_LIST) S.list_z[i] = z, S.list_at[i] = at;
            }
        };
        for (int x = tid; x < hold * steps; x += LP_THREADS) {
            const int v = sh.v0 + x / hold * LP_THREADS + S.hold[x % hold];
            if (v >= sh.v1) continue;
            float f[N];
            unpack<T>(reinterpret_cast<const uint4 *>(sh.body)[v], f);
#pragma unroll
            for (int i = 0; i < N; ++i) keep(f[i], sh.index(v) + i);
        }
        for (int i = tid; i < sh.extras; i += LP_THREADS) keep((float)sh.row[sh.extra(i)], sh.extra(i));
        __syncthreads();
        const int n = S.n_list;
        if (n > LP_LIST) {
            pick_slowly<T>(a, sh, S);
        } else {
            for (int x = tid; x < n; x += LP_THREADS) {
                const float z = S.list_z[x];
                const int at = S.list_at[x];
                int ahead = 0;
                for (int y = 0; y < n; ++y) ahead += precedes(S.list_z[y], S.list_at[y], z, at);
                if (ahead < a.top) S.part.top[ahead] = z, S.part.at[ahead] = at;
            }
            if (tid == 0) S.part.n = min(n, a.top);
        }
    }
    // the row, by its first CTA
    cg::cluster_group cl = cg::this_cluster();
    if (a.parts > 1)
        cl.sync();
    else
        __syncthreads();
    if (part == 0) {
        auto of = [&](int k) { return a.parts > 1 ? cl.map_shared_rank(&S.part, k) : &S.part; };
        if (tid == 0) {
            Sums t = S.part.sums;
            int before = S.part.before, bad = S.part.bad, infs = S.part.infs;
            for (int k = 1; k < a.parts; ++k) {
                const LpPart *p = of(k);
                t.join(p->sums, c);
                before += p->before, bad |= p->bad, infs += p->infs;
            }
            const bool ok = warm && !bad && t.m > -INFINITY;
            const bool inf = t.m == INFINITY;
            const float norm = logf(inf ? (float)infs : t.s);
            if (a.entropy) a.entropy[r] = !ok ? NAN : inf ? norm : norm - kLn2 * t.e / t.s;
            if (a.logprob)
                a.logprob[r] = !ok || !asked ? NAN : inf ? (zt == INFINITY ? -norm : -INFINITY) : (zt - t.m) / temp - norm;
            if (a.rank) a.rank[r] = !ok || !asked ? -1 : before;
            S.row_m = t.m, S.row_norm = norm, S.row_ok = ok;
        }
        __syncthreads();
        if (a.top > 0 && (a.top_token || a.top_logprob)) {
            // candidates of all parts, a thread to each place
            int total = 0;
            for (int k = 0; k < a.parts; ++k) total += of(k)->n;
            const int k = tid / LP_TOP, i = tid % LP_TOP;
            const float m = S.row_m, norm = S.row_norm;
            auto put = [&](int place, int at, float lp) {
                if (a.top_token) a.top_token[r * a.top + place] = at;
                if (a.top_logprob) a.top_logprob[r * a.top + place] = lp;
            };
            if (!S.row_ok) {
                if (tid < a.top) put(tid, -1, NAN);
            } else {
                if (k < a.parts && i < of(k)->n) {
                    const float z = of(k)->top[i];
                    const int at = of(k)->at[i];
                    int ahead = i;
                    for (int o = 0; o < a.parts; ++o)
                        if (o != k) {
                            const LpPart *p = of(o);
                            const int n = p->n;
                            int x = 0;
                            while (x < n && precedes(p->top[x], p->at[x], z, at)) ++x;
                            ahead += x;
                        }
                    if (ahead < a.top)
                        put(ahead, at, m == INFINITY ? (z == INFINITY ? -norm : -INFINITY) : (z - m) / temp - norm);
                }
                if (tid < a.top && tid >= total) put(tid, -1, -INFINITY);
            }
        }
    }
    if (a.parts > 1) cl.sync();  // nobody leaves while its part is read
}

// CTAs to a row: as many as leave each a few thousand logits, where the rows do not
// fill the SMs by themselves.
int parts_of(int rows, int vocab, int n_sm) {
    int parts = 1;
    while (parts < LP_PARTS && (long long)rows * parts * 2 <= 4ll * n_sm && vocab / (parts * 2) >= 2048) parts *= 2;
    return parts;
}

template <typename T>
bool launch_logprobs(const LpArgs &a, cudaStream_t st) {
    return launch_pdl_cluster(token_logprobs_kernel<T>, (unsigned)a.parts, dim3((unsigned)a.rows * (unsigned)a.parts),
                              LP_THREADS, 0, st, a);
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
