// Append to a paged KV cache with RoPE on the way: the queries and keys of
// each token rotated by its position, keys and values written to the page
// its sequence's table names.
//
//   y[c] = x[c] cos - x[c + h] sin,  y[c + h] = x[c] sin + x[c + h] cos,
//   h = head_dim / 2, (cos, sin) = rope[position][c]
//
// in fp32, rounded once to the cache's type (values: rounded, not rotated).
// A unit of work is 8 pairs of one head of one token: two 16-byte stores (and
// as wide loads as the input's type gives), the same two pieces that the
// rotation couples.  A thread keeps one pair range c .. c + 7 of one token and
// takes U heads of it, so its cos and sin are read once and U units' loads are
// in flight together, started before the position, the table entry and the
// rotation's row (three loads that wait for each other) are looked up.  The
// bound is HBM: every value is read and written once.  Measured: 3584 tokens of
// 32 + 2 x 16 heads of 128, FP16: 22.5 us, 5.3 TB/s (79 % of the copy rate;
// 35.9 us with one unit a thread loaded after the page lookup); 8191 tokens of 24
// + 2 x 8 heads of 64, BF16: 16.6 us, 5.2 TB/s; 16 tokens: 5.2 us, the time
// of the call itself.
#include "lf_paged.h"

namespace lf {
namespace {

constexpr int kAppendThreads = 128;
constexpr long long kAppendManyUnits = 1 << 17;
struct AppendArgs {
    PagedView kv;
    const void *q, *k, *v;
    long long ld_q, ld_k, ld_v, ld_qo;
    void *qo;
    int n_q;
    const int32_t *seq, *pos;
    int n_tokens;
    const float *rope;
    int rope_len;
    uint32_t *err;
};

// 8 consecutive values as they lie in memory, and as fp32.  (The input may be
// the output array itself, rotated in place: no read-only loads.)
template <typename T>
struct Eight;
template <>
struct Eight<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float *p) {
        a = reinterpret_cast<const float4 *>(p)[0];
        b = reinterpret_cast<const float4 *>(p)[1];
    }
    __device__ __forceinline__ void get(float (&f)[8]) const {
        f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
    }
};
template <>
struct Eight<__half> {
    uint4 u;
    __device__ __forceinline__ void load(const __half *p) { u = *reinterpret_cast<const uint4 *>(p); }
    __device__ __forceinline__ void get(float (&f)[8]) const {
        const __half2 *h = reinterpret_cast<const __half2 *>(&u);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 t = __half22float2(h[i]);
            f[2 * i] = t.x, f[2 * i + 1] = t.y;
        }
    }
};
template <>
struct Eight<__nv_bfloat16> {
    uint4 u;
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) { u = *reinterpret_cast<const uint4 *>(p); }
    __device__ __forceinline__ void get(float (&f)[8]) const {
        const __nv_bfloat162 *h = reinterpret_cast<const __nv_bfloat162 *>(&u);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 t = __bfloat1622float2(h[i]);
            f[2 * i] = t.x, f[2 * i + 1] = t.y;
        }
    }
};
__device__ __forceinline__ void store8(__half *p, const float (&f)[8]) {
    __half2 h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
    *reinterpret_cast<uint4 *>(p) = *reinterpret_cast<const uint4 *>(h);
}
__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float (&f)[8]) {
    __nv_bfloat162 h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    *reinterpret_cast<uint4 *>(p) = *reinterpret_cast<const uint4 *>(h);
}

// A token has per_token = pieces * slots threads (pieces = head_dim / 16 pair
// ranges, slots = heads / U rounded up); a block holds whole tokens.
template <typename TI, typename TO, int U>
__global__ void __launch_bounds__(kAppendThreads) kv_append_kernel(const AppendArgs a, int slots) {
    const int DH = a.kv.head_dim, half = DH / 2, pieces = DH / 16, per_token = pieces * slots;
    const long long t_ll = (long long)blockIdx.x * (blockDim.x / per_token) + threadIdx.x / per_token;
    if (t_ll >= a.n_tokens) return;
    const int t = (int)t_ll, x = threadIdx.x % per_token, c0 = x % pieces * 8, slot = x / pieces + slots * blockIdx.y * U;
    const int heads = a.n_q + 2 * a.kv.n_kv;
    pdl_wait();
    pdl_trigger();
    const int seq = a.seq ? a.seq[t] : t;
    const int p = a.pos[t];
    Eight<TI> lo[U], hi[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int h = slot + u * slots;
        if (h < heads) {
            const TI *src;
            if (h < a.n_q)
                src = static_cast<const TI *>(a.q) + (long long)t * a.ld_q + (long long)h * DH;
            else if (h < a.n_q + a.kv.n_kv)
                src = static_cast<const TI *>(a.k) + (long long)t * a.ld_k + (long long)(h - a.n_q) * DH;
            else
                src = static_cast<const TI *>(a.v) + (long long)t * a.ld_v + (long long)(h - a.n_q - a.kv.n_kv) * DH;
            lo[u].load(src + c0);
            hi[u].load(src + half + c0);
        }
    }
    if (seq < 0) return;  // padding
    int page = -1;
    if (seq < a.kv.n_seqs && p >= 0 && (p >> a.kv.ps_log2) < a.kv.max_pages && (!a.rope || p < a.rope_len))
        page = a.kv.table[(long long)seq * a.kv.max_pages + (p >> a.kv.ps_log2)];
    if (page < 0 || page >= a.kv.n_pages) {
        if (x == 0 && blockIdx.y == 0) atomicExch(a.err, 1u);
        return;
    }
    float cs[8], sn[8];
    if (a.rope) {
        const float4 *r = reinterpret_cast<const float4 *>(a.rope + ((long long)p * half + c0) * 2);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float4 y = r[i];
            cs[2 * i] = y.x, sn[2 * i] = y.y, cs[2 * i + 1] = y.z, sn[2 * i + 1] = y.w;
        }
    }
    const int row = p & ((1 << a.kv.ps_log2) - 1);
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int h = slot + u * slots;
        if (h >= heads) break;
        TO *dst;
        if (h < a.n_q) {
            dst = static_cast<TO *>(a.qo) + (long long)t * a.ld_qo + (long long)h * DH;
        } else {
            const int g = h < a.n_q + a.kv.n_kv ? h - a.n_q : h - a.n_q - a.kv.n_kv;
            TO *base = static_cast<TO *>(h < a.n_q + a.kv.n_kv ? a.kv.k : a.kv.v);
            dst = base + page * a.kv.page_stride + ((((long long)g << a.kv.ps_log2) + row) * DH);
        }
        float fl[8], fh[8];
        lo[u].get(fl);
        hi[u].get(fh);
        if (a.rope && h < a.n_q + a.kv.n_kv) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float y = fl[i], z = fh[i];
                fl[i] = y * cs[i] - z * sn[i];
                fh[i] = y * sn[i] + z * cs[i];
            }
        }
        store8(dst + c0, fl);
        store8(dst + half + c0, fh);
    }
}

template <typename TI, typename TO, int U>
bool launch_units(const AppendArgs &a, cudaStream_t st) {
    const int pieces = a.kv.head_dim / 16, heads = a.n_q + 2 * a.kv.n_kv;  // pieces: 1 .. 16
    const int slots = min((heads + U - 1) / U, kAppendThreads / pieces);
    const int tokens = kAppendThreads / (pieces * slots);  // per block
    const int y = (heads + slots * U - 1) / (slots * U);
    return launch_pdl(kv_append_kernel<TI, TO, U>, dim3((unsigned)((a.n_tokens - 1) / tokens + 1), (unsigned)y),
                      (unsigned)(pieces * slots * tokens), 0, st, a, slots);
}

template <typename TI, typename TO>
bool launch_append(const AppendArgs &a, cudaStream_t st) {
    // four units a thread once that still leaves a few blocks per SM, one for the few
    // tokens of a decode step (a shorter chain in each thread).  Measured on the device
    // (us, 1 | 4 units), 32 + 2 x 16 heads of 128, FP16: 64 tokens 1.9 | 2.3, 128 2.3 | 2.3,
    // 181 2.5 | 2.6, 256 (2^17 units) 3.3 | 2.7, 512 4.4 | 4.0, 2048 15.1 | 14.3; 24 + 2 x 8 heads
    // of 64, BF16: 409 2.6 | 2.4, 819 (2^17) 3.1 | 2.6, 3276 9.8 | 7.8, 11410 30.9 | 21.5.  From
    // FP32 four are slower again with many tokens of the larger heads (2048 18.4 | 20.0),
    // faster with the smaller (6553 22.0 | 20.3); two would do as well there (18.5, 18.4).
    const long long units = (long long)a.n_tokens * (a.n_q + 2 * a.kv.n_kv) * (a.kv.head_dim / 16);
    return units >= kAppendManyUnits ? launch_units<TI, TO, 4>(a, st) : launch_units<TI, TO, 1>(a, st);
}

template <typename TI>
bool launch_append_to(const AppendArgs &a, int dtype, cudaStream_t st) {
    return dtype == LF_F16 ? launch_append<TI, __half>(a, st) : launch_append<TI, __nv_bfloat16>(a, st);
}

}  // namespace
}  // namespace lf

extern "C" lf_status lf_kv_append_paged(const lf_paged_kv *kv, const void *q_in, const void *k_in, const void *v_in,
                                        int in_dtype, int64_t ld_q, int64_t ld_k, int64_t ld_v, int n_q_heads,
                                        void *q_out, int64_t ld_q_out, const int32_t *seq_device,
                                        const int32_t *pos_device, int n_tokens, const float *rope_device, int rope_len,
                                        uint32_t *err_device, void *cuda_stream) {
    lf::AppendArgs a;
    const lf_status vs = lf::paged_view(kv, &a.kv);
    if (vs != LF_OK) return vs;
    const int bytes = lf::dtype_bytes(in_dtype);
    if (!bytes || n_tokens < 0 || n_q_heads < 0 || n_q_heads > (1 << 16) || kv->n_kv_heads > (1 << 16) || !k_in ||
        !v_in || !pos_device || !err_device || (reinterpret_cast<uintptr_t>(err_device) & 3u) ||
        (reinterpret_cast<uintptr_t>(pos_device) & 3u) || (reinterpret_cast<uintptr_t>(seq_device) & 3u))
        return LF_ERR_INVALID_ARG;
    const int64_t q_row = (int64_t)n_q_heads * kv->head_dim, kv_row = (int64_t)kv->n_kv_heads * kv->head_dim;
    if (ld_k < kv_row || ld_v < kv_row || ld_k * bytes % 16 || ld_v * bytes % 16 || !lf::aligned16(k_in) ||
        !lf::aligned16(v_in))
        return LF_ERR_INVALID_ARG;
    if (n_q_heads > 0 && (!q_in || !q_out || ld_q < q_row || ld_q_out < q_row || ld_q * bytes % 16 ||
                          ld_q_out % 8 || !lf::aligned16(q_in) || !lf::aligned16(q_out)))
        return LF_ERR_INVALID_ARG;
    if (n_q_heads > 0 && q_in == q_out && (in_dtype != kv->dtype || ld_q != ld_q_out)) return LF_ERR_INVALID_ARG;
    if (rope_device && (rope_len < 1 || !lf::aligned16(rope_device))) return LF_ERR_INVALID_ARG;
    if (!seq_device && n_tokens > kv->n_seqs) return LF_ERR_INVALID_ARG;
    if (n_tokens == 0) return LF_OK;
    a.q = q_in;
    a.k = k_in;
    a.v = v_in;
    a.ld_q = ld_q;
    a.ld_k = ld_k;
    a.ld_v = ld_v;
    a.qo = q_out;
    a.ld_qo = ld_q_out;
    a.n_q = n_q_heads;
    a.seq = seq_device;
    a.pos = pos_device;
    a.n_tokens = n_tokens;
    a.rope = rope_device;
    a.rope_len = rope_len;
    a.err = err_device;
    cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
    const bool ok = in_dtype == LF_F32   ? lf::launch_append_to<float>(a, kv->dtype, st)
                    : in_dtype == LF_F16 ? lf::launch_append_to<__half>(a, kv->dtype, st)
                                         : lf::launch_append_to<__nv_bfloat16>(a, kv->dtype, st);
    return ok ? LF_OK : LF_ERR_CUDA;
}
