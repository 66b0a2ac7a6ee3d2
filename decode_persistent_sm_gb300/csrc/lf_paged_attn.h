// What the kernels of the paged attention share (private to the library).
#pragma once

#include "lf_paged.h"

namespace lf {

constexpr float kLog2e = 1.4426950408889634f;

struct AttnArgs {
    PagedView kv;
    const void *q;
    void *out;
    float *lse;
    long long ld_q, ld_out;
    int n_q, group;  // query heads, query heads per KV head
    const int32_t *lens;
    int max_len, shared, window;
    float scale_log2;  // scale * log2 e
    // common items: rows_c rows of a KV head (row = sequence * group + head), row_tiles of them, items_c = n_kv * row_tiles
    // items, tiles of keys_c keys,
    // shares of the first grid_c CTAs; page_align: 1, or the page size when the common range is cut to whole pages
    int rows_c, row_tiles, items_c, keys_c, grid_c, page_align;
    bool tc;           // the common items run in paged_attn_tc_kernel, not in the list below
    int grid;          // CTAs that share the list
    // workspace
    int *plan;         // the common range [lo, hi)
    int2 *span;        // first and last CTA of each item: common items [n_kv][row_tiles], then own ones [n_seqs][n_kv]
    // partials, common items' slots first: slots_c = n_kv * row_tiles + grid_c of rows_c rows, then n_seqs * n_kv + grid
    // of `group` rows
    int slots_c;
    float *part_o;     // [row][head_dim], unnormalised
    float2 *part_ml;   // [row] (max in the log2 domain, sum)
    uint32_t *err;
};


// What one sequence sees.
struct Span {
    int lo, len;   // positions [lo, len)
    bool member;   // shares the common range
};
__device__ __forceinline__ Span span_of(const AttnArgs &a, int b) {
    Span s;
    s.len = a.lens[b];
    if (s.len < 0 || s.len > a.max_len) s.len = 0;
    s.lo = a.window > 0 ? max(0, s.len - a.window) : 0;
    s.member = s.len >= a.shared && s.lo < a.shared;
    return s;
}
// The common range [lo, hi) for the latest window start among the sharing
// sequences (-1: there is none), whole pages only where page_align says so.
struct Common {
    int lo, hi;
    __device__ Common(const AttnArgs &a, int latest) {
        hi = a.shared & ~(a.page_align - 1);
        lo = (latest + a.page_align - 1) & ~(a.page_align - 1);
        if (latest < 0 || lo >= hi) lo = hi = a.shared;  // nothing in common
    }
};
// This lane's part of the latest window start (a warp takes the maximum).
__device__ __forceinline__ int latest_start(const AttnArgs &a, int lane) {
    int lo = -1;
    for (int b = lane; b < a.kv.n_seqs; b += 32) {
        const Span s = span_of(a, b);
        if (s.member) lo = max(lo, s.lo);
    }
    return lo;
}
// Positions of the sequence outside the common range.
__device__ __forceinline__ int own_count(const Span &s, const Common &c) {
    return s.member ? max(0, c.lo - s.lo) + (s.len - c.hi) : s.len - s.lo;
}

// u / d for u >= 0, d > 0.  The compiler's integer division is a call of some
// hundred cycles, which the start of a short kernel feels; below 2^20 a
// reciprocal is off by less than one.
__device__ __forceinline__ int quotient(int u, int d) {
    if (u >= 1 << 20) return u / d;
    int q = (int)((float)u * __fdividef(1.f, (float)d));
    const int r = u - q * d;
    q += (r >= d) - (r < 0);
    return q;
}

// The list's shares: the first total % ctas CTAs take one tile more.  No share
// is empty (a list shorter than the grid goes to its first tiles' CTAs).
struct Shares {
    int q, r;
    __device__ Shares(int total, int grid) {
        q = total < grid ? 1 : quotient(total, grid);
        r = total < grid ? 0 : total - q * grid;
    }
    __device__ int begin(int c) const { return c * q + min(c, r); }
};

template <typename T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The common items on the 5th-generation tensor cores (lf_paged_attn_tc.cu).
constexpr int kTcRows = 256, kTcKeys = 128;
lf_status paged_attn_tc(const AttnArgs &a, int dtype, cudaStream_t st);

}  // namespace lf
