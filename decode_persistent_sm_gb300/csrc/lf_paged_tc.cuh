// Building blocks of the paged attentions' tcgen05 kernels (private to the library).
#pragma once

#include <cuda.h>

#include <mutex>
#include <type_traits>

#include "lf_paged_attn.h"
#include "lf_tc.cuh"

namespace lf {

constexpr int T_HALF = 128 * 64 * 2;  // one swizzled [128 rows][64 dims] tile: 16 KB

__device__ __forceinline__ void tma_load_4d(void *dst, const CUtensorMap *map, int x, int y, int z, int w,
                                            uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
        "[%6];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_u32(bar))
        : "memory");
}

// max of three (one instruction on sm_100 and later)
__device__ __forceinline__ float max3(float a, float b, float c) {
    float y;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
    return y;
}

// Shared-memory descriptor of an MN-major tile with 128-byte swizzle: 64
// elements of the M/N dimension per 128-byte row, 8 rows (K) to a 1024-byte
// group, groups 1024 bytes apart (stride byte offset), the next 64 elements of
// M/N a whole half tile further (leading byte offset).
__device__ __forceinline__ uint64_t desc_mn_sw128(uint32_t saddr) {
    uint64_t d = smem_desc_sw128(saddr);
    d |= (uint64_t)(T_HALF >> 4) << 16;
    return d;
}

// Instruction descriptor, kind::f16, fp32 accumulators: A K-major, B K-major
// or (b_mn) MN-major, both of type T.
template <typename T>
constexpr uint32_t idesc(int M, int N, bool b_mn) {
    return idesc_f16(M, N) | (std::is_same<T, __nv_bfloat16>::value ? (1u << 7) | (1u << 10) : 0u) |
           (b_mn ? 1u << 16 : 0u);
}

using PagedEncode = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                 const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline PagedEncode paged_encoder() {
    static PagedEncode fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PagedEncode>(p);
    });
    return fn;
}

// The cache as a 4-D tensor (dim, row of the page, KV head, page), boxes of 64
// dims x min(page size, 128) rows, swizzled.
inline bool cache_map(CUtensorMap *map, void *base, const PagedView &kv, int dtype) {
    PagedEncode enc = paged_encoder();
    if (!enc) return false;
    const cuuint64_t ps = 1ull << kv.ps_log2, d = (cuuint64_t)kv.head_dim;
    const cuuint64_t dims[4] = {d, ps, (cuuint64_t)kv.n_kv, (cuuint64_t)kv.n_pages};
    const cuuint64_t str[3] = {d * 2, ps * d * 2, (cuuint64_t)kv.page_stride * 2};
    const cuuint32_t box[4] = {64, (cuuint32_t)min((int)ps, kTcKeys), 1, 1}, one[4] = {1, 1, 1, 1};
    return enc(map, dtype == LF_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, base, dims,
               str, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace lf
