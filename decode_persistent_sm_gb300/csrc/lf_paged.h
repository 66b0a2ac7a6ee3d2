// The paged KV cache as the kernels see it, and the host checks that its
// calls share (private to the library).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "laneformer.h"

namespace lf {

struct PagedView {
    void *k, *v;
    const int32_t *table;
    int n_pages, n_kv, ps_log2, head_dim, n_seqs, max_pages;
    long long page_stride;  // elements
};

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Bytes of one element, 0 for no lf_dtype.
inline int dtype_bytes(int dtype) { return dtype == LF_F32 ? 4 : dtype == LF_F16 || dtype == LF_BF16 ? 2 : 0; }

// Checks the description and fills *out.
inline lf_status paged_view(const lf_paged_kv *kv, PagedView *out) {
    if (!kv || !kv->k || !kv->v || !kv->page_table || !aligned16(kv->k) || !aligned16(kv->v) ||
        (reinterpret_cast<uintptr_t>(kv->page_table) & 3u))
        return LF_ERR_INVALID_ARG;
    if (kv->dtype != LF_F16 && kv->dtype != LF_BF16) return LF_ERR_INVALID_ARG;
    if (kv->n_pages < 1 || kv->n_kv_heads < 1 || kv->n_seqs < 1 || kv->max_pages < 1) return LF_ERR_INVALID_ARG;
    if (kv->page_size < 1 || kv->page_size > 1024 || (kv->page_size & (kv->page_size - 1))) return LF_ERR_INVALID_ARG;
    if (kv->head_dim < 16 || kv->head_dim > 256 || kv->head_dim % 16) return LF_ERR_INVALID_ARG;
    const long long dense = (long long)kv->n_kv_heads * kv->page_size * kv->head_dim;
    if (kv->page_stride != 0 && (kv->page_stride < dense || kv->page_stride % 8)) return LF_ERR_INVALID_ARG;
    // positions are 32-bit, and the last tile may run past the last one (by 4096: 32 TMA boxes)
    if ((long long)kv->max_pages * kv->page_size > 0x7fff0000LL) return LF_ERR_INVALID_ARG;
    int lg = 0;
    while ((1 << lg) < kv->page_size) ++lg;
    *out = PagedView{kv->k,         kv->v,        kv->page_table, kv->n_pages, kv->n_kv_heads, lg, kv->head_dim,
                     kv->n_seqs, kv->max_pages, kv->page_stride ? kv->page_stride : dense};
    return LF_OK;
}

// Programmatic dependent launch.  The kernels of these calls are launched so
// that they may become resident before the stream's previous kernel has
// finished; pdl_wait is the first thing they do, and returns when that kernel's
// results are visible.  What any kernel may have written is therefore read by
// plain loads: a read-only one (__ldg) may be moved above the wait.  pdl_trigger
// lets the next such kernel become resident in turn.  (A kernel launched without
// the attribute still waits for all of this one.)  It hides about 2 us of launch
// latency between these kernels.
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_trigger() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

template <typename... P, typename... A>
inline bool launch_pdl_cluster(void (*kernel)(P...), unsigned cluster, dim3 grid, unsigned threads, size_t smem,
                               cudaStream_t st, const A &...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = cluster;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    if (cudaLaunchKernelEx(&cfg, kernel, args...) != cudaSuccess) {
        (void)cudaGetLastError();
        return false;
    }
    return true;
}
template <typename... P, typename... A>
inline bool launch_pdl(void (*kernel)(P...), dim3 grid, unsigned threads, size_t smem, cudaStream_t st,
                       const A &...args) {
    return launch_pdl_cluster(kernel, 1, grid, threads, smem, st, args...);
}

// Raises a kernel's dynamic shared-memory limit once per device.
template <auto Kernel>
inline bool set_smem_once(int bytes) {
    static std::atomic<uint64_t> done{0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) {
        (void)cudaGetLastError();
        return false;
    }
    const uint64_t bit = 1ull << (dev & 63);
    if (done.load(std::memory_order_acquire) & bit) return true;
    if (cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) {
        (void)cudaGetLastError();
        return false;
    }
    done.fetch_or(bit, std::memory_order_release);
    return true;
}

}  // namespace lf
