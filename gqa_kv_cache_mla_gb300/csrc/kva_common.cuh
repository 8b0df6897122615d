// Host-side argument checks shared by the calls of kva.h.
#pragma once

#include <cmath>

#include "kva.h"
#include "kvw_device.cuh"

namespace kvw {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

inline uint32_t cache_esz(const kvw_paged_cache_t* c) {
    return c->dtype == KVW_DTYPE_FP8_E4M3 ? 1u : 2u;
}

// The descriptor's type, pointers, sizes and strides, for a call that reads
// or writes `planes` planes (K; K and V) in 16-byte vectors.
inline int check_cache(const kvw_paged_cache_t* c, uint32_t layer_idx, int planes) {
    if (!c || !c->data || !c->page_table || !c->cache_lengths) return KVW_EINVAL;
    if (c->dtype != KVW_DTYPE_BF16 && c->dtype != KVW_DTYPE_FP8_E4M3) return KVW_EUNSUPPORTED;
    if (c->dtype == KVW_DTYPE_FP8_E4M3 && !(c->scale > 0.0f && std::isfinite(c->scale)))
        return KVW_EINVAL;
    if (!aligned16(c->data) || !aligned4(c->page_table) || !aligned4(c->cache_lengths))
        return KVW_EINVAL;
    if (!c->num_pages || !c->page_size || !c->max_pages_per_seq || !c->num_heads ||
        !c->head_size || layer_idx >= c->num_layers)
        return KVW_EINVAL;
    const int64_t per16 = 16 / (int64_t)cache_esz(c);
    if (c->stride_page % per16 || c->stride_token % per16 ||
        (c->num_layers > 1 && c->stride_layer % per16) ||
        (c->num_heads > 1 && c->stride_head % per16) || (planes > 1 && c->stride_kv % per16))
        return KVW_EINVAL;
    return KVW_OK;
}

// Launches a kernel that may be scheduled before the one before it in the
// stream has ended; it calls wait_for_stream before it touches global memory.
template <class... P, class... A>
inline cudaError_t launch_early(void (*kernel)(P...), dim3 grid, int threads, size_t smem,
                                cudaStream_t stream, const A&... args) {
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
    if (e != cudaSuccess) cudaGetLastError();  // reported here, not by the caller's next call
    return e;
}

// Until what came before this kernel in the stream has ended and is visible.
__device__ __forceinline__ void wait_for_stream() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

// The value scale of an E4M3 cache (a bf16 cache ignores it).
inline bool value_scale_ok(const kvw_paged_cache_t* c, float v_scale) {
    return c->dtype != KVW_DTYPE_FP8_E4M3 || (v_scale > 0.0f && std::isfinite(v_scale));
}

}  // namespace kvw
