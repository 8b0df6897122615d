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

// The value scale of an E4M3 cache (a bf16 cache ignores it).
inline bool value_scale_ok(const kvw_paged_cache_t* c, float v_scale) {
    return c->dtype != KVW_DTYPE_FP8_E4M3 || (v_scale > 0.0f && std::isfinite(v_scale));
}

}  // namespace kvw
