// A cache held in 4 bits: checks of its descriptor, and codes to values and back.
#pragma once

#include "kva_common.cuh"

namespace kvw {

constexpr uint32_t kGroup = 64;  // columns that share a scale

inline bool int4_head(uint32_t d) { return d == 64 || d == 96 || d == 128 || d == 256; }

// The descriptors of a cache in 4 bits, for calls that read or write both
// planes.
inline int check_int4(const kvw_paged_cache_t* c, const kva_group_scales_t* s,
                      uint32_t layer_idx) {
    if (!c || !c->data || !c->page_table || !c->cache_lengths || !s || !s->data)
        return KVW_EINVAL;
    if (c->dtype != KVA_DTYPE_INT4) return KVW_EUNSUPPORTED;
    if (!aligned16(c->data) || !aligned16(s->data) || !aligned4(c->page_table) ||
        !aligned4(c->cache_lengths))
        return KVW_EINVAL;
    if (!c->num_pages || !c->page_size || !c->max_pages_per_seq || !c->num_heads ||
        !c->head_size || layer_idx >= c->num_layers)
        return KVW_EINVAL;
    if (!int4_head(c->head_size) || c->page_size % 16) return KVW_EUNSUPPORTED;
    if (c->stride_token != (int64_t)c->head_size) return KVW_EINVAL;
    auto whole = [](int64_t codes, int64_t scales, uint64_t n) {  // multiples of 16 bytes
        return n <= 1 || (codes % 32 == 0 && scales % 8 == 0);
    };
    // the kernels know a row without a page by a place below 0, and the copy engine
    // walks forwards only
    auto rising = [&](int64_t codes, int64_t scales, uint64_t n) {
        return whole(codes, scales, n) && (n <= 1 || (codes > 0 && scales > 0));
    };
    if (!rising(c->stride_page, s->stride_page, c->num_pages) ||
        !rising(c->stride_kv, s->stride_kv, 2) ||
        !whole(c->stride_layer, s->stride_layer, c->num_layers) ||
        !rising(c->stride_head, s->stride_head, c->num_heads))
        return KVW_EINVAL;
    return KVW_OK;
}

inline uint32_t groups_of(uint32_t head_size) { return (head_size + kGroup - 1) / kGroup; }

// First byte of the codes and first scale of a layer's plane.  A stride of a
// dimension of one index is not used.
inline unsigned char* int4_codes(const kvw_paged_cache_t* c, uint32_t layer_idx, uint32_t plane) {
    return static_cast<unsigned char*>(c->data) +
           ((int64_t)layer_idx * (c->num_layers > 1 ? c->stride_layer : 0) +
            (int64_t)plane * c->stride_kv) /
               2;
}
inline uint16_t* int4_scales(const kvw_paged_cache_t* c, const kva_group_scales_t* s,
                             uint32_t layer_idx, uint32_t plane) {
    return static_cast<uint16_t*>(s->data) +
           (int64_t)layer_idx * (c->num_layers > 1 ? s->stride_layer : 0) +
           (int64_t)plane * s->stride_kv;
}

// Scale of a group whose largest |value| has the fp32 pattern `top`.
__device__ __forceinline__ uint16_t group_scale(uint32_t top) {
    if (top >= 0x7f800000u) return 0x7fffu;  // an infinity or a NaN: NaN
    const __nv_bfloat16 s = __float2bfloat16_rn(__fmul_rn(__uint_as_float(top), 1.0f / 7.0f));
    return *reinterpret_cast<const uint16_t*>(&s);
}

// Eight values of a group as codes, the first in the lowest 4 bits.  Between
// 2^-60 and 2^60 the quotient comes from the scale's reciprocal and one
// correction step (div_refined), correctly rounded where it is 2^-14 or more,
// and is below 7.03: the scale is off by 2^-9 of itself at most.
__device__ __forceinline__ uint32_t codes_of(const float (&x)[8], uint16_t scale) {
    const float s = __uint_as_float((uint32_t)scale << 16);
    // 1.5 * 2^23, whose last bit is a unit: added to it, a code is the pattern's end
    constexpr float kMagic = 12582912.0f + 8.0f;
    constexpr uint32_t kPattern = 0x4b400000u;  // of 1.5 * 2^23
    uint32_t word = 0;
    if (refined_ok(s)) {
        const float y = __frcp_rn(s);
        // one shift and add a code; what the patterns begin with adds up to a constant
        uint32_t begin = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float q0 = __fmul_rn(x[i], y);
            const float q = __fmaf_rn(__fmaf_rn(-q0, s, x[i]), y, q0);
            word += __float_as_uint(__fadd_rn(q, kMagic)) << (4 * i);
            begin += kPattern << (4 * i);
        }
        word -= begin;
    } else if (s > 0.0f) {
#pragma unroll 1
        for (int i = 0; i < 8; ++i) {
            float v = x[0];
#pragma unroll
            for (int k = 1; k < 8; ++k) v = i == k ? x[k] : v;
            const float q = fminf(fmaxf(__fdiv_rn(v, s), -7.0f), 7.0f);
            word |= (__float_as_uint(__fadd_rn(q, kMagic)) & 15u) << (4 * i);
        }
    } else {  // 0 or NaN
        word = 0x88888888u;
    }
    return word;
}

}  // namespace kvw
