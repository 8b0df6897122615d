// Tiles of a paged cache by tensor-map copies (TMA), shared by the attention
// kernels of kva.h.
//
// The cache of one layer is a tensor (column, head, row of a page, page,
// plane) under the descriptor's own strides.  One copy takes R rows of one
// head of one page and 128 bytes of their columns into shared memory in
// the 128-byte swizzle (16-byte chunk c of a row lies in place c ^ (line & 7)),
// with columns past the head size filled with zeros.  R is the largest power
// of two up to 64 that divides the page size, so a copy never crosses a page
// and a tile of 64 positions is 64 / R copies for each 128 bytes of columns.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

#include "kva_common.cuh"

namespace kvw {

// cuTensorMapEncodeTiled of the installed driver (looked up once).
inline PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
    static std::atomic<void*> fn{nullptr};
    void* p = fn.load(std::memory_order_acquire);
    if (!p) {
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000,
                                             cudaEnableDefault, &found) != cudaSuccess ||
            found != cudaDriverEntryPointSuccess)
            return nullptr;
        fn.store(p, std::memory_order_release);
    }
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
}

inline uint32_t rows_per_copy(uint32_t page_size) {
    const uint32_t low = page_size & (0u - page_size);
    return low > 64 ? 64 : low;
}

// Strides that a tensor map takes: multiples of 16 bytes (checked by
// check_cache) that are positive and below 2^40 bytes, in every dimension
// with more than one index.
inline bool tma_strides_ok(const kvw_paged_cache_t* c, int planes) {
    const int64_t top = (1ll << 40) / cache_esz(c);
    auto ok = [&](int64_t s, uint64_t n) { return n <= 1 || (s > 0 && s < top); };
    return ok(c->stride_head, c->num_heads) && ok(c->stride_token, c->page_size) &&
           ok(c->stride_page, c->num_pages) && ok(c->stride_kv, (uint64_t)planes);
}

// Map of one layer's planes; 128 bytes of columns per copy, so that a copy of
// any number of rows starts on a 128-byte line of shared memory, as it must.
inline int encode_cache_map(CUtensorMap* map, const kvw_paged_cache_t* c, uint32_t layer_idx,
                            int planes) {
    const auto encode = tensor_map_encoder();
    if (!encode) return KVW_ECUDA;
    const uint64_t esz = cache_esz(c);
    const cuuint64_t dims[5] = {c->head_size, c->num_heads, c->page_size, c->num_pages,
                                (cuuint64_t)planes};
    // a dimension of one index takes any legal stride
    auto bytes = [&](int64_t s, uint64_t n) { return n > 1 ? (cuuint64_t)s * esz : (cuuint64_t)16; };
    const cuuint64_t strides[4] = {bytes(c->stride_head, c->num_heads),
                                   bytes(c->stride_token, c->page_size),
                                   bytes(c->stride_page, c->num_pages),
                                   bytes(c->stride_kv, (uint64_t)planes)};
    const cuuint32_t box[5] = {(cuuint32_t)(128 / esz), 1, rows_per_copy(c->page_size), 1, 1};
    const cuuint32_t ones[5] = {1, 1, 1, 1, 1};
    unsigned char* base = static_cast<unsigned char*>(c->data) +
                          (int64_t)layer_idx * (c->num_layers > 1 ? c->stride_layer : 0) *
                              (int64_t)esz;
    const CUresult r = encode(
        map, esz == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, base,
        dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
        CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? KVW_OK : KVW_EINVAL;
}

// One copy: columns from `col` of R rows from `row` of (page, plane, head).
__device__ __forceinline__ void tma_rows(uint32_t dst, const CUtensorMap* map, uint32_t col,
                                         uint32_t head, uint32_t row, uint32_t page,
                                         uint32_t plane, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], "
        "[%1, {%2, %3, %4, %5, %6}], [%7];"
        ::"r"(dst), "l"(map), "r"(col), "r"(head), "r"(row), "r"(page), "r"(plane), "r"(bar)
        : "memory");
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

// Order this thread's generic accesses to shared memory before later
// accesses of the copy engine or the matrix unit.
__device__ __forceinline__ void fence_async_smem() {
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

}  // namespace kvw
