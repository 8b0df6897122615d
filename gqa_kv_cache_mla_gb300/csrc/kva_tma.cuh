// Tiles of a paged cache by tensor-map copies (TMA), shared by the attention
// kernels of kva.h.
//
// The cache of one layer is a tensor (column, head, row of a page, page,
// plane) under the descriptor's own strides.  One copy takes some rows of one
// head of one page and 128 bytes of their columns into shared memory in the
// 128-byte swizzle (16-byte chunk c of a row lies in place c ^ (line & 7)),
// with columns past the head size filled with zeros.  A copy must not cross a
// page.  With R the largest power of two up to 64 that divides the page size,
// pages cut a tile of 64 positions at multiples of R only, so a tile is made
// of runs of R-row units; a run is copied greedily in pieces of 64, 16, 4 and 1
// units as far as these fit a tile and a page, one map for each piece size (one
// map in all for page sizes whose R is 32 or 64, and for those of 16 up to 48).
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

#include "kva_attention.cuh"

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

// A copy's coordinates (page, row of a page) are signed 32-bit: from 2^31 on it
// would read zeros.
inline bool tma_sizes_ok(const kvw_paged_cache_t* c) {
    return c->num_pages <= (1u << 31) && c->page_size <= (1u << 31);
}

// Maps of one layer's planes, map[i] for copies of R << 2i rows; 128 bytes of
// columns per copy, so that a copy of any number of rows starts on a 128-byte
// line of shared memory, as it must.
struct CacheMaps {
    CUtensorMap map[4];
    uint32_t levels, log_rows;  // maps in use; log2 of R
};

inline int encode_cache_maps(CacheMaps* m, const kvw_paged_cache_t* c, uint32_t layer_idx,
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
    const cuuint32_t ones[5] = {1, 1, 1, 1, 1};
    unsigned char* base = static_cast<unsigned char*>(c->data) +
                          (int64_t)layer_idx * (c->num_layers > 1 ? c->stride_layer : 0) *
                              (int64_t)esz;
    const uint32_t rows = rows_per_copy(c->page_size);
    m->log_rows = 0;
    while ((1u << m->log_rows) < rows) ++m->log_rows;
    m->levels = 0;
    for (uint32_t r = rows; r <= 64 && r <= c->page_size; r *= 4) {
        const cuuint32_t box[5] = {(cuuint32_t)(128 / esz), 1, r, 1, 1};
        if (encode(&m->map[m->levels++],
                   esz == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5,
                   base, dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                   CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return KVW_EINVAL;
    }
    return KVW_OK;
}

// For pages of whole tiles and one head: a map whose copies take 64 rows of
// `panels` neighbouring 128-byte panels of columns at once, each panel as one
// copy of its own would leave it (rows 128 bytes apart, panels 8 KB).  Only
// the columns of whole panels are in it.
inline int encode_panel_map(CUtensorMap* map, const kvw_paged_cache_t* c, uint32_t layer_idx,
                            uint32_t panels) {
    const auto encode = tensor_map_encoder();
    if (!encode) return KVW_ECUDA;
    const uint64_t esz = cache_esz(c);
    const cuuint64_t dims[4] = {128 / esz, c->page_size, c->head_size * esz / 128, c->num_pages};
    const cuuint64_t strides[3] = {
        c->page_size > 1 ? (cuuint64_t)c->stride_token * esz : (cuuint64_t)16, 128,
        c->num_pages > 1 ? (cuuint64_t)c->stride_page * esz : (cuuint64_t)16};
    const cuuint32_t box[4] = {(cuuint32_t)(128 / esz), 64, panels, 1}, ones[4] = {1, 1, 1, 1};
    unsigned char* base = static_cast<unsigned char*>(c->data) +
                          (int64_t)layer_idx * (c->num_layers > 1 ? c->stride_layer : 0) *
                              (int64_t)esz;
    const CUresult r = encode(
        map, esz == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, base,
        dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
        CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? KVW_OK : KVW_EINVAL;
}

__device__ __forceinline__ void tma_4d(uint32_t dst, const CUtensorMap* map, uint32_t c0,
                                       uint32_t c1, uint32_t c2, uint32_t c3, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], "
        "[%1, {%2, %3, %4, %5}], [%6];"
        ::"r"(dst), "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(bar)
        : "memory");
}

// The same columns and rows into L2 only.
__device__ __forceinline__ void tma_4d_prefetch(const CUtensorMap* map, uint32_t c0, uint32_t c1,
                                                uint32_t c2, uint32_t c3) {
    asm volatile("cp.async.bulk.prefetch.tensor.4d.L2.global.tile [%0, {%1, %2, %3, %4}];"
                 ::"l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
                 : "memory");
}

// Does a copy begin at unit x of a run of `run` units, and with which map?
__host__ __device__ __forceinline__ bool copy_begins(uint32_t x, uint32_t run, uint32_t levels,
                                                     uint32_t& level) {
    for (level = levels - 1; level > 0; --level) {
        const uint32_t in = (run >> (2 * level)) << (2 * level);
        if (x < in) return (x & ((1u << (2 * level)) - 1u)) == 0;
        x -= in;
        run -= in;
    }
    return true;
}

// What one lane copies for one unit of a tile.
struct UnitCopy {
    uint32_t page, row, level;  // level 4: nothing
    uint64_t there;             // positions of the tile that the unit holds
    bool bad_page;
};

// Unit c (of 64 >> log_rows) of the tile at position p_tile of request b, for
// positions [start, hi).
__host__ __device__ __forceinline__ UnitCopy plan_unit(const CacheMaps& m,
                                                       const uint32_t* page_table,
                                                       uint32_t max_pages, uint32_t num_pages,
                                                       const FastDiv& ps, uint32_t b,
                                                       int64_t p_tile, int64_t start, int64_t hi,
                                                       uint32_t c) {
    UnitCopy u;
    u.page = u.row = 0;
    u.level = 4;
    u.there = 0;
    u.bad_page = false;
    const int64_t p = p_tile + ((int64_t)c << m.log_rows);
    const int64_t p_end = p + (1ll << m.log_rows);
    if (c >= (64u >> m.log_rows) || p >= hi || p_end <= start) return u;
    const uint32_t idx = fast_div((uint32_t)p, ps);
    u.row = (uint32_t)p - idx * ps.d;
    u.page = KVW_PAGE_UNMAPPED;
    if (idx < max_pages) {
        const uint32_t* id = page_table + (uint64_t)b * max_pages + idx;
#ifdef __CUDA_ARCH__
        u.page = __ldg(id);
#else
        u.page = *id;
#endif
    }
    if (u.page >= num_pages) {
        u.bad_page = true;
        return u;
    }
    const int64_t lo = p > start ? p : start, top = p_end < hi ? p_end : hi;
    const uint32_t len = (uint32_t)(top - lo);
    u.there = (len == 64 ? ~0ull : (1ull << len) - 1) << (uint32_t)(lo - p_tile);
    // the run of units of this page that the tile uses
    const uint32_t u0 = start > p_tile ? (uint32_t)(start - p_tile) >> m.log_rows : 0;
    const uint32_t past = hi - p_tile < 64 ? (uint32_t)(hi - p_tile) : 64u;
    const uint32_t u1 = (past + (1u << m.log_rows) - 1) >> m.log_rows;
    const uint32_t back = u.row >> m.log_rows, ahead = (ps.d - u.row) >> m.log_rows;
    const uint32_t from = c - u0 < back ? u0 : c - back;
    const uint32_t to = u1 - c < ahead ? u1 : c + ahead;
    uint32_t level;
    if (copy_begins(c - from, to - from, m.levels, level)) u.level = level;
    return u;
}

// The same for a tile whose 64 positions all lie in [start, hi), in 32 bits:
// level 4 and no page where the page is not valid or no copy begins.
__host__ __device__ __forceinline__ UnitCopy plan_inner_unit(const CacheMaps& m,
                                                             const uint32_t* page_table,
                                                             uint32_t max_pages,
                                                             uint32_t num_pages,
                                                             const FastDiv& ps, uint32_t b,
                                                             uint32_t p_tile, uint32_t c) {
    UnitCopy u;
    u.level = 4;
    u.there = 0;
    const uint32_t units = 64u >> m.log_rows, p = p_tile + (c << m.log_rows);
    const uint32_t idx = fast_div(p, ps);
    u.row = p - idx * ps.d;
    u.page = KVW_PAGE_UNMAPPED;
    if (c < units && idx < max_pages) {
        const uint32_t* id = page_table + (uint64_t)b * max_pages + idx;
#ifdef __CUDA_ARCH__
        u.page = __ldg(id);
#else
        u.page = *id;
#endif
    }
    u.bad_page = c < units && u.page >= num_pages;
    if (c >= units || u.bad_page) return u;
    const uint32_t back = u.row >> m.log_rows, ahead = (ps.d - u.row) >> m.log_rows;
    const uint32_t from = c < back ? 0 : c - back, to = units - c < ahead ? units : c + ahead;
    uint32_t level;
    if (copy_begins(c - from, to - from, m.levels, level)) u.level = level;
    return u;
}

// What a warp copies for a tile: lane l units l and (of more than 32) l + 32.
struct TilePlan {
    UnitCopy copy[2];
    uint32_t n, t_lo, t_hi;  // units and positions that are there
};

// Sets bad_page where a position of the tile has no valid page.
__device__ __forceinline__ void plan_tile(const CacheMaps& m, const uint32_t* page_table,
                                          uint32_t max_pages, uint32_t num_pages,
                                          const FastDiv& ps, uint32_t b, int64_t p_tile,
                                          int64_t start, int64_t hi, TilePlan& t,
                                          uint32_t& bad_page) {
    const uint32_t lane = threadIdx.x & 31u, units = 64u >> m.log_rows;
    t.copy[1].level = 4;
    if (units <= 32 && start <= p_tile && p_tile + 64 <= hi) {
        // nearly all tiles: a feeding warp's instructions are what small pages
        // cost most (GQA, pages of 16, E4M3, 256 requests: 488 -> 449 us)
        t.copy[0] = plan_inner_unit(m, page_table, max_pages, num_pages, ps, b, (uint32_t)p_tile,
                                    lane);
        if (!__any_sync(0xffffffffu, t.copy[0].bad_page)) {
            t.n = units;
            t.t_lo = t.t_hi = ~0u;
            return;
        }
    }
    uint64_t there = 0;
    t.n = 0;
#pragma unroll 1
    for (uint32_t h = 0; h < 2; ++h) {
        UnitCopy u = plan_unit(m, page_table, max_pages, num_pages, ps, b, p_tile, start, hi,
                               lane + 32u * h);
        if (u.bad_page) bad_page = 1;
        t.n += __popc(__ballot_sync(0xffffffffu, u.there != 0));
        there |= u.there;
        if (h == 0)
            t.copy[0] = u;
        else
            t.copy[1] = u;
        if (units <= 32) break;
    }
    t.t_lo = __reduce_or_sync(0xffffffffu, (uint32_t)there);
    t.t_hi = __reduce_or_sync(0xffffffffu, (uint32_t)(there >> 32));
}

// The page id that plan_unit will look up for unit `lane`, on its way to L1.
__device__ __forceinline__ void prefetch_page(const CacheMaps& m, const uint32_t* page_table,
                                              uint32_t max_pages, const FastDiv& ps, uint32_t b,
                                              int64_t p_tile, uint32_t lane) {
    const uint32_t idx = fast_div((uint32_t)p_tile + (lane << m.log_rows), ps);
    if (lane < (64u >> m.log_rows) && idx < max_pages)
        asm volatile("prefetch.global.L1 [%0];" ::"l"(page_table + (uint64_t)b * max_pages + idx));
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

// The same columns and rows into L2 only.
__device__ __forceinline__ void tma_prefetch(const CUtensorMap* map, uint32_t col, uint32_t head,
                                             uint32_t row, uint32_t page, uint32_t plane) {
    asm volatile("cp.async.bulk.prefetch.tensor.5d.L2.global.tile [%0, {%1, %2, %3, %4, %5}];"
                 ::"l"(map), "r"(col), "r"(head), "r"(row), "r"(page), "r"(plane)
                 : "memory");
}

// The plan of a tile that lies in one page (log_rows 6), the same in all lanes.
struct PagePlan {
    uint32_t row, page;
    bool valid;
    uint64_t there;
};

__host__ __device__ __forceinline__ PagePlan plan_page(const uint32_t* page_table,
                                                       uint32_t max_pages, uint32_t num_pages,
                                                       const FastDiv& ps, uint32_t b,
                                                       uint32_t p_tile, int64_t start,
                                                       int64_t hi) {
    PagePlan t;
    const uint32_t idx = fast_div(p_tile, ps);
    t.page = KVW_PAGE_UNMAPPED;
    if (idx < max_pages) {
        const uint32_t* id = page_table + (uint64_t)b * max_pages + idx;
#ifdef __CUDA_ARCH__
        t.page = __ldg(id);
#else
        t.page = *id;
#endif
    }
    t.row = p_tile - idx * ps.d;
    t.valid = t.page < num_pages;
    const int64_t before = start - p_tile, left = hi - p_tile;
    t.there = t.valid ? ~0ull : 0ull;
    if (left < 64) t.there &= (1ull << (uint32_t)left) - 1;
    // a window past the page table's end begins behind the tile
    if (before > 0) t.there = before < 64 ? t.there & (~0ull << (uint32_t)before) : 0ull;
    return t;
}

// Calls issue(unit, row, page, map) for every copy that the lanes planned,
// every lane its own: the hardware takes them one by one, faster than a loop
// that hands them round to one elected thread (GQA, pages of 16, E4M3: 488 us
// against 513).
template <class Issue>
__device__ __forceinline__ void each_copy(const CacheMaps& m, const TilePlan& t, Issue&& issue) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
        if (t.copy[h].level != 4)
            issue((threadIdx.x & 31u) + 32u * h, t.copy[h].row, t.copy[h].page,
                  &m.map[t.copy[h].level]);
    __syncwarp();
}

// Queries [tokens, heads, width] in bf16: copies of 64 heads x 64 columns,
// heads past the last one filled with zeros.
inline int encode_query_map(CUtensorMap* map, const void* q, uint32_t width, uint32_t heads,
                            uint32_t tokens, int64_t row_stride) {
    const auto encode = tensor_map_encoder();
    if (!encode) return KVW_ECUDA;
    const cuuint64_t dims[3] = {width, heads, tokens};
    const cuuint64_t strides[2] = {(cuuint64_t)width * 2, (cuuint64_t)row_stride * 2};
    const cuuint32_t box[3] = {64, 64, 1}, ones[3] = {1, 1, 1};
    const CUresult r =
        encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(q), dims, strides, box,
               ones, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? KVW_OK : KVW_EINVAL;
}

__device__ __forceinline__ void tma_3d(uint32_t dst, const CUtensorMap* map, uint32_t c0,
                                       uint32_t c1, uint32_t c2, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], "
        "[%1, {%2, %3, %4}], [%5];"
        ::"r"(dst), "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
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
