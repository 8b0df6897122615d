// Rows of a cache held in 4 bits as contiguous bf16 rows: what the attention
// within a chunk of a prompt reads of the positions before it.
//
// Mathematics, per group of 64 columns of a row with scale s and codes u:
// bf16(s * (u - 8)).  A code minus 8 is exact in bf16 (the pattern 0x4300 | u
// is 128 + u), and the product of two bf16 numbers rounded once is what one
// bf16 multiplication gives, so all of it is packed bf16 arithmetic, a pair of
// columns at a time.
//
// Bound: HBM, and of it the writes: 16 bits a value against 4.25 read.
//
// Layout: a warp takes 16 rows of the output (8 of 256-wide heads; of any
// requests) and some of the (plane, head) pairs.  One lane a row finds its
// request, page and place, once for all pairs; the places wait in shared memory,
// as registers they would halve the warps of an SM.  Then a lane takes words of
// 8 codes in row order, so that a load instruction covers whole rows of codes
// (two for heads of 128) and a store 512 contiguous bytes.  The next pair's
// words are loaded before a pair's values are stored.
#include <cstdint>

#include "kva_int4.cuh"

namespace kvw {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

struct GatherArgs {
    uint16_t* out[2];
    int64_t out_stride;
    const unsigned char* codes[2];
    const uint16_t* scales[2];
    int64_t s_page, s_head, sc_page, sc_head;  // bytes of codes, scales
    const uint32_t* offsets;
    const uint32_t* first;
    const uint32_t* page_table;
    uint32_t* err_flags;
    uint32_t B, rows, Hk, num_pages, max_pages;
    uint32_t pairs, chunks, items;  // (plane, head) pairs of an item; items of 16 rows
    uint32_t plane0, planes;        // planes asked for
    FastDiv ps, chunk_div;
};

// Eight codes times the scale (twice in `s2`) as bf16, in order.
__device__ __forceinline__ uint4 values_of(uint32_t word, uint32_t s2) {
    const __nv_bfloat162 scale = *reinterpret_cast<const __nv_bfloat162*>(&s2);
    const __nv_bfloat162 offset = __floats2bfloat162_rn(136.0f, 136.0f);
    uint32_t p[4];  // columns i and i + 4
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t u = ((word >> (4 * i)) & 0x000f000fu) | 0x43004300u;
        const __nv_bfloat162 v =
            __hmul2(__hsub2(*reinterpret_cast<const __nv_bfloat162*>(&u), offset), scale);
        p[i] = *reinterpret_cast<const uint32_t*>(&v);
    }
    return make_uint4(__byte_perm(p[0], p[1], 0x5410), __byte_perm(p[2], p[3], 0x5410),
                      __byte_perm(p[0], p[1], 0x7632), __byte_perm(p[2], p[3], 0x7632));
}

template <int D>
constexpr uint32_t item_rows() {
    return D == 256 ? 8 : 16;
}

// Where a row's codes (bytes) and scales (elements) begin in a plane and head;
// codes below 0: nowhere.
struct __align__(16) RowPlace {
    int64_t codes, scales;
};

// CTAs of an SM: as many as leave the words of two pairs in registers (24 x
// 16 k rows of 8 heads of 128: three CTAs 441 us, two 337; the same of heads of
// 64, pages of 16: two 237, three 182, four 171).
template <int D>
__global__ void __launch_bounds__(kThreads, D == 64 ? 4 : 2) gather_kernel(const GatherArgs a) {
    extern __shared__ uint32_t s_off[];
    constexpr uint32_t R = item_rows<D>(), W = D / 8;  // rows of an item; words of a row
    constexpr int kEach = R * W / 32;                  // words of a lane
    __shared__ RowPlace s_place[kWarps][R];
    const uint32_t lane = threadIdx.x & 31u, warps = gridDim.x * kWarps;
    RowPlace* place = s_place[threadIdx.x >> 5];
    wait_for_stream();
    int ok = 1;
    for (uint32_t i = threadIdx.x; i <= a.B; i += kThreads) {
        const uint32_t o = __ldg(a.offsets + i);
        s_off[i] = o;
        if ((i == 0 && o != 0) || (i == a.B && o != a.rows) ||
            (i < a.B && o > __ldg(a.offsets + i + 1)))
            ok = 0;
    }
    if (!__syncthreads_and(ok)) {
        if (blockIdx.x == 0 && threadIdx.x == 0) flag(a.err_flags, KVW_ERR_OFFSETS);
        return;
    }
    for (uint32_t item = blockIdx.x * kWarps + (threadIdx.x >> 5); item < a.items; item += warps) {
        const uint32_t block = fast_div(item, a.chunk_div), chunk = item - block * a.chunks;
        const uint32_t r0 = block * R;
        // ---- lane i: where row r0 + i is
        if (lane < R) {
            RowPlace x = {-1, 0};
            if (r0 + lane < a.rows) {
                const uint32_t b = find_request(s_off, a.B, r0 + lane);
                const uint64_t pos = (uint64_t)(a.first ? __ldg(a.first + b) : 0u) +
                                     (r0 + lane - s_off[b]);
                if (pos >> 32 == 0) {
                    const uint32_t idx = fast_div((uint32_t)pos, a.ps);
                    const uint32_t row = (uint32_t)pos - idx * a.ps.d;
                    const uint32_t page = idx < a.max_pages
                                              ? __ldg(a.page_table + (uint64_t)b * a.max_pages + idx)
                                              : KVW_PAGE_UNMAPPED;
                    if (page < a.num_pages) {
                        x.codes = (int64_t)page * a.s_page + (int64_t)row * (D / 2);
                        x.scales = (int64_t)page * a.sc_page + row;
                    }
                }
                if (x.codes < 0 && chunk == 0) flag(a.err_flags, KVW_ERR_PAGE);
            }
            place[lane] = x;
        }
        __syncwarp();
        // word k of the lane: word e % W of row r0 + e / W, e = lane + 32 k
        auto load = [&](uint32_t p, uint32_t (&word)[kEach], uint32_t (&scale)[kEach]) {
            const uint32_t second = p >= a.Hk, plane = a.plane0 + second, h = p - second * a.Hk;
            const unsigned char* src = a.codes[plane] + (int64_t)h * a.s_head;
            const uint16_t* sc = a.scales[plane] + (int64_t)h * a.sc_head;
#pragma unroll
            for (int k = 0; k < kEach; ++k) {
                const uint32_t e = lane + 32u * k, r = e / W, w = e - r * W;
                const RowPlace x = place[r];
                word[k] = scale[k] = 0;
                if (x.codes >= 0) {
                    word[k] = __ldcs(reinterpret_cast<const uint32_t*>(src + x.codes + 4 * w));
                    scale[k] = __ldg(sc + x.scales + (int64_t)(w / (kGroup / 8)) * a.ps.d);
                }
            }
        };
        auto store = [&](uint32_t p, const uint32_t (&word)[kEach], const uint32_t (&scale)[kEach]) {
            const uint32_t second = p >= a.Hk, plane = a.plane0 + second, h = p - second * a.Hk;
            uint16_t* dst = a.out[plane] + (int64_t)r0 * a.out_stride + (int64_t)h * D;
#pragma unroll
            for (int k = 0; k < kEach; ++k) {
                const uint32_t e = lane + 32u * k, r = e / W, w = e - r * W;
                if (place[r].codes >= 0)
                    st_stream(reinterpret_cast<uint4*>(dst + (int64_t)r * a.out_stride + 8 * w),
                              values_of(word[k], scale[k] * 0x10001u));
            }
        };
        const uint32_t p1 = min((chunk + 1) * a.pairs, a.planes * a.Hk);
        uint32_t w0[kEach], s0[kEach], w1[kEach], s1[kEach];
        load(chunk * a.pairs, w0, s0);
#pragma unroll 1
        for (uint32_t p = chunk * a.pairs; p < p1; p += 2) {
            if (p + 1 < p1) load(p + 1, w1, s1);
            store(p, w0, s0);
            if (p + 1 < p1) {
                if (p + 2 < p1) load(p + 2, w0, s0);
                store(p + 1, w1, s1);
            }
        }
        __syncwarp();  // the places are read until here
    }
}

template <int D>
cudaError_t launch(GatherArgs& a, cudaStream_t stream) {
    const size_t smem = (a.B + 1ull) * 4;
    uint64_t wave = 0;
    const cudaError_t e = wave_ctas<&gather_kernel<D>>(kThreads, smem, wave);
    if (e != cudaSuccess) return e;
    if (wave == 0) return cudaErrorInvalidConfiguration;
    // Pairs of an item: as many as leave every resident warp four items.
    constexpr uint32_t R = item_rows<D>();
    const uint32_t blocks = (a.rows + R - 1) / R, all = a.planes * a.Hk;
    const uint64_t want = 4 * wave * kWarps;
    uint64_t chunks = (want + blocks - 1) / blocks;
    if (chunks > all) chunks = all;
    a.pairs = (uint32_t)((all + chunks - 1) / chunks);
    a.chunks = (all + a.pairs - 1) / a.pairs;
    a.items = blocks * a.chunks;
    a.chunk_div = make_fast_div(a.chunks);
    uint64_t grid = ((uint64_t)a.items + kWarps - 1) / kWarps;
    if (grid > wave) grid = wave;
    return launch_early(&gather_kernel<D>, dim3((unsigned)grid), kThreads, smem, stream, a);
}

}  // namespace
}  // namespace kvw

extern "C" int kva_gather_kv_int4(void* k_out, void* v_out, int64_t out_row_stride,
                                  const kvw_paged_cache_t* cache,
                                  const kva_group_scales_t* scales, uint32_t layer_idx,
                                  const uint32_t* ctx_offsets, const uint32_t* first_positions,
                                  uint32_t num_batches, uint32_t total_rows, uint32_t* err_flags,
                                  cudaStream_t stream) {
    using namespace kvw;
    const int st = check_int4(cache, scales, layer_idx);
    if (st != KVW_OK) return st;
    if (num_batches > KVW_MAX_BATCHES || total_rows > (1u << 31)) return KVW_EUNSUPPORTED;
    const uint32_t D = cache->head_size, Hk = cache->num_heads;
    if ((uint64_t)Hk * 2 > 4096) return KVW_EUNSUPPORTED;
    if ((!k_out && !v_out) || !ctx_offsets || num_batches == 0) return KVW_EINVAL;
    if (!aligned16(k_out) || !aligned16(v_out) || !aligned4(ctx_offsets) ||
        !aligned4(first_positions) || !aligned4(err_flags))
        return KVW_EINVAL;
    if (out_row_stride < (int64_t)Hk * D || out_row_stride % 8) return KVW_EINVAL;
    if (total_rows == 0) return KVW_OK;

    GatherArgs a = {};
    a.out[0] = static_cast<uint16_t*>(k_out);
    a.out[1] = static_cast<uint16_t*>(v_out);
    a.out_stride = out_row_stride;
    for (uint32_t plane = 0; plane < 2; ++plane) {
        a.codes[plane] = int4_codes(cache, layer_idx, plane);
        a.scales[plane] = int4_scales(cache, scales, layer_idx, plane);
    }
    a.s_page = cache->stride_page / 2;
    a.s_head = cache->stride_head / 2;
    a.sc_page = scales->stride_page;
    a.sc_head = scales->stride_head;
    a.offsets = ctx_offsets;
    a.first = first_positions;
    a.page_table = cache->page_table;
    a.err_flags = err_flags;
    a.B = num_batches;
    a.rows = total_rows;
    a.Hk = Hk;
    a.num_pages = cache->num_pages;
    a.max_pages = cache->max_pages_per_seq;
    a.plane0 = k_out ? 0 : 1;
    a.planes = k_out && v_out ? 2 : 1;
    a.ps = make_fast_div(cache->page_size);
    cudaError_t e;
    switch (D) {
        case 64: e = launch<64>(a, stream); break;
        case 96: e = launch<96>(a, stream); break;
        case 128: e = launch<128>(a, stream); break;
        default: e = launch<256>(a, stream); break;
    }
    return e == cudaSuccess ? KVW_OK : KVW_ECUDA;
}
