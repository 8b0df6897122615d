// Page tables for a step: the pages that its new tokens need are taken from
// the list of free ones, requests in order, and each new token's slot is
// worked out.
//
// Mathematics: a prefix sum over the requests' counts of further pages gives
// each request its first place in the list.  A further page holds a new token
// in its first row, so the tokens alone write the table: the one in row 0
// enters the page's id.
//
// Bound: latency - launch, lengths, prefix sum, one lookup, one store.  Every
// CTA adds up all requests (at most 8 a thread) instead of passing sums on, and
// takes a token a thread.  Where the count of taken pages is updated in place, it
// may be written only after every CTA has read it: then one cluster of up to 8
// CTAs does it all, whose barrier says when (130 k tokens 17.1 us; on as many
// CTAs as it has tokens for 6.3, the call itself).
#include <cstdint>

#include "kva_common.cuh"

namespace kvw {
namespace {

constexpr int kThreads = 1024;
constexpr uint32_t kMostCtas = 8;  // of a cluster

struct TablesArgs {
    uint32_t* page_table;
    const uint32_t* cache_lengths;
    const uint32_t* offsets;
    const uint32_t* free_pages;
    const uint32_t* taken;
    uint32_t* taken_out;
    int64_t* slot_map;
    uint32_t* err_flags;
    uint32_t B, T, max_pages, num_pages, num_free;
    FastDiv ps;
};

__device__ __forceinline__ void cluster_arrive() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
    __syncwarp();
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// ceil(x / page size), at most `top`; x < 2^33
__device__ __forceinline__ uint32_t pages_for(uint64_t x, const FastDiv& ps, uint32_t top) {
    if (x == 0) return 0;
    const uint64_t last = x - 1;
    const uint64_t n = (last >> 32 ? last / ps.d : fast_div((uint32_t)last, ps)) + 1ull;
    return n < top ? (uint32_t)n : top;
}

// IN_PLACE: taken_out is taken, and the CTAs are one cluster.
template <bool IN_PLACE>
__global__ void __launch_bounds__(kThreads) extend_kernel(const TablesArgs a) {
    extern __shared__ uint32_t dyn[];
    uint32_t* s_off = dyn;                // [B + 1]
    uint32_t* s_len = dyn + a.B + 1;      // [B]
    uint32_t* s_base = dyn + 2 * a.B + 1; // [B] further pages of the requests before
    __shared__ uint64_t s_warp[kThreads / 32];
    const uint32_t tid = threadIdx.x, lane = tid & 31u, warp = tid >> 5;
    wait_for_stream();
    // ---- further pages of each request, and their sums
    const uint32_t per = (a.B + kThreads - 1) / kThreads;
    const uint32_t lo = min(tid * per, a.B), hi = min(lo + per, a.B);
    const uint32_t taken = min(__ldcv(a.taken), a.num_free);
    uint64_t mine = 0;
    int ok = 1;
    for (uint32_t r = lo; r < hi; ++r) {
        const uint32_t o0 = __ldg(a.offsets + r), o1 = __ldg(a.offsets + r + 1);
        const uint32_t len = __ldg(a.cache_lengths + r);
        s_off[r] = o0;
        s_len[r] = len;
        s_base[r] = (uint32_t)mine;
        if (o1 < o0 || o1 > a.T || (r == 0 && o0 != 0) || (r == a.B - 1 && o1 != a.T)) {
            ok = 0;
        } else {
            const uint32_t have = pages_for(len, a.ps, a.max_pages);
            mine += pages_for((uint64_t)len + (o1 - o0), a.ps, a.max_pages) - have;
        }
    }
    if (tid == 0) s_off[a.B] = a.T;
    uint64_t scan = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint64_t v = __shfl_up_sync(0xffffffffu, scan, o);
        if (lane >= (uint32_t)o) scan += v;
    }
    if (lane == 31) s_warp[warp] = scan;
    const bool good = __syncthreads_and(ok);
    if constexpr (IN_PLACE) cluster_arrive();  // this CTA has read `taken`
    if (good) {
        uint64_t before = scan - mine, total = 0;
        for (uint32_t w = 0; w < kThreads / 32; ++w) {
            if (w < warp) before += s_warp[w];
            total += s_warp[w];
        }
        // counts past the list's end are all the same (B + T < 2^33, sums kept
        // to 32 bits by num_free)
        for (uint32_t r = lo; r < hi; ++r) {
            const uint64_t v = before + s_base[r];
            s_base[r] = v < a.num_free ? (uint32_t)v : a.num_free;
        }
        __syncthreads();
        // ---- the tokens
        uint32_t bad = 0;
        for (uint64_t t = blockIdx.x * kThreads + tid; t < a.T; t += gridDim.x * kThreads) {
            const uint32_t b = find_request(s_off, a.B, (uint32_t)t);
            const uint32_t len = s_len[b];
            const uint64_t pos = (uint64_t)len + ((uint32_t)t - s_off[b]);
            uint32_t page = KVW_PAGE_UNMAPPED, row = 0;
            if (pos >> 32 == 0) {
                const uint32_t idx = fast_div((uint32_t)pos, a.ps);
                row = (uint32_t)pos - idx * a.ps.d;
                if (idx < a.max_pages) {
                    uint32_t* entry = a.page_table + (uint64_t)b * a.max_pages + idx;
                    const uint32_t have = pages_for(len, a.ps, a.max_pages);
                    if (idx < have) {
                        page = *entry;
                    } else {
                        const uint64_t at = (uint64_t)taken + s_base[b] + (idx - have);
                        if (at < a.num_free) page = __ldg(a.free_pages + at);
                    }
                    if (page >= a.num_pages) page = KVW_PAGE_UNMAPPED;
                    if (idx >= have && row == 0) *entry = page;
                }
            }
            if (page == KVW_PAGE_UNMAPPED) bad = KVW_ERR_PAGE;
            if (a.slot_map)
                a.slot_map[t] = page == KVW_PAGE_UNMAPPED
                                    ? -1
                                    : (int64_t)((uint64_t)page * a.ps.d + row);
        }
        if (bad) flag(a.err_flags, bad);
        if constexpr (IN_PLACE) cluster_wait();
        if (blockIdx.x == 0 && tid == 0) {
            const uint64_t all = taken + total;
            *a.taken_out = all < a.num_free ? (uint32_t)all : a.num_free;
        }
    } else {
        if (blockIdx.x == 0 && tid == 0) flag(a.err_flags, KVW_ERR_OFFSETS);
        if constexpr (IN_PLACE) cluster_wait();
    }
}

template <bool IN_PLACE>
cudaError_t launch(const TablesArgs& a, cudaStream_t stream) {
    const size_t smem = (3ull * a.B + 1) * 4;
    cudaError_t e = prepare_smem<&extend_kernel<IN_PLACE>>(smem);
    if (e != cudaSuccess) return e;
    uint32_t most = kMostCtas, ctas = 1;
    if constexpr (!IN_PLACE) {
        int sms = 0;
        if ((e = sm_count(sms)) != cudaSuccess) return e;
        most = (uint32_t)sms;
    }
    const uint32_t want = (a.T - 1) / kThreads + 1;
    if constexpr (IN_PLACE)
        while (ctas < most && ctas < want) ctas *= 2;
    else
        ctas = want < most ? want : most;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = ctas;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = at;
    cfg.numAttrs = IN_PLACE ? 2 : 1;
    e = cudaLaunchKernelEx(&cfg, &extend_kernel<IN_PLACE>, a);
    if (e != cudaSuccess) cudaGetLastError();  // reported here, not by the caller's next call
    return e;
}

}  // namespace
}  // namespace kvw

extern "C" int kva_extend_page_tables(uint32_t* page_table, uint32_t max_pages_per_seq,
                                      const uint32_t* cache_lengths,
                                      const uint32_t* input_row_offsets, uint32_t num_batches,
                                      uint32_t tot_seq_len, uint32_t page_size,
                                      uint32_t num_pages, const uint32_t* free_pages,
                                      uint32_t num_free, const uint32_t* taken,
                                      uint32_t* taken_out, int64_t* slot_map, uint32_t* err_flags,
                                      cudaStream_t stream) {
    using namespace kvw;
    if (num_batches > KVW_MAX_BATCHES || tot_seq_len > (1u << 31)) return KVW_EUNSUPPORTED;
    if (!page_table || !cache_lengths || !input_row_offsets || !taken || !taken_out ||
        (num_free && !free_pages) || num_batches == 0 || max_pages_per_seq == 0 ||
        page_size == 0 || num_pages == 0)
        return KVW_EINVAL;
    if (!aligned4(page_table) || !aligned4(cache_lengths) || !aligned4(input_row_offsets) ||
        !aligned4(free_pages) || !aligned4(taken) || !aligned4(taken_out) ||
        (reinterpret_cast<uintptr_t>(slot_map) & 7u) || !aligned4(err_flags))
        return KVW_EINVAL;
    if (tot_seq_len == 0) return KVW_OK;
    TablesArgs a = {};
    a.page_table = page_table;
    a.cache_lengths = cache_lengths;
    a.offsets = input_row_offsets;
    a.free_pages = free_pages;
    a.taken = taken;
    a.taken_out = taken_out;
    a.slot_map = slot_map;
    a.err_flags = err_flags;
    a.B = num_batches;
    a.T = tot_seq_len;
    a.max_pages = max_pages_per_seq;
    a.num_pages = num_pages;
    a.num_free = num_free;
    a.ps = make_fast_div(page_size);
    const cudaError_t e = taken == taken_out ? launch<true>(a, stream) : launch<false>(a, stream);
    return e == cudaSuccess ? KVW_OK : KVW_ECUDA;
}
