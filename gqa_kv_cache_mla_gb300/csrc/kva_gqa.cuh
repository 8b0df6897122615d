// What the attention calls over a paged GQA cache share, whatever the cache
// holds: arguments and their checks, the products of 16 rows, the pieces'
// places in the workspace and their join.
#pragma once

#include "kva_attention.cuh"
#include "kva_split.cuh"

namespace kvw {
namespace {

constexpr int kRows = 16;                   // rows of a row block, at most
// tanh y for u = 2 log2(e) y: the series' coefficients in u^2, and u at y = 1/4
constexpr float kHalfLn2 = 0.5f * kLn2, kTanh3 = kHalfLn2 * kHalfLn2 / 3.0f;
constexpr float kTanh5 = 2.0f / 15.0f * kHalfLn2 * kHalfLn2 * kHalfLn2 * kHalfLn2;
constexpr float kTanh7 = 17.0f / 42.0f * kTanh5 * kHalfLn2 * kHalfLn2, kTanhNear = 0.5f * kLog2e;
constexpr float kMostCap = 0x1p64f;  // a cap above it is none

struct GqaArgs {
    SplitArgs split;
    uint16_t* out;
    float* lse;
    const uint16_t* q;
    int64_t q_stride;
    const uint32_t* page_table;
    const float* slopes;
    uint32_t* err_flags;
    unsigned char* workspace;
    float sm_scale, k_scale, v_scale;
    float softcap, cap_factor, cap_half;  // in units of log2; 2 log2(e) / the cap; half the cap
    uint32_t Hq, G, HB, D;  // query heads, group size, row blocks per group, head size
    uint32_t per_token;     // rows of a token in a row block: G, or all with several blocks
    uint32_t num_pages, max_pages, pieces;
    uint32_t lanes;  // row blocks that CTAs of the same piece take side by side
    FastDiv ps;
    int64_t wait_limit;  // cycles
};

template <int DP>
constexpr uint32_t slot_floats() {
    return kRows * DP + 2 * kRows;
}

template <int DP>
__device__ __forceinline__ float* slot_of(unsigned char* ws, uint32_t c, uint32_t s) {
    return reinterpret_cast<float*>(ws + kMaxPieces * sizeof(OpenPiece)) +
           (uint64_t)(2 * c + s) * slot_floats<DP>();
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4_trans(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

template <bool F16>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
    if constexpr (F16)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
            "{%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
            "{%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Joins a (chunk, row block) that piece blockIdx.x began and others went on
// with: weights 2^(m_i - M) per row, then one weighted sum over the pieces in
// their order, the pieces dealt to groups of threads and the groups' sums
// added up in order.  A long join's rows are dealt to several blocks (one
// context of 7118, E4M3, 5 heads of 256: 26 -> 17 us).
//
// With row blocks of 8 the usual join, of two to four pieces, takes one round
// trip: all that they hold is loaded beside the word that says how many there
// are.  Blocks of 256 threads, all resident at once (256 requests of up to 8192
// over 4 bits 201 -> 197 us, 64 of 4 tokens 113 -> 108).

// BLOCK: rows of a row block.
template <uint32_t BLOCK>
constexpr int join_threads() {
    return BLOCK == kRows ? 512 : 256;
}

template <int DP, uint32_t BLOCK>
__global__ void __launch_bounds__(join_threads<BLOCK>()) gqa_join_kernel(const GqaArgs a) {
    constexpr int kJoinThreads = join_threads<BLOCK>();
    __shared__ float s_w[BLOCK][kMaxPieces];
    __shared__ float s_top[BLOCK], s_sum[BLOCK];
    __shared__ float4 s_acc[kJoinThreads];
    constexpr int kEach = (BLOCK * DP / 4 + kJoinThreads - 1) / kJoinThreads;  // float4 of a thread
    constexpr int kFew = DP <= 128 ? 4 : 2;  // pieces loaded at once
    [[maybe_unused]] float4 x[kEach][kFew];
    [[maybe_unused]] float x_m[kEach][kFew], x_l[kEach][kFew];
    wait_for_stream();
    if constexpr (BLOCK < kRows) {
        if (gridDim.y == 1) {
#pragma unroll
            for (int i = 0; i < kFew; ++i) {
                // (a slot past the last piece's is not looked at in the end)
                const uint32_t c = blockIdx.x + i * a.lanes;
                const float* from = slot_of<DP>(a.workspace, c < kMaxPieces ? c : 0, i == 0);
#pragma unroll
                for (int k = 0; k < kEach; ++k) {
                    const uint32_t e = threadIdx.x + k * kJoinThreads, r = e / (a.D / 4);
                    if (r >= BLOCK) continue;
                    x[k][i] = load_part(from + r * DP + 4 * (e - r * (a.D / 4)));
                    x_m[k][i] = __ldcg(from + kRows * DP + r);
                    x_l[k][i] = __ldcg(from + kRows * DP + kRows + r);
                }
            }
        }
    }
    const OpenPiece open = reinterpret_cast<const OpenPiece*>(a.workspace)[blockIdx.x];
    if (open.n == 0) return;
    const uint32_t c0 = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31u;
    const uint32_t n = open.n, kvh = a.HB == 1 ? open.block : open.block / a.HB;
    const uint32_t hb = open.block - kvh * a.HB;
    const uint32_t in_block = a.G - hb * BLOCK < a.per_token ? a.G - hb * BLOCK : a.per_token;
    // the rows r0 .. r0 + rows - 1 of this block
    const uint32_t every = open.tokens * in_block, share = (every + gridDim.y - 1) / gridDim.y;
    const uint32_t r0 = blockIdx.y * share;
    if (r0 >= every) return;
    const uint32_t rows = every - r0 < share ? every - r0 : share;
    const uint32_t head0 = kvh * a.G + hb * BLOCK;
    auto part = [&](uint32_t i) { return slot_of<DP>(a.workspace, c0 + i * a.lanes, i == 0 ? 1 : 0); };
    if constexpr (BLOCK < kRows) {
        if (n <= kFew && gridDim.y == 1) {
#pragma unroll
            for (int k = 0; k < kEach; ++k) {
                const uint32_t e = tid + k * kJoinThreads, r = e / (a.D / 4);
                const uint32_t d = 4 * (e - r * (a.D / 4));
                if (r >= rows) continue;
                float top = x_m[k][0];
#pragma unroll
                for (int i = 1; i < kFew; ++i)
                    if ((uint32_t)i < n) top = fmaxf(top, x_m[k][i]);
                const float base = top == -INFINITY ? 0.0f : top;
                float l = 0.0f;
                float4 o = make_float4(0, 0, 0, 0);
#pragma unroll
                for (int i = 0; i < kFew; ++i)
                    if ((uint32_t)i < n) {
                        const float f = fast_exp2(x_m[k][i] - base);
                        l += f * x_l[k][i];
                        o.x += f * x[k][i].x;
                        o.y += f * x[k][i].y;
                        o.z += f * x[k][i].z;
                        o.w += f * x[k][i].w;
                    }
                const float inv = l == 0.0f ? 0.0f : a.v_scale / l;
                const uint32_t ct = r / in_block;
                const uint64_t row =
                    (uint64_t)(open.t + ct) * a.Hq + head0 + (r - ct * in_block);
                uint2 y;
                y.x = pack_bf16x2(o.x * inv, o.y * inv);
                y.y = pack_bf16x2(o.z * inv, o.w * inv);
                *reinterpret_cast<uint2*>(a.out + row * a.D + d) = y;
                if (d == 0 && a.lse) a.lse[row] = l == 0.0f ? -INFINITY : (top + log2f(l)) * kLn2;
            }
            return;
        }
    }

    for (uint32_t r = warp; r < rows; r += kJoinThreads / 32) {
        float top = -INFINITY, l_first = 0.0f;  // of the lane's first piece
        if (lane < n) l_first = part(lane)[kRows * DP + kRows + r0 + r];
        for (uint32_t i = lane; i < n; i += 32) {
            const float m = part(i)[kRows * DP + r0 + r];
            s_w[r][i] = m;
            top = fmaxf(top, m);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        const float base = top == -INFINITY ? 0.0f : top;
        float l = 0.0f;
        for (uint32_t i = lane; i < n; i += 32) {
            const float f = fast_exp2(s_w[r][i] - base);
            s_w[r][i] = f;
            l += f * (i == lane ? l_first : part(i)[kRows * DP + kRows + r0 + r]);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
        if (lane == 0) {
            s_top[r] = top;
            s_sum[r] = l;
        }
    }
    __syncthreads();
    const uint32_t quads = a.D / 4, all = rows * quads;
    // `groups` threads share an element; all <= 16 * 64, so at most two rounds
    const uint32_t groups = all >= kJoinThreads ? 1 : kJoinThreads / all;
    for (uint32_t e0 = 0; e0 < all; e0 += kJoinThreads) {
        const uint32_t g = groups == 1 ? 0 : tid / all;
        const uint32_t e = e0 + (groups == 1 ? tid : tid - g * all);
        float4 o = make_float4(0, 0, 0, 0);
        const bool in = e < all && g < groups;
        const uint32_t r = in ? e / quads : 0, d = in ? (e - r * quads) * 4 : 0;
        if (in) {
            constexpr uint32_t kAtOnce = 8;  // loads in flight
            for (uint32_t i0 = g; i0 < n; i0 += kAtOnce * groups) {
                float4 x[kAtOnce];
#pragma unroll
                for (uint32_t k = 0; k < kAtOnce; ++k) {
                    const uint32_t i = i0 + k * groups;
                    if (i < n) x[k] = load_part(part(i) + (r0 + r) * DP + d);
                }
#pragma unroll
                for (uint32_t k = 0; k < kAtOnce; ++k) {
                    const uint32_t i = i0 + k * groups;
                    if (i < n) {
                        const float f = s_w[r][i];
                        o.x += f * x[k].x;
                        o.y += f * x[k].y;
                        o.z += f * x[k].z;
                        o.w += f * x[k].w;
                    }
                }
            }
        }
        if (groups > 1) {
            s_acc[tid] = o;
            __syncthreads();
            if (in && g == 0) {
                for (uint32_t k = 1; k < groups; ++k) {
                    const float4 x = s_acc[tid + k * all];
                    o.x += x.x;
                    o.y += x.y;
                    o.z += x.z;
                    o.w += x.w;
                }
            }
        }
        if (in && g == 0) {
            const uint32_t ct = (r0 + r) / in_block;
            const uint64_t row = (uint64_t)(open.t + ct) * a.Hq + head0 + (r0 + r - ct * in_block);
            const float l = s_sum[r], inv = l == 0.0f ? 0.0f : a.v_scale / l;
            uint2 y;
            y.x = pack_bf16x2(o.x * inv, o.y * inv);
            y.y = pack_bf16x2(o.z * inv, o.w * inv);
            *reinterpret_cast<uint2*>(a.out + row * a.D + d) = y;
            if (d == 0 && a.lse) a.lse[row] = l == 0.0f ? -INFINITY : (s_top[r] + log2f(l)) * kLn2;
        }
    }
}

inline uint32_t padded_head(uint32_t d) { return d <= 64 ? 64 : d <= 128 ? 128 : 256; }

inline int workspace_bytes_for(uint32_t num_q_heads, uint32_t num_kv_heads, uint32_t head_size,
                        uint64_t* bytes) {
    if (!bytes || !num_q_heads || !num_kv_heads || num_q_heads % num_kv_heads) return KVW_EINVAL;
    if (head_size == 0 || head_size % 16 || head_size > 256 || num_q_heads > 4096)
        return KVW_EUNSUPPORTED;
    const uint64_t dp = padded_head(head_size);
    *bytes = kMaxPieces * (sizeof(OpenPiece) + 2 * (kRows * dp + 2 * kRows) * sizeof(float));
    return KVW_OK;
}

// Row blocks that CTAs take side by side: as many as leave less than a 16th of
// the `wave` resident CTAs idle.  Returns the CTAs of the launch.
inline uint32_t side_by_side(GqaArgs& a, uint64_t wave) {
    if (wave > kMaxPieces) wave = kMaxPieces;
    const uint32_t blocks = a.split.blocks;
    a.lanes = blocks;
    while (blocks % a.lanes || wave / a.lanes * a.lanes * 16 < wave * 15) --a.lanes;
    a.split.blocks = blocks / a.lanes;
    a.pieces = (uint32_t)wave / a.lanes;
    return a.pieces * a.lanes;
}

template <int DP, uint32_t BLOCK = kRows>
inline cudaError_t launch_join(const GqaArgs& a, uint32_t ctas, cudaStream_t stream) {
    // where a join may be of more than 48 pieces on average, eight blocks take
    // it (one token over 901 positions: 10.4 us with one, 11.4 with eight)
    const uint32_t y = a.pieces > 48ull * a.split.T * a.split.blocks ? 8 : 1;
    return launch_early(&gqa_join_kernel<DP, BLOCK>, dim3(ctas, y), join_threads<BLOCK>(), 0, stream,
                        a);
}

// Checks a call's arguments (what the cache's type asks of sizes, values and
// strides is given) and fills in all but the scales and the wait limit.  With
// no tokens nothing is filled in.
inline int gqa_arguments(GqaArgs& a, void* out, float* lse, const void* q, int64_t q_row_stride,
                         const uint32_t* input_row_offsets, uint32_t num_batches,
                         uint32_t tot_seq_len, uint32_t num_q_heads,
                         const kvw_paged_cache_t* cache, float sm_scale, float softcap,
                         uint32_t window, const float* alibi_slopes, void* workspace,
                         uint64_t workspace_bytes, uint32_t* err_flags, bool sizes_ok,
                         bool values_ok, bool strides_ok, uint32_t block_rows = kRows) {
    const uint32_t D = cache->head_size, Hk = cache->num_heads;
    uint64_t need = 0;
    const int ws = workspace_bytes_for(num_q_heads, Hk, D, &need);
    if (ws != KVW_OK) return ws;
    if (num_batches > KVW_MAX_BATCHES || tot_seq_len > (1u << 20) || !sizes_ok)
        return KVW_EUNSUPPORTED;
    if (!values_ok) return KVW_EINVAL;
    if (!out || !q || !input_row_offsets || num_batches == 0 || !workspace ||
        workspace_bytes < need)
        return KVW_EINVAL;
    if (!aligned16(out) || !aligned16(q) || !aligned16(workspace) || !aligned4(lse) ||
        !aligned4(input_row_offsets) || !aligned4(alibi_slopes) || !aligned4(err_flags))
        return KVW_EINVAL;
    if (!strides_ok) return KVW_EINVAL;
    if (q_row_stride < (int64_t)num_q_heads * D || q_row_stride % 8) return KVW_EINVAL;
    if (!(sm_scale > 0.0f) || !std::isfinite(sm_scale)) return KVW_EINVAL;
    if (!(softcap >= 0.0f) || !std::isfinite(softcap)) return KVW_EINVAL;
    if (tot_seq_len == 0) return KVW_OK;
    if (softcap > kMostCap) softcap = 0.0f;

    a.split.offsets = input_row_offsets;
    a.split.cache_lengths = cache->cache_lengths;
    a.split.B = num_batches;
    a.split.T = tot_seq_len;
    a.G = num_q_heads / Hk;
    a.HB = (a.G + block_rows - 1) / block_rows;
    a.split.blocks = Hk * a.HB;
    a.per_token = a.HB == 1 ? a.G : block_rows;
    // tokens of a chunk: as many as fit the rows (a power of two), or 8 of 16
    // where that holds the average request's (any number of tokens is right)
    const uint64_t per_request = ((uint64_t)tot_seq_len + num_batches - 1) / num_batches;
    const uint32_t fit = per_request * a.G <= 8 ? 8 : block_rows;
    while (a.HB == 1 && (2u << a.split.log_c) * a.G <= fit) ++a.split.log_c;
    a.split.min_units = 1;
    a.split.overhead = 3;  // a segment's cost beside its tiles, in tiles (1 to 5: within 2 %)
    const uint64_t reach = (uint64_t)cache->max_pages_per_seq * cache->page_size;
    a.split.cap = reach > kMaxReach ? (int64_t)kMaxReach : (int64_t)reach;
    a.split.window = window ? (int64_t)window : 1ll << 40;
    a.out = static_cast<uint16_t*>(out);
    a.lse = lse;
    a.q = static_cast<const uint16_t*>(q);
    a.q_stride = q_row_stride;
    a.page_table = cache->page_table;
    a.slopes = alibi_slopes;
    a.err_flags = err_flags;
    a.workspace = static_cast<unsigned char*>(workspace);
    a.sm_scale = sm_scale;
    a.softcap = softcap * kLog2e;
    a.cap_factor = softcap > 0.0f ? 2.0f * kLog2e / softcap : 0.0f;
    a.cap_half = 0.5f * softcap;
    a.Hq = num_q_heads;
    a.D = D;
    a.num_pages = cache->num_pages;
    a.max_pages = cache->max_pages_per_seq;
    a.ps = make_fast_div(cache->page_size);
    return KVW_OK;
}
}  // namespace
}  // namespace kvw
