// Appending keys and values to the paged cache: split of the fused QKV
// projection, per-head RMSNorm of queries and keys (optional), rotation, and
// the store of queries to their buffer and of keys and values to their cache
// slots (bf16, or E4M3 with a static scale).
//
// Mathematics, per head x of head_size values: y = x * rsqrt(mean(x^2) + eps)
// * (gamma + offset); then each pair (a, b) of the first rope_dim columns
// becomes (a c - b s, a s + b c) with the (c, s) of the token's position.  All
// of it in fp32 between one widening and one rounding.
//
// Bound: HBM streaming (every projected value is read once and written once,
// under two flops per byte).  A small batch is bound by latency instead: two
// dependent round trips (offsets and lengths; then page id and angles), which
// the head rows' own loads overlap because they need neither.
//
// Layout: a team of TL lanes owns a head row, TL the power of two that covers
// head_size / 16; each lane holds the two 16-byte vectors whose elements form
// pairs with each other (vectors j and j + rope_dim/16 half-split, 2j and
// 2j + 1 interleaved; past the rotated columns two neighbours), so a pair
// never crosses lanes, the norm is one TL-wide butterfly, and in either
// pairing lane j needs the 16 angle values [16 j, 16 j + 16): four float4,
// kept in registers for all the head rows of its token.  A warp takes items
// of one token and `passes` passes of 32 / TL rows; the rows' vectors are
// loaded two passes ahead of their use.  CTAs are persistent and stage the
// ragged tables once.
//
// Measured, 32 ragged requests of up to 2048 new tokens, 32 + 2 x 8 heads of
// 128 (780 MB): 127 us, 6.1 TB/s, 90 % of the card's copy rate.  Three CTAs
// per SM (80 registers, a few scalars spilled) against two and four (64
// registers): bf16 130, 131, 138 us; E4M3 133, 151, 129 us; with norms 133,
// 142, 190 us.  One pass ahead instead of two: 134, 140 and 136 us; the next
// item's first rows loaded before an item ends: 143, 154, 146 us (spills).  A
// cache in 4 bits (683 MB) has more to compute between load and store: four CTAs
// and one pass ahead 121 us, 84 % of the copy rate (half-split 132, with norms
// 160; 64 registers, 64 to 68 bytes a thread spilled); five CTAs 138 (146, 196),
// three 134 (140, 157), three and two passes ahead 153, two and two 138.  One
// token: 2.3 us on the device.  With few rows a token (4 + 2 x 1 heads of 96) the
// lookups of a token are most of its work: 46 k tokens 58 us, a quarter of the
// copy rate.
#include <cstdint>

#include "kva_common.cuh"
#include "kva_int4.cuh"

namespace kvw {
namespace {

enum class Held { kBf16, kE4m3, kInt4 };

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

struct AppendArgs {
    uint16_t* q_out;
    const uint16_t* qkv;
    int64_t q_out_stride, qkv_stride;
    const uint32_t* offsets;
    const uint32_t* cache_lengths;
    const uint32_t* page_table;
    const uint16_t* q_gamma;
    const uint16_t* k_gamma;
    const float* freqs;
    const uint32_t* position_ids;
    uint32_t* err_flags;
    unsigned char* k_base;  // K plane of the layer
    unsigned char* v_base;
    int64_t s_page, s_token, s_head;  // elements (of 4 bits: bytes)
    uint16_t* k_scales;               // of a cache in 4 bits, as are the strides
    uint16_t* v_scales;
    int64_t sc_page, sc_head;
    float eps, weight_offset, k_scale, v_scale, inv_d;
    uint32_t B, T, Hq, Hk, D, rope, freqs_rows, num_pages, max_pages;
    uint32_t rows, passes, chunks, items;  // head rows per token; passes per item; items per token
    uint32_t sec0, sec01;                  // mrope section ends, in pairs
    FastDiv ps, chunk_div;
};

// The fp32 pattern of the largest |value| of eight (a NaN's above all).
__device__ __forceinline__ uint32_t top_of(const float (&x)[8]) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(x[i]) & 0x7fffffffu);
    return m;
}

template <int TL, bool INTERLEAVED, Held HELD, bool MROPE>
__global__ void __launch_bounds__(kThreads, HELD == Held::kInt4 ? 4 : 3) append_kernel(const AppendArgs a) {
    extern __shared__ uint32_t s_tables[];
    uint32_t* s_off = s_tables;
    uint32_t* s_clen = s_tables + a.B + 1;
    constexpr uint32_t kTeams = 32 / TL;
    constexpr int kAhead = HELD == Held::kInt4 ? 1 : 2;
    const uint32_t lane = threadIdx.x & 31u, team = lane / TL, j = lane % TL;
    const uint32_t half = a.rope / 16;  // lanes whose pairs turn
    const bool active = j < a.D / 16;
    const bool turns = j < half;
    // element offsets of the lane's two vectors in a head row
    const uint32_t e0 = INTERLEAVED || !turns ? 16u * j : 8u * j;
    const uint32_t e1 = INTERLEAVED || !turns ? e0 + 8u : e0 + a.rope / 2;
    const uint32_t warps = gridDim.x * kWarps;
    uint32_t item = blockIdx.x * kWarps + (threadIdx.x >> 5);

    uint4 buf[kAhead][2];
    auto fetch = [&](uint32_t it, uint32_t pass, uint4 (&v)[2]) {
        const uint32_t t = fast_div(it, a.chunk_div);
        const uint32_t row = ((it - t * a.chunks) * a.passes + pass) * kTeams + team;
        if (active && row < a.rows) {
            const uint16_t* p = a.qkv + (int64_t)t * a.qkv_stride + (int64_t)row * a.D;
            v[0] = ld_stream(reinterpret_cast<const uint4*>(p + e0));
            v[1] = ld_stream(reinterpret_cast<const uint4*>(p + e1));
        } else {
            v[0] = v[1] = make_uint4(0, 0, 0, 0);
        }
    };
    wait_for_stream();
    RaggedLoads ragged;
    ragged.issue(a.offsets, a.cache_lengths, a.B);
    if (item < a.items) {
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
            if ((uint32_t)k < a.passes) fetch(item, k, buf[k]);
    }
    if (!ragged.commit(a.offsets, a.cache_lengths, a.B, a.T, s_off, s_clen)) {
        if (blockIdx.x == 0 && threadIdx.x == 0) flag(a.err_flags, KVW_ERR_OFFSETS);
        return;
    }

    bool first = true;
    for (; item < a.items; item += warps) {
        const uint32_t t = fast_div(item, a.chunk_div);
        const uint32_t chunk = item - t * a.chunks;
        if (!first) {
#pragma unroll
            for (int k = 0; k < kAhead; ++k)
                if ((uint32_t)k < a.passes) fetch(item, k, buf[k]);
        }
        first = false;
        const uint32_t b = find_request(s_off, a.B, t);
        const uint64_t pos = (uint64_t)s_clen[b] + (t - s_off[b]);
        // does the item hold key or value rows?
        const bool stores_kv = ((chunk + 1) * a.passes) * kTeams > a.Hq;
        const int64_t slot = stores_kv ? slot_row(a.page_table, a.max_pages, a.num_pages, a.ps,
                                                  a.s_page, a.s_token, 0, b, pos)
                                       : -1;
        [[maybe_unused]] int64_t scale_slot = 0;
        if constexpr (HELD == Held::kInt4) {
            // the page and the row once more, from what slot_row has looked up
            if (slot >= 0) {
                const uint32_t idx = fast_div((uint32_t)pos, a.ps);
                scale_slot = (int64_t)__ldg(a.page_table + (uint64_t)b * a.max_pages + idx) *
                                 a.sc_page +
                             ((uint32_t)pos - idx * a.ps.d);
            }
        }
        float cs[16];
        bool position_ok = true;
        if (a.rope) {
            if constexpr (MROPE) {
                const uint32_t p0 = __ldg(a.position_ids + t);
                const uint32_t p1 = __ldg(a.position_ids + (uint64_t)a.T + t);
                const uint32_t p2 = __ldg(a.position_ids + 2ull * a.T + t);
                // rows of empty sections are never read
                position_ok = (a.sec0 == 0 || p0 < a.freqs_rows) &&
                              (a.sec01 == a.sec0 || p1 < a.freqs_rows) &&
                              (a.sec01 == a.rope / 2 || p2 < a.freqs_rows);
                if (turns && position_ok) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const uint32_t pair = 8u * j + i;
                        const uint32_t p = pair < a.sec0 ? p0 : pair < a.sec01 ? p1 : p2;
                        const float2 f = __ldg(reinterpret_cast<const float2*>(
                            a.freqs + (uint64_t)p * a.rope + 2u * pair));
                        cs[2 * i] = f.x;
                        cs[2 * i + 1] = f.y;
                    }
                }
            } else {
                const uint64_t p = a.position_ids ? __ldg(a.position_ids + t) : pos;
                position_ok = p < a.freqs_rows;
                if (turns && position_ok) {
                    const float4* f = reinterpret_cast<const float4*>(a.freqs + p * a.rope + 16u * j);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float4 v = ld_table(f + i);
                        cs[4 * i] = v.x;
                        cs[4 * i + 1] = v.y;
                        cs[4 * i + 2] = v.z;
                        cs[4 * i + 3] = v.w;
                    }
                }
            }
        }
        if (lane == 0) {
            const uint32_t bad = (position_ok ? 0u : (uint32_t)KVW_ERR_POSITION) |
                                 (stores_kv && position_ok && slot < 0 ? (uint32_t)KVW_ERR_PAGE : 0u);
            if (bad) flag(a.err_flags, bad);
        }
        if (!position_ok) continue;

        for (uint32_t pass0 = 0; pass0 < a.passes; pass0 += kAhead) {
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const uint32_t pass = pass0 + k;
                if (pass >= a.passes) break;
                const uint32_t row = (chunk * a.passes + pass) * kTeams + team;
                float x0[8], x1[8];
                unpack8(buf[k][0], x0);
                unpack8(buf[k][1], x1);
                if (pass + kAhead < a.passes) fetch(item, pass + kAhead, buf[k]);
                const bool is_q = row < a.Hq, is_v = row >= a.Hq + a.Hk;
                if (a.q_gamma || a.k_gamma) {  // uniform: the butterfly takes all lanes
                    float ss = 0.0f;
#pragma unroll
                    for (int i = 0; i < 8; ++i) ss = fmaf(x0[i], x0[i], fmaf(x1[i], x1[i], ss));
#pragma unroll
                    for (int o = TL / 2; o > 0; o >>= 1)
                        ss += __shfl_xor_sync(0xffffffffu, ss, o);
                    const uint16_t* g = is_v ? nullptr : is_q ? a.q_gamma : a.k_gamma;
                    if (g && active && row < a.rows) {
                        const float r = __fdiv_rn(1.0f, __fsqrt_rn(fmaf(ss, a.inv_d, a.eps)));
                        float g0[8], g1[8];
                        unpack8(ld_table(reinterpret_cast<const uint4*>(g + e0)), g0);
                        unpack8(ld_table(reinterpret_cast<const uint4*>(g + e1)), g1);
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            x0[i] = x0[i] * r * (g0[i] + a.weight_offset);
                            x1[i] = x1[i] * r * (g1[i] + a.weight_offset);
                        }
                    }
                }
                if (turns && !is_v) {
                    if constexpr (INTERLEAVED) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            rope_pair(x0[2 * i], x0[2 * i + 1], cs[2 * i], cs[2 * i + 1], x0[2 * i],
                                      x0[2 * i + 1]);
                            rope_pair(x1[2 * i], x1[2 * i + 1], cs[8 + 2 * i], cs[9 + 2 * i],
                                      x1[2 * i], x1[2 * i + 1]);
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            float y0, y1;
                            rope_pair(x0[i], x1[i], cs[2 * i], cs[2 * i + 1], y0, y1);
                            x0[i] = y0;
                            x1[i] = y1;
                        }
                    }
                }
                [[maybe_unused]] uint32_t tops[TL < 8 ? 2 : 4];  // of the row's groups
                if constexpr (HELD == Held::kInt4) {
                    // uniform: some row of the pass is a key or a value
                    if ((chunk * a.passes + pass + 1) * kTeams > a.Hq) {
                        const uint32_t t0 = top_of(x0), t1 = top_of(x1);
#pragma unroll
                        for (uint32_t g = 0; g < sizeof(tops) / 4; ++g) {
                            if (g * kGroup >= a.D) break;
                            uint32_t m = max(e0 / kGroup == g ? t0 : 0u, e1 / kGroup == g ? t1 : 0u);
#pragma unroll
                            for (int o = TL / 2; o > 0; o >>= 1)
                                m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
                            tops[g] = m;
                        }
                    }
                }
                if (!active || row >= a.rows) continue;
                if (is_q) {
                    uint16_t* p = a.q_out + (int64_t)t * a.q_out_stride + (int64_t)row * a.D;
                    st_stream(reinterpret_cast<uint4*>(p + e0), pack8_bf16(x0));
                    st_stream(reinterpret_cast<uint4*>(p + e1), pack8_bf16(x1));
                } else if (slot >= 0 && HELD == Held::kInt4) {
                    const uint32_t h = row - a.Hq - (is_v ? a.Hk : 0u);
                    uint16_t sc0 = 0, sc1 = 0;
#pragma unroll
                    for (uint32_t g = 0; g < sizeof(tops) / 4; ++g) {
                        if (g * kGroup >= a.D) break;
                        const uint16_t sc = group_scale(tops[g]);
                        if (e0 / kGroup == g) sc0 = sc;
                        if (e1 / kGroup == g) sc1 = sc;
                        if (j == g)
                            (is_v ? a.v_scales : a.k_scales)[scale_slot + (int64_t)h * a.sc_head +
                                                             (int64_t)g * a.ps.d] = sc;
                    }
                    unsigned char* p = (is_v ? a.v_base : a.k_base) + slot + (int64_t)h * a.s_head;
                    *reinterpret_cast<uint32_t*>(p + e0 / 2) = codes_of(x0, sc0);
                    *reinterpret_cast<uint32_t*>(p + e1 / 2) = codes_of(x1, sc1);
                } else if (slot >= 0) {
                    constexpr bool FP8 = HELD == Held::kE4m3;
                    constexpr int esz = FP8 ? 1 : 2;
                    const uint32_t h = row - a.Hq - (is_v ? a.Hk : 0u);
                    unsigned char* p =
                        (is_v ? a.v_base : a.k_base) + (slot + (int64_t)h * a.s_head) * esz;
                    const float sc = is_v ? a.v_scale : a.k_scale;
                    store_k8<FP8>(p + e0 * esz, x0, sc);
                    store_k8<FP8>(p + e1 * esz, x1, sc);
                }
            }
        }
    }
}

template <int TL, bool IL, Held HELD, bool MROPE>
cudaError_t launch(AppendArgs& a, cudaStream_t stream) {
    const size_t smem = (2ull * a.B + 1) * 4;
    uint64_t wave = 0;
    cudaError_t e = wave_ctas<&append_kernel<TL, IL, HELD, MROPE>>(kThreads, smem, wave);
    if (e != cudaSuccess) return e;
    if (wave == 0) return cudaErrorInvalidConfiguration;
    // Passes per item: as many as leave every resident warp two items (angles
    // and lookups are paid once per item), down to one for small batches.
    const uint32_t all = (a.rows + 32 / TL - 1) / (32 / TL);
    const uint64_t want = 2 * wave * kWarps;
    uint64_t chunks = (want + a.T - 1) / a.T;
    if (chunks > all) chunks = all;
    a.passes = (uint32_t)((all + chunks - 1) / chunks);
    a.chunks = (all + a.passes - 1) / a.passes;
    a.items = a.T * a.chunks;
    a.chunk_div = make_fast_div(a.chunks);
    uint64_t grid = ((uint64_t)a.items + kWarps - 1) / kWarps;
    if (grid > wave) grid = wave;
    return launch_early(&append_kernel<TL, IL, HELD, MROPE>, dim3((unsigned)grid), kThreads, smem,
                        stream, a);
}

template <int TL, bool IL, Held HELD>
cudaError_t pick(AppendArgs& a, bool mrope, cudaStream_t s) {
    return mrope ? launch<TL, IL, HELD, true>(a, s) : launch<TL, IL, HELD, false>(a, s);
}

template <int TL, bool IL>
cudaError_t pick(AppendArgs& a, Held held, bool mrope, cudaStream_t s) {
    switch (held) {
        case Held::kBf16: return pick<TL, IL, Held::kBf16>(a, mrope, s);
        case Held::kE4m3: return pick<TL, IL, Held::kE4m3>(a, mrope, s);
        default:
            if constexpr (TL < 32) return pick<TL, IL, Held::kInt4>(a, mrope, s);
            return cudaErrorInvalidValue;  // heads of 4 bits have 256 columns at most
    }
}

// Checks the arguments that all kinds of cache share and launches; `a` holds
// where the cache's values (and scales) go.
int append(AppendArgs& a, Held held, bool values_ok, void* q_out, int64_t q_out_row_stride,
           const void* qkv, int64_t qkv_row_stride, const uint32_t* input_row_offsets,
           uint32_t num_batches, uint32_t tot_seq_len, uint32_t num_q_heads, const void* q_gamma,
           const void* k_gamma, float epsilon, float weight_offset, const void* freqs_cis,
           uint32_t freqs_rows, uint32_t rope_dim, const uint32_t* position_ids, int interleaved,
           const uint32_t* mrope_section, const kvw_paged_cache_t* cache, uint32_t* err_flags,
           cudaStream_t stream) {
    const uint32_t D = cache->head_size, Hk = cache->num_heads;
    if (D % 16 || D > 512 || num_batches > KVW_MAX_BATCHES) return KVW_EUNSUPPORTED;
    if ((uint64_t)num_q_heads + 2ull * Hk > 4096) return KVW_EUNSUPPORTED;
    const uint32_t rows = num_q_heads + 2 * Hk;
    if ((uint64_t)tot_seq_len * rows > (1ull << 31)) return KVW_EUNSUPPORTED;
    if (!values_ok) return KVW_EINVAL;
    if (!qkv || !input_row_offsets || num_batches == 0 || (num_q_heads && !q_out))
        return KVW_EINVAL;
    if (!aligned16(qkv) || !aligned16(q_out) || !aligned4(input_row_offsets) ||
        !aligned4(position_ids) || !aligned16(freqs_cis) || !aligned16(q_gamma) ||
        !aligned16(k_gamma) || !aligned4(err_flags))
        return KVW_EINVAL;
    if (qkv_row_stride < (int64_t)rows * D || qkv_row_stride % 8) return KVW_EINVAL;
    if (num_q_heads && (q_out_row_stride < (int64_t)num_q_heads * D || q_out_row_stride % 8))
        return KVW_EINVAL;
    if (num_q_heads && q_out == qkv && q_out_row_stride != qkv_row_stride) return KVW_EINVAL;
    if (rope_dim % 16 || rope_dim > D) return KVW_EINVAL;
    if (rope_dim && (!freqs_cis || freqs_rows == 0)) return KVW_EINVAL;
    if (!(epsilon >= 0.0f) || !std::isfinite(epsilon) || !std::isfinite(weight_offset))
        return KVW_EINVAL;
    if (mrope_section) {
        if (!position_ids || !rope_dim) return KVW_EINVAL;
        if ((uint64_t)mrope_section[0] + mrope_section[1] + mrope_section[2] != rope_dim / 2)
            return KVW_EINVAL;
    }
    if (tot_seq_len == 0) return KVW_OK;

    a.q_out = static_cast<uint16_t*>(q_out);
    a.qkv = static_cast<const uint16_t*>(qkv);
    a.q_out_stride = q_out_row_stride;
    a.qkv_stride = qkv_row_stride;
    a.offsets = input_row_offsets;
    a.cache_lengths = cache->cache_lengths;
    a.page_table = cache->page_table;
    a.q_gamma = static_cast<const uint16_t*>(q_gamma);
    a.k_gamma = static_cast<const uint16_t*>(k_gamma);
    a.freqs = static_cast<const float*>(freqs_cis);
    a.position_ids = position_ids;
    a.err_flags = err_flags;
    a.eps = epsilon;
    a.weight_offset = weight_offset;
    a.inv_d = 1.0f / (float)D;
    a.B = num_batches;
    a.T = tot_seq_len;
    a.Hq = num_q_heads;
    a.Hk = Hk;
    a.D = D;
    a.rope = rope_dim;
    a.freqs_rows = freqs_rows;
    a.num_pages = cache->num_pages;
    a.max_pages = cache->max_pages_per_seq;
    a.rows = rows;
    if (mrope_section) {
        a.sec0 = mrope_section[0];
        a.sec01 = mrope_section[0] + mrope_section[1];
    }
    a.ps = make_fast_div(cache->page_size);
    const bool mr = mrope_section != nullptr;
    const uint32_t n = D / 16;
    cudaError_t e;
    if (interleaved)
        e = n <= 4    ? pick<4, true>(a, held, mr, stream)
            : n <= 8  ? pick<8, true>(a, held, mr, stream)
            : n <= 16 ? pick<16, true>(a, held, mr, stream)
                      : pick<32, true>(a, held, mr, stream);
    else
        e = n <= 4    ? pick<4, false>(a, held, mr, stream)
            : n <= 8  ? pick<8, false>(a, held, mr, stream)
            : n <= 16 ? pick<16, false>(a, held, mr, stream)
                      : pick<32, false>(a, held, mr, stream);
    return e == cudaSuccess ? KVW_OK : KVW_ECUDA;
}

}  // namespace
}  // namespace kvw

extern "C" int kva_append_qkv_paged(void* q_out, int64_t q_out_row_stride, const void* qkv,
                                    int64_t qkv_row_stride, const uint32_t* input_row_offsets,
                                    uint32_t num_batches, uint32_t tot_seq_len,
                                    uint32_t num_q_heads, const void* q_gamma,
                                    const void* k_gamma, float epsilon, float weight_offset,
                                    const void* freqs_cis, uint32_t freqs_rows, uint32_t rope_dim,
                                    const uint32_t* position_ids, int interleaved,
                                    const uint32_t* mrope_section, const kvw_paged_cache_t* cache,
                                    float v_scale, uint32_t layer_idx, uint32_t* err_flags,
                                    cudaStream_t stream) {
    using namespace kvw;
    const int st = check_cache(cache, layer_idx, 2);
    if (st != KVW_OK) return st;
    AppendArgs a = {};
    const bool fp8 = cache->dtype == KVW_DTYPE_FP8_E4M3;
    const int64_t esz = cache_esz(cache);
    a.k_base = static_cast<unsigned char*>(cache->data) +
               (int64_t)layer_idx * cache->stride_layer * esz;
    a.v_base = a.k_base + cache->stride_kv * esz;
    a.s_page = cache->stride_page;
    a.s_token = cache->stride_token;
    a.s_head = cache->stride_head;
    a.k_scale = cache->scale;
    a.v_scale = v_scale;
    return append(a, fp8 ? Held::kE4m3 : Held::kBf16, value_scale_ok(cache, v_scale), q_out, q_out_row_stride, qkv, qkv_row_stride,
                  input_row_offsets, num_batches, tot_seq_len, num_q_heads, q_gamma, k_gamma,
                  epsilon, weight_offset, freqs_cis, freqs_rows, rope_dim, position_ids,
                  interleaved, mrope_section, cache, err_flags, stream);
}

extern "C" int kva_append_qkv_int4(void* q_out, int64_t q_out_row_stride, const void* qkv,
                                   int64_t qkv_row_stride, const uint32_t* input_row_offsets,
                                   uint32_t num_batches, uint32_t tot_seq_len,
                                   uint32_t num_q_heads, const void* q_gamma,
                                   const void* k_gamma, float epsilon, float weight_offset,
                                   const void* freqs_cis, uint32_t freqs_rows, uint32_t rope_dim,
                                   const uint32_t* position_ids, int interleaved,
                                   const uint32_t* mrope_section, const kvw_paged_cache_t* cache,
                                   const kva_group_scales_t* scales, uint32_t layer_idx,
                                   uint32_t* err_flags, cudaStream_t stream) {
    using namespace kvw;
    const int st = check_int4(cache, scales, layer_idx);
    if (st != KVW_OK) return st;
    AppendArgs a = {};
    a.k_base = int4_codes(cache, layer_idx, 0);
    a.v_base = int4_codes(cache, layer_idx, 1);
    a.s_page = cache->stride_page / 2;
    a.s_token = cache->stride_token / 2;
    a.s_head = cache->stride_head / 2;
    a.k_scales = int4_scales(cache, scales, layer_idx, 0);
    a.v_scales = int4_scales(cache, scales, layer_idx, 1);
    a.sc_page = scales->stride_page;
    a.sc_head = scales->stride_head;
    return append(a, Held::kInt4, true, q_out, q_out_row_stride, qkv, qkv_row_stride,
                  input_row_offsets, num_batches, tot_seq_len, num_q_heads, q_gamma, k_gamma,
                  epsilon, weight_offset, freqs_cis, freqs_rows, rope_dim, position_ids,
                  interleaved, mrope_section, cache, err_flags, stream);
}
