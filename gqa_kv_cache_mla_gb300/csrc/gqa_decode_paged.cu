// Attention of new tokens over a paged GQA key-value cache.
//
// Mathematics, for one token and one group of up to 16 query heads that read
// the same key-value head: one pass over the context with the running maximum
// m and sum l of a softmax.  For each 16 positions, S = Q K^T (16 heads x 16
// positions), the scores' cap, distance bias and mask, m' = max(m, rowmax S),
// P = 2^(S - m'), l' = l 2^(m - m') + sum P, O' = O 2^(m - m') + P V; pieces
// with their own (m, l, O) join by the same rule.
//
// Bound: HBM.  Each cache row is read once for 4 * heads flops per byte, far
// below the ridge, so what counts is bytes in flight.  The units of all
// tokens are cut into equal pieces (kva_split.cuh), one per resident CTA.
// Inside a CTA every warp is a stream of its own: it takes every fourth slice
// of 16 positions, keeps a private ring of slices in shared memory filled by
// 16-byte asynchronous copies (any page size and stride; rows that are not
// there are zero-filled), and its own (m, l, O) in registers; no barrier
// stands between warps until a segment ends, where the four join through
// their own ring memory.  With 96 KB of ring per CTA and two CTAs per SM about
// 130 KB are in flight per SM, three times what HBM latency asks for.
//
// The products use mma.sync m16n8k16: at 16 rows of which a group fills 4 to
// 16, the kernel needs about 1% of the matrix units' rate, and these
// instructions take their operands from registers, where the E4M3 codes are
// converted (exactly) to fp16 on the way.
#include <cstdint>
#include <type_traits>

#include "kva_split.cuh"

namespace kvw {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kSlice = kTile / kWarps;  // positions a warp takes at a time
constexpr int kRows = 16;               // query heads of a row block
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
static_assert(kSlice == 16, "one m16n8k16 operand");

struct GqaArgs {
    SplitArgs split;
    uint16_t* out;
    float* lse;
    const uint16_t* q;
    int64_t q_stride;
    const unsigned char* k_base;  // K plane of the layer
    int64_t kv_bytes;             // from the K plane to the V plane
    int64_t s_page, s_token, s_head;
    const uint32_t* page_table;
    const float* slopes;
    uint32_t* err_flags;
    unsigned char* workspace;
    float sm_scale, softcap, k_scale, v_scale;
    uint32_t Hq, Hk, G, HB, D;  // query heads, kv heads, group, row blocks per group, head size
    uint32_t num_pages, max_pages, pieces;
    FastDiv ps;
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

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
                 "r"(there ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
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

__device__ __forceinline__ float fast_exp2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Two E4M3 codes (low byte first) -> f16x2, exact.
__device__ __forceinline__ uint32_t codes_to_f16x2(uint32_t two) {
    const __half2_raw h =
        __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(two & 0xffffu), __NV_E4M3);
    return (uint32_t)h.x | ((uint32_t)h.y << 16);
}

template <bool F16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    if constexpr (F16) {
        const __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&h);
    } else {
        return pack_bf16x2(lo, hi);
    }
}

// Power of two that brings a row whose largest |value| has the bf16 pattern
// `top` to [2^14, 2^15), and its inverse; 1 for a row of zeros or one that
// holds an infinity or a NaN.  fp16 then holds the row's bf16 values exactly
// down to 2^-31 of the largest.
__device__ __forceinline__ void row_power(uint32_t top, float& up, float& down) {
    const int e = (int)(top >> 7);
    if (top == 0 || e == 255) {
        up = down = 1.0f;
        return;
    }
    const int ue = 268 - e > 254 ? 254 : 268 - e, de = e - 14 < 1 ? 1 : e - 14;
    up = __uint_as_float((uint32_t)ue << 23);
    down = __uint_as_float((uint32_t)de << 23);
}

template <int DP, bool FP8>
struct Shape {
    static constexpr int kEsz = FP8 ? 1 : 2;
    static constexpr int kRowBytes = DP * kEsz;
    static constexpr int kChunks = kRowBytes / 16;  // 16-byte chunks of a row
    static constexpr int kPlane = kSlice * kRowBytes;
    static constexpr int kStage = 2 * kPlane;  // K and V of one slice
    static constexpr int kBudget = (DP > 128 && !FP8 ? 192 : 96) * 1024;
    static constexpr int kFit = kBudget / (kWarps * kStage);
    static constexpr int kStages = kFit > 8 ? 8 : kFit;
    static constexpr int kCtasPerSm = DP > 128 && !FP8 ? 1 : 2;
    static constexpr bool kQInRegs = DP <= 128;
    static constexpr int kQBytes = kQInRegs ? 0 : DP / 16 * 512;
    static constexpr int kScratchPitch = DP + 4;
    static constexpr int kSmem = kWarps * kStages * kStage + kQBytes;
    static_assert(kStages >= 3 && kStages * kStage >= kRows * kScratchPitch * 4, "ring size");
};

// Byte offset of chunk c of row r in a plane: the chunk is exchanged within
// its 128-byte line so that eight rows of one chunk fall on distinct banks.
template <int CHUNKS>
__device__ __forceinline__ uint32_t chunk_at(uint32_t r, uint32_t c) {
    if constexpr (CHUNKS >= 8)
        return (r * CHUNKS + (c ^ (r & 7u))) * 16u;
    else
        return (r * CHUNKS + (c ^ ((r >> 1) & 3u))) * 16u;
}

template <int DP, bool FP8>
__global__ void __launch_bounds__(kThreads, (Shape<DP, FP8>::kCtasPerSm))
    gqa_decode_kernel(const GqaArgs a) {
    using Sh = Shape<DP, FP8>;
    constexpr int KS = DP / 16, NT = DP / 8, CH = Sh::kChunks;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ SplitShared<kThreads> s_split;
    __shared__ float s_m[kWarps][kRows], s_l[kWarps][kRows];
    __shared__ uint32_t s_there[kWarps][Sh::kStages];

    const uint32_t tid = threadIdx.x, warp = tid >> 5, lane = tid & 31u;
    const uint32_t quad = lane >> 2, in_quad = lane & 3u;
    unsigned char* ring = smem + warp * (Sh::kStages * Sh::kStage);
    const uint32_t ring_addr = smem_addr(ring);
    [[maybe_unused]] uint32_t* s_q = reinterpret_cast<uint32_t*>(smem + kWarps * Sh::kStages * Sh::kStage);

    // the join of the pieces may be scheduled; it waits for this grid's end
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    PieceStart piece;
    const bool ok = find_piece(a.split, a.pieces, blockIdx.x, s_split, piece);
    OpenPiece* open = reinterpret_cast<OpenPiece*>(a.workspace) + blockIdx.x;
    if (tid == 0) open->units = 0;
    if (!ok) {
        if (blockIdx.x == 0 && tid == 0) flag(a.err_flags, KVW_ERR_OFFSETS);
        return;
    }
    Walk w;
    w.begin(a.split, piece);
    uint32_t bad_page = 0;

    while (w.u < w.u1) {
        uint32_t block, first, last;
        uint64_t end;
        w.segment(block, first, last, end);
        const uint32_t kvh = block / a.HB, hb = block - kvh * a.HB;
        const uint32_t rows = a.G - hb * kRows < kRows ? a.G - hb * kRows : kRows;
        const uint32_t head0 = kvh * a.G + hb * kRows;
        const uint64_t pos = w.len0 + w.i;
        const uint64_t start = w.span.start, hi = w.span.hi;
        const int64_t head_off = (int64_t)kvh * a.s_head;
        if (pos >= a.split.cap) bad_page = 1;

        // ---- one slice of K and V on its way into stage `st`
        const uint32_t slices = last - first;
        const uint32_t p_first = (w.span.tile0 + first) * kTile + warp * kSlice;
        auto issue = [&](uint32_t k) {
            const uint32_t st = k % Sh::kStages;
            const uint32_t p0 = p_first + k * kTile;
            int64_t off = -1;
            if (lane < kSlice) {
                const uint64_t p = (uint64_t)p0 + lane;
                if (p >= start && p < hi) {
                    off = slot_row(a.page_table, a.max_pages, a.num_pages, a.ps, a.s_page,
                                   a.s_token, head_off, w.b, p);
                    if (off < 0)
                        bad_page = 1;
                    else
                        off *= Sh::kEsz;
                }
            }
            const uint32_t there = __ballot_sync(0xffffffffu, off >= 0);
            if (lane == 0) s_there[warp][st] = there;
            const uint32_t k_dst = ring_addr + st * Sh::kStage, v_dst = k_dst + Sh::kPlane;
            constexpr int kRowsPer = 32 / CH > 0 ? 32 / CH : 1;
            constexpr int kIters = kSlice * CH / 32;
#pragma unroll
            for (int it = 0; it < kIters; ++it) {
                const uint32_t r = CH >= 32 ? it * 32 / CH : it * kRowsPer + lane / CH;
                const uint32_t c = CH >= 32 ? lane + (it * 32) % CH : lane % CH;
                const int64_t o = __shfl_sync(0xffffffffu, off, r);
                const bool in = o >= 0 && c * (16 / Sh::kEsz) < a.D;
                const unsigned char* src = a.k_base + (in ? o + c * 16 : 0);
                cp_async16(k_dst + chunk_at<CH>(r, c), src, in);
                cp_async16(v_dst + chunk_at<CH>(r, c), src + a.kv_bytes, in);
            }
        };
#pragma unroll
        for (int k = 0; k < Sh::kStages - 1; ++k) {
            if ((uint32_t)k < slices) issue(k);
            cp_commit();
        }

        // ---- queries: A operands, fp16 rows brought into range by 2^x
        const uint32_t r0 = quad, r1 = quad + 8;
        const uint16_t* q0 = a.q + (int64_t)w.t * a.q_stride + (int64_t)(head0 + r0) * a.D;
        const uint16_t* q1 = q0 + 8ll * a.D;
        // two neighbouring values of a row; column order of the k16 operand
        // (bf16: as the instruction has it; fp16: the order in which the
        // E4M3 codes of a lane's 4-byte word are unpacked)
        auto q_word = [&](const uint16_t* p, uint32_t r, int ks, int half) -> uint32_t {
            const uint32_t d = 16 * ks + (FP8 ? 4 * in_quad + 2 * half : 2 * in_quad + 8 * half);
            return r < rows && d < a.D ? __ldg(reinterpret_cast<const uint32_t*>(p + d)) : 0u;
        };
        float qs0 = a.sm_scale, qs1 = a.sm_scale, up0 = 1.0f, up1 = 1.0f;
        if constexpr (FP8) {
            uint32_t t0 = 0, t1 = 0;
#pragma unroll
            for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    t0 = __vmaxu2(t0, q_word(q0, r0, ks, h) & 0x7fff7fffu);
                    t1 = __vmaxu2(t1, q_word(q1, r1, ks, h) & 0x7fff7fffu);
                }
#pragma unroll
            for (int o = 1; o < 4; o <<= 1) {
                t0 = __vmaxu2(t0, __shfl_xor_sync(0xffffffffu, t0, o));
                t1 = __vmaxu2(t1, __shfl_xor_sync(0xffffffffu, t1, o));
            }
            t0 = max(t0 & 0xffffu, t0 >> 16);
            t1 = max(t1 & 0xffffu, t1 >> 16);
            float d0, d1;
            row_power(t0, up0, d0);
            row_power(t1, up1, d1);
            qs0 = a.sm_scale * a.k_scale * d0;
            qs1 = a.sm_scale * a.k_scale * d1;
        }
        auto q_conv = [&](uint32_t v, float up) -> uint32_t {
            if constexpr (FP8) return pack2<true>(bf16_lo(v) * up, bf16_hi(v) * up);
            return v;
        };
        uint32_t qf[Sh::kQInRegs ? KS : 1][4];
        if constexpr (Sh::kQInRegs) {
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                qf[ks][0] = q_conv(q_word(q0, r0, ks, 0), up0);
                qf[ks][1] = q_conv(q_word(q1, r1, ks, 0), up1);
                qf[ks][2] = q_conv(q_word(q0, r0, ks, 1), up0);
                qf[ks][3] = q_conv(q_word(q1, r1, ks, 1), up1);
            }
        } else {  // one copy for the four warps, in operand order
            for (int ks = warp; ks < KS; ks += kWarps) {
                uint4 v;
                v.x = q_conv(q_word(q0, r0, ks, 0), up0);
                v.y = q_conv(q_word(q1, r1, ks, 0), up1);
                v.z = q_conv(q_word(q0, r0, ks, 1), up0);
                v.w = q_conv(q_word(q1, r1, ks, 1), up1);
                *reinterpret_cast<uint4*>(s_q + (ks * 32 + lane) * 4) = v;
            }
            __syncthreads();
        }
        float slope0 = 0.0f, slope1 = 0.0f;
        if (a.slopes) {
            slope0 = r0 < rows ? __ldg(a.slopes + head0 + r0) : 0.0f;
            slope1 = r1 < rows ? __ldg(a.slopes + head0 + r1) : 0.0f;
        }

        float acc[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n) acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.0f;
        float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.0f, l1 = 0.0f;

        for (uint32_t k = 0; k < slices; ++k) {
            if (k + Sh::kStages - 1 < slices) issue(k + Sh::kStages - 1);
            cp_commit();
            cp_wait<Sh::kStages - 1>();
            __syncwarp();
            const uint32_t st = k % Sh::kStages;
            const uint32_t there = s_there[warp][st];
            const uint32_t k_src = ring_addr + st * Sh::kStage, v_src = k_src + Sh::kPlane;

            // ---- S = Q K^T
            float s[2][4] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
            const uint32_t mat = lane >> 3, mrow = lane & 7u;
            auto q_frag = [&](int ks, uint32_t(&f)[4]) {
                if constexpr (Sh::kQInRegs) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) f[i] = qf[ks][i];
                } else {
                    const uint4 v = *reinterpret_cast<const uint4*>(s_q + (ks * 32 + lane) * 4);
                    f[0] = v.x; f[1] = v.y; f[2] = v.z; f[3] = v.w;
                }
            };
            if constexpr (!FP8) {
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) {
                    uint32_t kf[4], f[4];
                    ldsm4(kf, k_src + chunk_at<CH>((mat >> 1) * 8 + mrow, 2 * ks + (mat & 1)));
                    q_frag(ks, f);
                    mma16816<false>(s[0], f, kf[0], kf[1]);
                    mma16816<false>(s[1], f, kf[2], kf[3]);
                }
            } else {
#pragma unroll
                for (int ks = 0; ks < KS; ks += 2) {
                    uint32_t kf[4], f[4];
                    ldsm4(kf, k_src + chunk_at<CH>((mat & 1) * 8 + mrow, ks + (mat >> 1)));
                    q_frag(ks, f);
                    mma16816<true>(s[0], f, codes_to_f16x2(kf[0]), codes_to_f16x2(kf[0] >> 16));
                    mma16816<true>(s[1], f, codes_to_f16x2(kf[1]), codes_to_f16x2(kf[1] >> 16));
                    q_frag(ks + 1, f);
                    mma16816<true>(s[0], f, codes_to_f16x2(kf[2]), codes_to_f16x2(kf[2] >> 16));
                    mma16816<true>(s[1], f, codes_to_f16x2(kf[3]), codes_to_f16x2(kf[3] >> 16));
                }
            }

            // ---- scores in units of log2: cap, distance bias, mask
            const uint32_t p0 = p_first + k * kTile;
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t j = n * 8 + 2 * in_quad + (e & 1);
                    float x = s[n][e] * (e < 2 ? qs0 : qs1);
                    if (a.softcap > 0.0f) {
                        // tanh y = 1 - 2 / (e^2y + 1): absolute error of a few
                        // 2^-24, so the capped score is off by that times the cap
                        const float z = fast_exp2(x / a.softcap * (2.0f * kLog2e));
                        x = a.softcap * (1.0f - __fdividef(2.0f, z + 1.0f));
                    }
                    if (a.slopes)
                        x -= (e < 2 ? slope0 : slope1) * (float)((int64_t)pos - (int64_t)(p0 + j));
                    s[n][e] = (there >> j) & 1u ? x * kLog2e : -INFINITY;
                }
            float top0 = fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[1][0], s[1][1]));
            float top1 = fmaxf(fmaxf(s[0][2], s[0][3]), fmaxf(s[1][2], s[1][3]));
#pragma unroll
            for (int o = 1; o < 4; o <<= 1) {
                top0 = fmaxf(top0, __shfl_xor_sync(0xffffffffu, top0, o));
                top1 = fmaxf(top1, __shfl_xor_sync(0xffffffffu, top1, o));
            }
            const bool grows = top0 > m0 || top1 > m1;
            if (__any_sync(0xffffffffu, grows)) {
                const float n0 = fmaxf(m0, top0), n1 = fmaxf(m1, top1);
                const float f0 = n0 == m0 ? 1.0f : fast_exp2(m0 - n0);
                const float f1 = n1 == m1 ? 1.0f : fast_exp2(m1 - n1);
                m0 = n0;
                m1 = n1;
                l0 *= f0;
                l1 *= f1;
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    acc[n][0] *= f0;
                    acc[n][1] *= f0;
                    acc[n][2] *= f1;
                    acc[n][3] *= f1;
                }
            }
            // a row that has seen no position keeps m = -inf: subtract 0
            const float b0 = m0 == -INFINITY ? 0.0f : m0, b1 = m1 == -INFINITY ? 0.0f : m1;
            float p[2][4];
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    p[n][e] = fast_exp2(s[n][e] - (e < 2 ? b0 : b1));
                    if (e < 2) l0 += p[n][e];
                    else l1 += p[n][e];
                }
            uint32_t pf[4];
            pf[0] = pack2<FP8>(p[0][0], p[0][1]);
            pf[1] = pack2<FP8>(p[0][2], p[0][3]);
            pf[2] = pack2<FP8>(p[1][0], p[1][1]);
            pf[3] = pack2<FP8>(p[1][2], p[1][3]);

            // ---- O += P V
#pragma unroll
            for (int c = 0; c < CH; c += 2) {
                uint32_t vf[4];
                ldsm4_trans(vf, v_src + chunk_at<CH>((mat & 1) * 8 + mrow, c + (mat >> 1)));
                if constexpr (!FP8) {  // a chunk is 8 columns
                    mma16816<false>(acc[c], pf, vf[0], vf[1]);
                    mma16816<false>(acc[c + 1], pf, vf[2], vf[3]);
                } else {
                    // a chunk is 16 columns; a word holds two columns of two
                    // positions: even columns to one operand, odd to the next
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t x0 = codes_to_f16x2(vf[2 * h]),
                                       x1 = codes_to_f16x2(vf[2 * h] >> 16);
                        const uint32_t y0 = codes_to_f16x2(vf[2 * h + 1]),
                                       y1 = codes_to_f16x2(vf[2 * h + 1] >> 16);
                        mma16816<true>(acc[2 * (c + h)], pf, __byte_perm(x0, x1, 0x5410),
                                       __byte_perm(y0, y1, 0x5410));
                        mma16816<true>(acc[2 * (c + h) + 1], pf, __byte_perm(x0, x1, 0x7632),
                                       __byte_perm(y0, y1, 0x7632));
                    }
                }
            }
            __syncwarp();  // the stage may be filled again
        }
        cp_wait<0>();
        __syncwarp();

        // ---- the four warps join, in their own rings' memory
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
            l0 += __shfl_xor_sync(0xffffffffu, l0, o);
            l1 += __shfl_xor_sync(0xffffffffu, l1, o);
        }
        if (in_quad == 0) {
            s_m[warp][r0] = m0;
            s_m[warp][r1] = m1;
            s_l[warp][r0] = l0;
            s_l[warp][r1] = l1;
        }
        float* mine = reinterpret_cast<float*>(ring);
        constexpr int pitch = Sh::kScratchPitch;
#pragma unroll
        for (int n = 0; n < NT; n += 2) {
            if constexpr (!FP8) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint32_t d = 8 * (n + i) + 2 * in_quad;
                    *reinterpret_cast<float2*>(mine + r0 * pitch + d) =
                        make_float2(acc[n + i][0], acc[n + i][1]);
                    *reinterpret_cast<float2*>(mine + r1 * pitch + d) =
                        make_float2(acc[n + i][2], acc[n + i][3]);
                }
            } else {
                const uint32_t d = 8 * n + 4 * in_quad;
                *reinterpret_cast<float4*>(mine + r0 * pitch + d) =
                    make_float4(acc[n][0], acc[n + 1][0], acc[n][1], acc[n + 1][1]);
                *reinterpret_cast<float4*>(mine + r1 * pitch + d) =
                    make_float4(acc[n][2], acc[n + 1][2], acc[n][3], acc[n + 1][3]);
            }
        }
        __syncthreads();
        const bool whole = first == 0 && w.u + (last - first) == end;
        float* part = slot_of<DP>(a.workspace, blockIdx.x, first == 0 ? 1 : 0);
        const uint32_t quads = a.D / 4;
        for (uint32_t e = tid; e < rows * quads; e += kThreads) {
            const uint32_t r = e / quads, d = (e - r * quads) * 4;
            float top = s_m[0][r];
#pragma unroll
            for (int v = 1; v < kWarps; ++v) top = fmaxf(top, s_m[v][r]);
            const float base = top == -INFINITY ? 0.0f : top;
            float l = 0.0f;
            float4 o = make_float4(0, 0, 0, 0);
#pragma unroll
            for (int v = 0; v < kWarps; ++v) {
                const float f = fast_exp2(s_m[v][r] - base);
                const float4 x = *reinterpret_cast<const float4*>(
                    smem + v * (Sh::kStages * Sh::kStage) + (r * pitch + d) * 4);
                l += f * s_l[v][r];
                o.x += f * x.x;
                o.y += f * x.y;
                o.z += f * x.z;
                o.w += f * x.w;
            }
            if (whole) {
                const uint64_t row = (uint64_t)w.t * a.Hq + head0 + r;
                const float inv = l == 0.0f ? 0.0f : a.v_scale / l;
                uint2 y;
                y.x = pack_bf16x2(o.x * inv, o.y * inv);
                y.y = pack_bf16x2(o.z * inv, o.w * inv);
                *reinterpret_cast<uint2*>(a.out + row * a.D + d) = y;
                if (d == 0 && a.lse) a.lse[row] = l == 0.0f ? -INFINITY : (top + log2f(l)) * kLn2;
            } else {
                *reinterpret_cast<float4*>(part + r * DP + d) = o;
                if (d == 0) {
                    part[kRows * DP + r] = top;
                    part[kRows * DP + kRows + r] = l;
                }
            }
        }
        if (!whole && first == 0 && tid == 0) {
            open->end = end;
            open->pieces = piece.pieces;
            open->t = w.t;
            open->block = block;
            open->units = piece.units;
        }
        __syncthreads();  // scratch is read: the rings are free
        w.advance(a.split, last - first);
    }
    if (bad_page) flag(a.err_flags, KVW_ERR_PAGE);
}

// Joins a (token, row block) that piece blockIdx.x began and others went on
// with: weights 2^(m_i - M) per row, then one weighted sum over the pieces in
// their order, the pieces dealt to groups of threads and the groups' sums
// added up in order.
constexpr int kJoinThreads = 512;

template <int DP>
__global__ void __launch_bounds__(kJoinThreads) gqa_join_kernel(const GqaArgs a) {
    __shared__ float s_w[kRows][kMaxPieces];
    __shared__ float s_top[kRows], s_sum[kRows];
    __shared__ float4 s_acc[kJoinThreads];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const OpenPiece open = reinterpret_cast<const OpenPiece*>(a.workspace)[blockIdx.x];
    if (open.units == 0) return;
    const uint32_t c0 = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31u;
    // pieces that start before the end: a binary search, the starts ascend
    uint32_t lo = c0 + 1, hi = open.pieces;
    while (lo < hi) {
        const uint32_t mid = (lo + hi) >> 1;
        if (piece_start(open.units, open.pieces, mid) < open.end)
            lo = mid + 1;
        else
            hi = mid;
    }
    const uint32_t n = lo - c0;
    const uint32_t kvh = open.block / a.HB, hb = open.block - kvh * a.HB;
    const uint32_t rows = a.G - hb * kRows < kRows ? a.G - hb * kRows : kRows;
    const uint32_t head0 = kvh * a.G + hb * kRows;
    auto part = [&](uint32_t i) { return slot_of<DP>(a.workspace, c0 + i, i == 0 ? 1 : 0); };

    for (uint32_t r = warp; r < rows; r += kJoinThreads / 32) {
        float top = -INFINITY;
        for (uint32_t i = lane; i < n; i += 32) {
            const float m = part(i)[kRows * DP + r];
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
            l += f * part(i)[kRows * DP + kRows + r];
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
#pragma unroll 4
            for (uint32_t i = g; i < n; i += groups) {
                const float4 x = *reinterpret_cast<const float4*>(part(i) + r * DP + d);
                const float f = s_w[r][i];
                o.x += f * x.x;
                o.y += f * x.y;
                o.z += f * x.z;
                o.w += f * x.w;
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
            const uint64_t row = (uint64_t)open.t * a.Hq + head0 + r;
            const float l = s_sum[r], inv = l == 0.0f ? 0.0f : a.v_scale / l;
            uint2 y;
            y.x = pack_bf16x2(o.x * inv, o.y * inv);
            y.y = pack_bf16x2(o.z * inv, o.w * inv);
            *reinterpret_cast<uint2*>(a.out + row * a.D + d) = y;
            if (d == 0 && a.lse) a.lse[row] = l == 0.0f ? -INFINITY : (s_top[r] + log2f(l)) * kLn2;
        }
    }
}

template <int DP, bool FP8>
cudaError_t launch(GqaArgs& a, cudaStream_t stream) {
    using Sh = Shape<DP, FP8>;
    uint64_t wave = 0;
    cudaError_t e = wave_ctas<&gqa_decode_kernel<DP, FP8>>(kThreads, Sh::kSmem, wave);
    if (e != cudaSuccess) return e;
    if (wave == 0) return cudaErrorInvalidConfiguration;
    if (wave > kMaxPieces) wave = kMaxPieces;
    a.pieces = (uint32_t)wave;
    gqa_decode_kernel<DP, FP8><<<a.pieces, kThreads, Sh::kSmem, stream>>>(a);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.pieces);
    cfg.blockDim = dim3(kJoinThreads);
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, gqa_join_kernel<DP>, a);
}

uint32_t padded_head(uint32_t d) { return d <= 64 ? 64 : d <= 128 ? 128 : 256; }

}  // namespace
}  // namespace kvw

extern "C" int kva_gqa_decode_workspace(uint32_t num_q_heads, uint32_t num_kv_heads,
                                        uint32_t head_size, uint64_t* bytes) {
    using namespace kvw;
    if (!bytes || !num_q_heads || !num_kv_heads || num_q_heads % num_kv_heads) return KVW_EINVAL;
    if (head_size == 0 || head_size % 16 || head_size > 256 || num_q_heads > 4096)
        return KVW_EUNSUPPORTED;
    const uint64_t dp = padded_head(head_size);
    *bytes = kMaxPieces * (sizeof(OpenPiece) + 2 * (kRows * dp + 2 * kRows) * sizeof(float));
    return KVW_OK;
}

extern "C" int kva_gqa_decode_paged(void* out, float* lse, const void* q, int64_t q_row_stride,
                                    const uint32_t* input_row_offsets, uint32_t num_batches,
                                    uint32_t tot_seq_len, uint32_t num_q_heads,
                                    const kvw_paged_cache_t* cache, float v_scale,
                                    uint32_t layer_idx, float sm_scale, float softcap,
                                    uint32_t window, const float* alibi_slopes, void* workspace,
                                    uint64_t workspace_bytes, uint32_t* err_flags,
                                    cudaStream_t stream) {
    using namespace kvw;
    const int st = check_cache(cache, layer_idx, 2);
    if (st != KVW_OK) return st;
    const uint32_t D = cache->head_size, Hk = cache->num_heads;
    uint64_t need = 0;
    const int ws = kva_gqa_decode_workspace(num_q_heads, Hk, D, &need);
    if (ws != KVW_OK) return ws;
    if (num_batches > KVW_MAX_BATCHES || tot_seq_len > (1u << 20)) return KVW_EUNSUPPORTED;
    if (!value_scale_ok(cache, v_scale)) return KVW_EINVAL;
    if (!out || !q || !input_row_offsets || num_batches == 0 || !workspace ||
        workspace_bytes < need)
        return KVW_EINVAL;
    if (!aligned16(out) || !aligned16(q) || !aligned16(workspace) || !aligned4(lse) ||
        !aligned4(input_row_offsets) || !aligned4(alibi_slopes) || !aligned4(err_flags))
        return KVW_EINVAL;
    if (q_row_stride < (int64_t)num_q_heads * D || q_row_stride % 8) return KVW_EINVAL;
    if (!(sm_scale > 0.0f) || !std::isfinite(sm_scale)) return KVW_EINVAL;
    if (!(softcap >= 0.0f) || !std::isfinite(softcap)) return KVW_EINVAL;
    if (tot_seq_len == 0) return KVW_OK;

    GqaArgs a = {};
    a.split.offsets = input_row_offsets;
    a.split.cache_lengths = cache->cache_lengths;
    a.split.B = num_batches;
    a.split.T = tot_seq_len;
    a.G = num_q_heads / Hk;
    a.HB = (a.G + kRows - 1) / kRows;
    a.split.blocks = Hk * a.HB;
    a.split.min_units = 1;
    a.split.cap = (uint64_t)cache->max_pages_per_seq * cache->page_size;
    if (a.split.cap > (1ull << 32)) a.split.cap = 1ull << 32;
    a.split.window = window ? window : 1ull << 40;
    a.out = static_cast<uint16_t*>(out);
    a.lse = lse;
    a.q = static_cast<const uint16_t*>(q);
    a.q_stride = q_row_stride;
    const int64_t esz = cache_esz(cache);
    const bool fp8 = esz == 1;
    a.k_base = static_cast<const unsigned char*>(cache->data) +
               (int64_t)layer_idx * cache->stride_layer * esz;
    a.kv_bytes = cache->stride_kv * esz;
    a.s_page = cache->stride_page;
    a.s_token = cache->stride_token;
    a.s_head = cache->stride_head;
    a.page_table = cache->page_table;
    a.slopes = alibi_slopes;
    a.err_flags = err_flags;
    a.workspace = static_cast<unsigned char*>(workspace);
    a.sm_scale = sm_scale;
    a.softcap = softcap;
    a.k_scale = fp8 ? cache->scale : 1.0f;
    a.v_scale = fp8 ? v_scale : 1.0f;
    a.Hq = num_q_heads;
    a.Hk = Hk;
    a.D = D;
    a.num_pages = cache->num_pages;
    a.max_pages = cache->max_pages_per_seq;
    a.ps = make_fast_div(cache->page_size);
    cudaError_t e;
    switch (padded_head(D)) {
        case 64: e = fp8 ? launch<64, true>(a, stream) : launch<64, false>(a, stream); break;
        case 128: e = fp8 ? launch<128, true>(a, stream) : launch<128, false>(a, stream); break;
        default: e = fp8 ? launch<256, true>(a, stream) : launch<256, false>(a, stream); break;
    }
    return e == cudaSuccess ? KVW_OK : KVW_ECUDA;
}
