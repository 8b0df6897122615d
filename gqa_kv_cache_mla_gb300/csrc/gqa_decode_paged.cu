// Attention of new tokens over a paged GQA key-value cache.
//
// Mathematics, for a row block of up to 16 rows (the query heads of a group
// times the tokens of a chunk) that read the same key-value head: one pass
// over the context with the running maximum m and sum l of a softmax.  For
// each 16 positions, S = Q K^T (16 rows x 16 positions), the scores' cap,
// distance bias and mask, m' = max(m, rowmax S), P = 2^(S - m'),
// l' = l 2^(m - m') + sum P, O' = O 2^(m - m') + P V; parts with their own
// (m, l, O) join by the same rule.
//
// Bound: HBM.  Each cache row is read once for 4 * 16 flops per value at
// most, far below the ridge, so what counts is bytes in flight.  The units of
// all chunks are cut into equal pieces (kva_split.cuh), one per resident CTA,
// two CTAs per SM.  In a CTA one warp feeds a ring of half tiles (64
// positions of K or of V) with tensor-map copies, running ahead across the
// ends of segments, and four warps consume it, 16 positions of each tile
// each, with (m, l, O) in registers of their own; nothing stands between the
// four until a segment ends, where they join in shared memory.  96 KB of ring
// per CTA keep up to 190 KB in flight per SM.
//
// Measured, 32 query and 8 key-value heads of 128: 8 requests of up to 131072
// positions, bf16 302 us (6.7 TB/s, 99 % of the card's copy rate); 256 of up to
// 8192, E4M3 331 us (6.5 TB/s, 96 %), with a cap 365, with a distance bias 372,
// pages of 16 454, of 100 457, heads of 64 222 (72 %), of 96 328 (73 %); 32 of
// up to 4096, bf16 53 us (5.2 TB/s, some 12 us of it before the first and after
// the last byte); one token over 901 positions 9.9 us.
//
// CTAs of neighbouring key-value heads walk the same piece side by side
// (`lanes`): a token's heads lie next to each other, so what one CTA reads
// completes the DRAM rows and L2 lines that the others read at that time.  In
// turn, one head's contexts after the other's, 256 requests of up to 8192
// positions took: E4M3 heads of 96 546 us (side by side 362), of 128 371 (364),
// bf16 heads of 64 403 (323: 6.7 TB/s), 64 requests of 4 new tokens 153 (119).
//
// The products use mma.sync m16n8k16: at 16 rows the kernel needs a few
// percent of the matrix units' rate, and these instructions take their
// operands from registers, where the E4M3 codes are converted (exactly) to
// fp16 on the way.
#include <cstdint>
#include <type_traits>

#include "kva_gqa.cuh"
#include "kva_tma.cuh"

namespace kvw {
namespace {

constexpr int kWarps = 4;                   // consumers
// Two warpgroups: the consumers, and one whose first warp feeds.  The launch
// gives every thread 128 registers (two CTAs fill an SM's file); the feeding
// group hands 72 of them on to the consumers.
constexpr int kThreads = 32 * 2 * kWarps;
constexpr int kConsumerRegs = 200, kFeederRegs = 56;
static_assert(kConsumerRegs + kFeederRegs <= 2 * 128, "registers of the launch");
constexpr int kSlice = kTile / kWarps;      // positions of a tile that a warp takes
static_assert(kSlice == 16, "one m16n8k16 operand");
template <int DP, bool FP8>
struct Shape {
    static constexpr int kEsz = FP8 ? 1 : 2;
    // Bytes of a swizzled line.  Always 128: a copy may be a single row, and
    // its place in shared memory has to be 128-byte aligned (64-wide E4M3
    // rows leave half of a line empty).
    static constexpr int kLine = 128;
    static constexpr int kBlocks = (DP * kEsz + kLine - 1) / kLine;  // lines of a row
    static constexpr int kBlock = kTile * kLine;     // one line of every row of a tile
    static constexpr int kHalf = kBlocks * kBlock;   // K or V of one tile
    static constexpr int kHalves = 96 * 1024 / kHalf > 12 ? 12 : 96 * 1024 / kHalf;
    static constexpr bool kPair = kHalves >= 12;  // two slices at a time: half the softmax's cost
    static constexpr int kRing = kHalves * kHalf;
    // queries stay in registers while the accumulators leave room
    static constexpr bool kQInRegs = DP <= 128;
    static constexpr int kQBufs = DP <= 64 ? 2 : 1;
    // eight rows on distinct banks (256-wide heads have no memory left for it)
    static constexpr int kQPitch = DP * 2 + (DP <= 128 ? 16 : 0);
    // rows that join at a time; their memory holds Q's operands in between
    // where these are not in registers
    static constexpr int kJoinRows = 1024 / (kWarps * DP / 2);
    static constexpr int kJoin = 8192;
    static_assert(kHalves >= 3 && kWarps * kJoinRows * DP * 4 == kJoin, "shared memory");
    static_assert(kQInRegs || DP / 16 * 512 <= kJoin, "Q operands");
};

template <int DP, bool FP8>
struct Smem {
    using Sh = Shape<DP, FP8>;
    unsigned char ring[Sh::kRing];
    unsigned char q_raw[Sh::kQBufs][kRows * Sh::kQPitch];
    unsigned char join[Sh::kJoin];
    uint64_t full[Sh::kHalves], empty[Sh::kHalves], q_full[2], q_empty[2], meet;
    uint64_t there[Sh::kHalves];  // of a K half: positions of the tile that are there
    float m[kWarps][kRows], l[kWarps][kRows];
    SplitShared<kThreads> split;
    uint32_t stop;  // a wait ran out
};

// Byte offset in a half tile of 16-byte chunk c of row r.
template <int DP, bool FP8>
__device__ __forceinline__ uint32_t chunk_at(uint32_t r, uint32_t c) {
    return (c >> 3) * Shape<DP, FP8>::kBlock + r * 128u + (((c ^ r) & 7u) << 4);
}

// The feeding warp: walks the piece's tiles ahead of the arithmetic.
template <int DP, bool FP8, Hook HOOK>
__device__ __forceinline__ void feed(const GqaArgs& a, const CacheMaps& maps,
                                     Smem<DP, FP8>& sm) {
    using Sh = Shape<DP, FP8>;
    const uint32_t lane = threadIdx.x & 31u;
    Walk w;
    w.begin(a.split, sm.split.start);
    RingPos<Sh::kHalves> at;
    RingPos<Sh::kQBufs> q_at;
    uint32_t bad_page = 0, issued = 0;
    bool ok = true, first_half = true;
    while (ok && !w.done()) {
        const uint32_t block = w.block * a.lanes + blockIdx.x % a.lanes;
        const uint32_t kvh = a.HB == 1 ? block : block / a.HB, hb = block - kvh * a.HB;
        const uint32_t in_block = a.G - hb * kRows < a.per_token ? a.G - hb * kRows : a.per_token;
        prefetch_page(maps, a.page_table, a.max_pages, a.ps, w.b,
                      (int64_t)(w.span.tile0 + w.first) * kTile, lane);
        // ---- the queries: one copy per row
        ok = wait_phase(&sm.q_empty[q_at.slot], q_at.parity ^ 1u, &sm.stop, a.wait_limit);
        if (!ok) break;
        const uint32_t rows = w.span.tokens * in_block;
        if (lane == 0) mbar_arrive_expect_tx(&sm.q_full[q_at.slot], rows * a.D * 2);
        __syncwarp();
        if (lane < rows) {
            const uint32_t ct = w.span.tokens == 1 ? 0 : lane / in_block;
            bulk_load(sm.q_raw[q_at.slot] + lane * Sh::kQPitch,
                      a.q + (int64_t)(w.t + ct) * a.q_stride +
                          (int64_t)(kvh * a.G + hb * kRows + (lane - ct * in_block)) * a.D,
                      a.D * 2, &sm.q_full[q_at.slot]);
        }
        q_at.step();
        // ---- the tiles
        if (maps.log_rows == 6) {
            // A tile lies in one page: one copy of each half, and all that it
            // takes is the same in every lane.  (The general way below takes
            // longer to feed than E4M3 tiles take to consume: 256 requests, 363
            // us against 329 when it was added, heads of 64 330 against 232.)
            auto plan = [&](uint32_t i) {
                return plan_page(a.page_table, a.max_pages, a.num_pages, a.ps, w.b,
                                 (w.span.tile0 + i) * kTile, w.span.start, w.span.hi);
            };
            PagePlan next = plan(w.first);
            for (uint32_t i = w.first; ok && i < w.last; ++i) {
                const PagePlan t = next;
                if (i + 1 < w.last) next = plan(i + 1);
                if (!t.valid) bad_page = 1;
#pragma unroll 1
                for (uint32_t plane = 0; plane < 2; ++plane) {
                    ok = wait_phase(&sm.empty[at.slot], at.parity ^ 1u, &sm.stop, a.wait_limit);
                    if (!ok) break;
                    if (elect_one()) {
                        uint64_t* full = &sm.full[at.slot];
                        if (plane == 0) sm.there[at.slot] = t.there;
                        mbar_arrive_expect_tx(full, t.valid ? Sh::kHalf : 0);
                        const uint32_t dst = smem_addr(sm.ring + at.slot * Sh::kHalf);
                        if (t.valid && !(HOOK == Hook::kWithheld && first_half)) {
#pragma unroll
                            for (int blk = 0; blk < Sh::kBlocks; ++blk)
                                tma_rows(dst + blk * Sh::kBlock, &maps.map[0],
                                         blk * (Sh::kLine / Sh::kEsz), kvh, t.row, t.page, plane,
                                         smem_addr(full));
                        }
                    }
                    __syncwarp();
                    first_half = false;
                    at.step();
                    ++issued;
                }
            }
            if (ok) w.next(a.split);
            continue;
        }
        for (uint32_t i = w.first; ok && i < w.last; ++i) {
            const int64_t p_tile = (int64_t)(w.span.tile0 + i) * kTile;
            TilePlan t;
            plan_tile(maps, a.page_table, a.max_pages, a.num_pages, a.ps, w.b, p_tile,
                      w.span.start, w.span.hi, t, bad_page);
#pragma unroll 1
            for (uint32_t plane = 0; plane < 2; ++plane) {
                ok = wait_phase(&sm.empty[at.slot], at.parity ^ 1u, &sm.stop, a.wait_limit);
                if (!ok) break;
                if (lane == 0) {
                    if (plane == 0) sm.there[at.slot] = ((uint64_t)t.t_hi << 32) | t.t_lo;
                    mbar_arrive_expect_tx(&sm.full[at.slot],
                                          (t.n << maps.log_rows) * Sh::kLine * Sh::kBlocks);
                }
                __syncwarp();
                if (!(HOOK == Hook::kWithheld && first_half)) {
                    const uint32_t bar = smem_addr(&sm.full[at.slot]);
                    const uint32_t base = smem_addr(sm.ring + at.slot * Sh::kHalf);
                    each_copy(maps, t, [&](uint32_t unit, uint32_t row, uint32_t page,
                                              const CUtensorMap* map) {
                        const uint32_t dst = base + (unit << maps.log_rows) * Sh::kLine;
#pragma unroll
                        for (int blk = 0; blk < Sh::kBlocks; ++blk)
                            tma_rows(dst + blk * Sh::kBlock, map, blk * (Sh::kLine / Sh::kEsz), kvh,
                                     row, page, plane, bar);
                    });
                }
                first_half = false;
                at.step();
                ++issued;
            }
        }
        if (ok) w.next(a.split);
    }
    if (bad_page) flag(a.err_flags, KVW_ERR_PAGE);
    if (!ok && lane == 0) flag(a.err_flags, KVW_ERR_TIMEOUT);
    // Whether or not this warp had to wait in vain: it leaves when the last copy
    // into each place has landed, or after a bounded time.
    const uint32_t n = issued < (uint32_t)Sh::kHalves ? issued : (uint32_t)Sh::kHalves;
    for (uint32_t i = 0; i < n; ++i) {
        const uint32_t x = issued - 1 - i;
        leave_phase<HOOK>(&sm.full[x % Sh::kHalves], (x / Sh::kHalves) & 1u, a.wait_limit,
                          a.err_flags);
    }
    for (uint32_t i = 0; i < (uint32_t)Sh::kQBufs; ++i)
        leave_phase<HOOK>(&sm.q_full[i], q_at.parity ^ (i < q_at.slot ? 0u : 1u), a.wait_limit,
                          a.err_flags);
}

// HIGH: a row block may have more than 8 rows; without it the upper half of
// every operand is constant zeros and nothing is computed for it (256 requests,
// E4M3, groups of 4: 383 -> 374 us, with distance bias 435 -> 400 us).
template <int DP, bool FP8, bool MODS, bool HIGH, Hook HOOK>
__global__ void __launch_bounds__(kThreads, 2)
    gqa_decode_kernel(const GqaArgs a, const __grid_constant__ CacheMaps maps) {
    using Sh = Shape<DP, FP8>;
    constexpr int KS = DP / 16, NT = DP / 8, CH = DP * Sh::kEsz / 16, NP = Sh::kPair ? 2 : 1;
    constexpr int kEach = HIGH ? 4 : 2;  // scores of a product that are looked at
    extern __shared__ __align__(1024) unsigned char dyn[];
    Smem<DP, FP8>& sm = *reinterpret_cast<Smem<DP, FP8>*>(dyn);

    const uint32_t tid = threadIdx.x, warp = tid >> 5, lane = tid & 31u;
    // the join of the pieces may be scheduled; it waits for this grid's end
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    if (tid == kThreads - 32) {  // not a thread that the division of the work waits for
        for (int i = 0; i < Sh::kHalves; ++i) {
            mbar_init(&sm.full[i], 1);
            mbar_init(&sm.empty[i], kWarps);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sm.q_full[i], 1);
            mbar_init(&sm.q_empty[i], kWarps);
        }
        mbar_init(&sm.meet, kWarps);
        sm.stop = 0;
        mbar_init_fence();
        prefetch_map(&maps.map[0]);
    }
    // All that touches global memory comes after the kernel before this one in
    // the stream; its launch and the lines above do not (calls in a row,
    // one token over 901 positions 14.4 -> 12.3 us).
    wait_for_stream();
    const bool ok = find_piece(a.split, a.pieces, blockIdx.x / a.lanes, sm.split);
    OpenPiece* open = reinterpret_cast<OpenPiece*>(a.workspace) + blockIdx.x;
    if (tid == 0) open->n = 0;
    if (!ok) {
        if (blockIdx.x == 0 && tid == 0) flag(a.err_flags, KVW_ERR_OFFSETS);
        return;
    }
    if (warp >= kWarps) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kFeederRegs));
        if (warp == kWarps) feed<DP, FP8, HOOK>(a, maps, sm);
        return;
    }
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kConsumerRegs));

    const uint32_t quad = lane >> 2, in_quad = lane & 3u;
    const uint32_t ring_addr = smem_addr(sm.ring);
    float* s_join = reinterpret_cast<float*>(sm.join);
    [[maybe_unused]] uint32_t* s_q = reinterpret_cast<uint32_t*>(sm.join);
    RingPos<Sh::kHalves> at;
    RingPos<Sh::kQBufs> q_at;
    uint32_t meet_parity = 0;
    auto ready = [&](const RingPos<Sh::kHalves>& x) {
        return wait_phase(&sm.full[x.slot], x.parity, &sm.stop, a.wait_limit);
    };
    // the consumers meet (bounded, so that one that gave up strands nobody)
    auto meet = [&]() {
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.meet);
        const bool met = wait_phase(&sm.meet, meet_parity, &sm.stop, a.wait_limit);
        meet_parity ^= 1u;
        return met;
    };
    Walk w;
    w.begin(a.split, sm.split.start);
    bool alive = true;
    if constexpr (HOOK == Hook::kAbandoned) {
        *reinterpret_cast<volatile uint32_t*>(&sm.stop) = 1;
        alive = false;
    }
    while (alive && !w.done()) {
        const uint32_t block = w.block * a.lanes + blockIdx.x % a.lanes;
        const uint32_t kvh = a.HB == 1 ? block : block / a.HB, hb = block - kvh * a.HB;
        const uint32_t in_block = a.G - hb * kRows < a.per_token ? a.G - hb * kRows : a.per_token;
        const uint32_t rows = w.span.tokens * in_block;
        const uint32_t head0 = kvh * a.G + hb * kRows;
        const int64_t pos0 = (int64_t)w.len0 + ((int64_t)w.k << a.split.log_c);
        if (pos0 + w.span.tokens > a.split.cap && tid == 0) flag(a.err_flags, KVW_ERR_PAGE);

        const uint32_t shared_by = w.first == 0 && !w.whole()
                                       ? sharers(a.split, sm.split.start, w, blockIdx.x / a.lanes)
                                       : 0;

        // ---- queries: A operands, fp16 rows brought into range by 2^x
        const uint32_t r0 = quad, r1 = quad + 8;
        const uint32_t t0 = w.span.tokens == 1 ? 0 : r0 / in_block;  // tokens of the chunk
        const uint32_t t1 = w.span.tokens == 1 ? 0 : r1 / in_block;
        alive = wait_phase(&sm.q_full[q_at.slot], q_at.parity, &sm.stop, a.wait_limit);
        if (!alive) break;
        const unsigned char* q0 = sm.q_raw[q_at.slot] + r0 * Sh::kQPitch;
        const unsigned char* q1 = q0 + 8 * Sh::kQPitch;
        // two neighbouring values of a row; column order of the k16 operand
        // (bf16: as the instruction has it; fp16: the order in which the
        // E4M3 codes of a lane's 4-byte word are unpacked)
        auto q_word = [&](const unsigned char* p, uint32_t r, int ks, int half) -> uint32_t {
            const uint32_t d = 16 * ks + (FP8 ? 4 * in_quad + 2 * half : 2 * in_quad + 8 * half);
            return r < rows && d < a.D ? *reinterpret_cast<const uint32_t*>(p + 2 * d) : 0u;
        };
        constexpr int kStep = Sh::kQInRegs ? 1 : kWarps;  // or one copy for the four warps
        uint32_t qf[KS / kStep][4];
#pragma unroll
        for (int i = 0; i < KS / kStep; ++i) {
            const int ks = Sh::kQInRegs ? i : i * kWarps + (int)warp;
            qf[i][0] = q_word(q0, r0, ks, 0);
            qf[i][1] = HIGH ? q_word(q1, r1, ks, 0) : 0u;
            qf[i][2] = q_word(q0, r0, ks, 1);
            qf[i][3] = HIGH ? q_word(q1, r1, ks, 1) : 0u;
        }
        float qs0 = a.sm_scale, qs1 = a.sm_scale;
        if constexpr (FP8) {
            uint32_t top0 = 0, top1 = 0;
#pragma unroll
            for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t x0 = kStep == 1 ? qf[ks / kStep][2 * h] : q_word(q0, r0, ks, h);
                    const uint32_t x1 = !HIGH ? 0u
                                        : kStep == 1 ? qf[ks / kStep][2 * h + 1]
                                                     : q_word(q1, r1, ks, h);
                    top0 = __vmaxu2(top0, x0 & 0x7fff7fffu);
                    top1 = __vmaxu2(top1, x1 & 0x7fff7fffu);
                }
#pragma unroll
            for (int o = 1; o < 4; o <<= 1) {
                top0 = __vmaxu2(top0, __shfl_xor_sync(0xffffffffu, top0, o));
                top1 = __vmaxu2(top1, __shfl_xor_sync(0xffffffffu, top1, o));
            }
            top0 = max(top0 & 0xffffu, top0 >> 16);
            top1 = max(top1 & 0xffffu, top1 >> 16);
            float up0, up1, d0, d1;
            row_power(top0, up0, d0);
            row_power(top1, up1, d1);
            qs0 = a.sm_scale * a.k_scale * d0;
            qs1 = a.sm_scale * a.k_scale * d1;
#pragma unroll
            for (int i = 0; i < KS / kStep; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t x0 = qf[i][2 * h], x1 = qf[i][2 * h + 1];
                    qf[i][2 * h] = pack2<true>(bf16_lo(x0) * up0, bf16_hi(x0) * up0);
                    if constexpr (HIGH)
                        qf[i][2 * h + 1] = pack2<true>(bf16_lo(x1) * up1, bf16_hi(x1) * up1);
                }
        }
        // scores in units of log2 straight from the product, or 2 log2(e) / cap
        // of them
        qs0 *= MODS && a.softcap > 0.0f ? a.cap_factor : kLog2e;
        qs1 *= MODS && a.softcap > 0.0f ? a.cap_factor : kLog2e;
        // never 0, a masked score is -inf times this, and never infinite (a tiny
        // cap), as a score may be 0
        qs0 = fminf(fmaxf(qs0, 1.17549435e-38f), 3.4028234e38f);
        qs1 = fminf(fmaxf(qs1, 1.17549435e-38f), 3.4028234e38f);
        if constexpr (!Sh::kQInRegs) {
#pragma unroll
            for (int i = 0; i < KS / kStep; ++i)
                *reinterpret_cast<uint4*>(s_q + ((i * kWarps + warp) * 32 + lane) * 4) =
                    make_uint4(qf[i][0], qf[i][1], qf[i][2], qf[i][3]);
            alive = meet();
            if (!alive) break;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.q_empty[q_at.slot]);
        q_at.step();
        auto q_frag = [&](int ks, uint32_t(&f)[4]) {
            if constexpr (Sh::kQInRegs) {
#pragma unroll
                for (int i = 0; i < 4; ++i) f[i] = HIGH || !(i & 1) ? qf[ks / kStep][i] : 0u;
            } else {
                const uint4 v = *reinterpret_cast<const uint4*>(s_q + (ks * 32 + lane) * 4);
                f[0] = v.x; f[1] = HIGH ? v.y : 0u; f[2] = v.z; f[3] = HIGH ? v.w : 0u;
            }
        };
        float slope0 = 0.0f, slope1 = 0.0f;
        if constexpr (MODS) {
            if (a.slopes) {
                slope0 = r0 < rows ? kLog2e * __ldg(a.slopes + head0 + (r0 - t0 * in_block)) : 0.0f;
                slope1 = r1 < rows ? kLog2e * __ldg(a.slopes + head0 + (r1 - t1 * in_block)) : 0.0f;
            }
        }
        // positions every row of the block sees, and each row's own
        const int64_t all_hi = pos0, all_lo = pos0 + w.span.tokens - a.split.window;
        const int64_t own0 = pos0 + t0, own1 = pos0 + t1;
        auto sees = [&](int64_t own, int64_t p) { return p <= own && p > own - a.split.window; };

        float acc[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n) acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.0f;
        float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.0f, l1 = 0.0f;
        const uint32_t mat = lane >> 3, mrow = lane & 7u;
        const int64_t p_first = (int64_t)(w.span.tile0 + w.first) * kTile + warp * kSlice;

        // Is every position of this warp's slice there, in the K half at x?
        auto full_slice = [&](const RingPos<Sh::kHalves>& x) {
            return ((uint32_t)(sm.there[x.slot] >> (warp * kSlice)) & 0xffffu) == 0xffffu;
        };
        // `N` slices of tiles k, k + 1, ... whose K halves have arrived; EDGE:
        // positions may be missing, or seen by some rows only
        auto slices = [&](uint32_t k, auto n_const, auto edge_const) -> bool {
            constexpr int N = decltype(n_const)::value;
            constexpr bool EDGE = decltype(edge_const)::value;
            RingPos<Sh::kHalves> h[2 * N];  // K and V of each
            h[0] = at;
#pragma unroll
            for (int i = 1; i < 2 * N; ++i) {
                h[i] = h[i - 1];
                h[i].step();
            }
            at = h[2 * N - 1];
            at.step();
            float s[2 * N][4];
#pragma unroll
            for (int i = 0; i < 2 * N; ++i) s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.0f;
            [[maybe_unused]] uint32_t there[N];
            // ---- S = Q K^T
#pragma unroll
            for (int i = 0; i < N; ++i) {
                if constexpr (EDGE)
                    there[i] = (uint32_t)(sm.there[h[2 * i].slot] >> (warp * kSlice)) & 0xffffu;
                const uint32_t src = ring_addr + h[2 * i].slot * Sh::kHalf;
                const uint32_t row0 = warp * kSlice;
                if constexpr (!FP8) {
#pragma unroll
                    for (int ks = 0; ks < KS; ++ks) {
                        uint32_t kf[4], f[4];
                        ldsm4(kf, src + chunk_at<DP, FP8>(row0 + (mat >> 1) * 8 + mrow,
                                                          2 * ks + (mat & 1)));
                        q_frag(ks, f);
                        mma16816<false>(s[2 * i], f, kf[0], kf[1]);
                        mma16816<false>(s[2 * i + 1], f, kf[2], kf[3]);
                    }
                } else {
#pragma unroll
                    for (int ks = 0; ks < KS; ks += 2) {
                        uint32_t kf[4], f[4], x, y;
                        ldsm4(kf, src + chunk_at<DP, FP8>(row0 + (mat & 1) * 8 + mrow,
                                                          ks + (mat >> 1)));
#pragma unroll
                        for (int hh = 0; hh < 2; ++hh) {
                            q_frag(ks + hh, f);
                            codes_to_f16(kf[2 * hh], x, y);
                            mma16816<true>(s[2 * i], f, x, y);
                            codes_to_f16(kf[2 * hh + 1], x, y);
                            mma16816<true>(s[2 * i + 1], f, x, y);
                        }
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.empty[h[2 * i].slot]);
            }
            // ---- cap, distance bias, mask
#pragma unroll
            for (int i = 0; i < N; ++i) {
                [[maybe_unused]] const int64_t p0 = p_first + (int64_t)(k + i) * kTile;
                if constexpr (MODS) {  // into units of log2
                    if (a.softcap > 0.0f) {
                        // With u = 2 log2(e) y: tanh y = 1 - 2 / (2^u + 1), off by
                        // 1.6 * 2^-22 of the cap, which is 2^-19 of the capped
                        // score from y = 1/4 on; below, where a cap far above
                        // the scores would lose them in that, the odd series
                        // y - y^3/3 + 2 y^5/15 - 17 y^7/315, off by 2^-21 of
                        // itself there (256 requests, E4M3: 353 -> 363 us; bf16
                        // with cap and window the same).
#pragma unroll
                        for (int n = 0; n < 2; ++n)
#pragma unroll
                            for (int e = 0; e < kEach; ++e) {
                                const float u = s[2 * i + n][e] * (e < 2 ? qs0 : qs1), w = u * u;
                                const float near =
                                    a.cap_half * u *
                                    fmaf(w, fmaf(w, fmaf(w, -kTanh7, kTanh5), -kTanh3), 1.0f);
                                const float far =
                                    a.softcap - __fdividef(2.0f * a.softcap, fast_exp2(u) + 1.0f);
                                s[2 * i + n][e] = fabsf(u) < kTanhNear ? near : far;
                            }
                    }
                    if (a.slopes) {
                        // slope * (offset in the slice - distance of its start)
                        const float f0 = a.softcap > 0.0f ? 1.0f : qs0;
                        const float f1 = a.softcap > 0.0f ? 1.0f : qs1;
                        const int64_t from = p0 + 2 * in_quad;
                        const float away0 = slope0 * (float)(own0 - from);
                        const float away1 = slope1 * (float)(own1 - from);
#pragma unroll
                        for (int n = 0; n < 2; ++n)
#pragma unroll
                            for (int e = 0; e < kEach; ++e) {
                                const float bias = fmaf(e < 2 ? slope0 : slope1,
                                                        (float)(n * 8 + (e & 1)),
                                                        e < 2 ? -away0 : -away1);
                                s[2 * i + n][e] = fmaf(s[2 * i + n][e], e < 2 ? f0 : f1, bias);
                            }
                    }
                }
                if constexpr (EDGE) {
#pragma unroll
                    for (int n = 0; n < 2; ++n)
#pragma unroll
                        for (int e = 0; e < kEach; ++e) {
                            const uint32_t j = n * 8 + 2 * in_quad + (e & 1);
                            if (!((there[i] >> j) & 1u) || !sees(e < 2 ? own0 : own1, p0 + j))
                                s[2 * i + n][e] = -INFINITY;
                        }
                }
            }
            // ---- running maximum, weights
            float top0 = -INFINITY, top1 = -INFINITY;
#pragma unroll
            for (int i = 0; i < 2 * N; ++i) {
                top0 = fmaxf(top0, fmaxf(s[i][0], s[i][1]));
                if constexpr (HIGH) top1 = fmaxf(top1, fmaxf(s[i][2], s[i][3]));
            }
#pragma unroll
            for (int o = 1; o < 4; o <<= 1) {
                top0 = fmaxf(top0, __shfl_xor_sync(0xffffffffu, top0, o));
                if constexpr (HIGH) top1 = fmaxf(top1, __shfl_xor_sync(0xffffffffu, top1, o));
            }
            if constexpr (!MODS) {
                top0 *= qs0;
                top1 *= qs1;
            }
            constexpr float kLift = weight_lift<FP8>();
            const bool grows =
                top0 > m0 + (kSlack + kLift) || (HIGH && top1 > m1 + (kSlack + kLift));
            if (__any_sync(0xffffffffu, grows)) {
                const float n0 = fmaxf(m0, top0 - kLift), n1 = fmaxf(m1, top1 - kLift);
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
                    if constexpr (HIGH) {
                        acc[n][2] *= f1;
                        acc[n][3] *= f1;
                    }
                }
            }
            // a row that has seen no position keeps m = -inf: subtract 0
            const float b0 = m0 == -INFINITY ? 0.0f : m0, b1 = m1 == -INFINITY ? 0.0f : m1;
            uint32_t pf[N][4];
#pragma unroll
            for (int i = 0; i < N; ++i) {
                float p[2][4];
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int e = 0; e < kEach; ++e) {
                        const float x = s[2 * i + n][e], b = e < 2 ? b0 : b1;
                        p[n][e] = fast_exp2(MODS ? x - b : fmaf(x, e < 2 ? qs0 : qs1, -b));
                        if (e < 2) l0 += p[n][e];
                        else l1 += p[n][e];
                    }
                pf[i][0] = pack2<FP8>(p[0][0], p[0][1]);
                pf[i][1] = HIGH ? pack2<FP8>(p[0][2], p[0][3]) : 0u;
                pf[i][2] = pack2<FP8>(p[1][0], p[1][1]);
                pf[i][3] = HIGH ? pack2<FP8>(p[1][2], p[1][3]) : 0u;
            }
            // ---- O += P V
            auto times_v = [&](uint32_t src, const uint32_t(&p)[4], auto masked, uint32_t low,
                               uint32_t high, bool row0, bool row1) {
                constexpr bool kMasked = decltype(masked)::value;
                auto add = [&](float(&c)[4], uint32_t x, uint32_t y) {
                    if constexpr (!kMasked) {
                        mma16816<FP8>(c, p, x, y);
                    } else {
                        float t[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                        mma16816<FP8>(t, p, x, y);
                        if (row0) {
                            c[0] += t[0];
                            c[1] += t[1];
                        }
                        if (row1) {
                            c[2] += t[2];
                            c[3] += t[3];
                        }
                    }
                };
#pragma unroll
                for (int c = 0; c < CH; c += 2) {
                    uint32_t vf[4];
                    ldsm4_trans(vf, src + chunk_at<DP, FP8>(warp * kSlice + (mat & 1) * 8 + mrow,
                                                            c + (mat >> 1)));
                    if constexpr (kMasked) {
                        vf[0] &= low;
                        vf[1] &= high;
                        vf[2] &= low;
                        vf[3] &= high;
                    }
                    if constexpr (!FP8) {  // a chunk is 8 columns
                        add(acc[c], vf[0], vf[1]);
                        add(acc[c + 1], vf[2], vf[3]);
                    } else {
                        // a chunk is 16 columns; a word holds two columns of two
                        // positions: even columns to one operand, odd to the next
#pragma unroll
                        for (int hh = 0; hh < 2; ++hh) {
                            uint32_t x0, x1, y0, y1;
                            codes_to_f16(__byte_perm(vf[2 * hh], 0, 0x3120), x0, x1);
                            codes_to_f16(__byte_perm(vf[2 * hh + 1], 0, 0x3120), y0, y1);
                            add(acc[2 * (c + hh)], x0, y0);
                            add(acc[2 * (c + hh) + 1], x1, y1);
                        }
                    }
                }
            };
#pragma unroll
            for (int i = 0; i < N; ++i) {
                if (!ready(h[2 * i + 1])) return false;
                const uint32_t src = ring_addr + h[2 * i + 1].slot * Sh::kHalf;
                if constexpr (!EDGE) {
                    times_v(src, pf[i], std::false_type{}, 0u, 0u, true, true);
                } else if (there[i]) {
                    // A weight of 0 does not keep out a value that is not
                    // finite (a row that is not there holds anything): one
                    // token of the chunk at a time, with the values that it
                    // does not see taken out.
                    const int64_t p = p_first + (int64_t)(k + i) * kTile;
#pragma unroll 1
                    for (uint32_t ct = 0; ct < w.span.tokens; ++ct) {
                        auto keep = [&](uint32_t j) {
                            return ((there[i] >> j) & 1u) && sees(pos0 + ct, p + j);
                        };
                        auto pair = [&](uint32_t j) {
                            return (keep(j) ? 0xffffu : 0u) | (keep(j + 1) ? 0xffff0000u : 0u);
                        };
                        times_v(src, pf[i], std::true_type{}, pair(2 * in_quad),
                                pair(2 * in_quad + 8), t0 == ct, t1 == ct);
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.empty[h[2 * i + 1].slot]);
            }
            return true;
        };
        // tiles [even0, even1) of the segment: this warp's slices are seen by
        // every row of the block alike
        const uint32_t count = w.last - w.first;
        const int64_t lo_gap = all_lo - p_first, hi_gap = all_hi + 1 - kSlice - p_first;
        const uint32_t even0 = lo_gap <= 0 ? 0u : (uint32_t)((lo_gap + kTile - 1) / kTile);
        const uint32_t even1 = hi_gap < 0 ? 0u : (uint32_t)(hi_gap / kTile) + 1;
        using One = std::integral_constant<int, 1>;
        using Two = std::integral_constant<int, 2>;
        for (uint32_t k = 0; alive && k < count;) {
            alive = ready(at);
            if (!alive) break;
            if constexpr (NP == 2) {
                if (k >= even0 && k + 1 < count && k + 1 < even1) {
                    RingPos<Sh::kHalves> x = at;
                    x.step();
                    x.step();
                    alive = ready(x);
                    if (!alive) break;
                    if (full_slice(at) && full_slice(x)) {
                        alive = slices(k, Two{}, std::false_type{});
                        k += 2;
                        continue;
                    }
                }
            } else {
                if (k >= even0 && k < even1 && full_slice(at)) {
                    alive = slices(k, One{}, std::false_type{});
                    ++k;
                    continue;
                }
            }
            alive = slices(k, One{}, std::true_type{});
            ++k;
        }
        if (!alive) break;

        // ---- the four warps join, a few rows at a time
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
            l0 += __shfl_xor_sync(0xffffffffu, l0, o);
            l1 += __shfl_xor_sync(0xffffffffu, l1, o);
        }
        if (in_quad == 0) {
            sm.m[warp][r0] = m0;
            sm.m[warp][r1] = m1;
            sm.l[warp][r0] = l0;
            sm.l[warp][r1] = l1;
        }
        if constexpr (!Sh::kQInRegs) {  // Q's memory is free
            alive = meet();
            if (!alive) break;
        }
        const bool whole = w.whole();
        float* part = slot_of<DP>(a.workspace, blockIdx.x, w.first == 0 ? 1 : 0);
        const uint32_t quads = a.D / 4;
        constexpr uint32_t JR = Sh::kJoinRows;
#pragma unroll
        for (uint32_t round = 0; round < kRows / JR; ++round) {
            if (round * JR >= rows) break;
            if ((quad / JR) == (round & (8 / JR - 1))) {
                const bool high = HIGH && round >= 8 / JR;
                float* mine = s_join + (warp * JR + quad % JR) * DP;
#pragma unroll
                for (int n = 0; n < NT; n += 2) {
                    if constexpr (!FP8) {
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            *reinterpret_cast<float2*>(mine + 8 * (n + i) + 2 * in_quad) =
                                high ? make_float2(acc[n + i][2], acc[n + i][3])
                                     : make_float2(acc[n + i][0], acc[n + i][1]);
                    } else {
                        *reinterpret_cast<float4*>(mine + 8 * n + 4 * in_quad) =
                            high ? make_float4(acc[n][2], acc[n + 1][2], acc[n][3], acc[n + 1][3])
                                 : make_float4(acc[n][0], acc[n + 1][0], acc[n][1], acc[n + 1][1]);
                    }
                }
            }
            alive = meet();
            if (!alive) break;
            const uint32_t here = rows - round * JR < JR ? rows - round * JR : JR;
            for (uint32_t e = tid; e < here * quads; e += 32 * kWarps) {
                const uint32_t rj = e / quads, d = (e - rj * quads) * 4, r = round * JR + rj;
                float top = sm.m[0][r];
#pragma unroll
                for (int v = 1; v < kWarps; ++v) top = fmaxf(top, sm.m[v][r]);
                const float base = top == -INFINITY ? 0.0f : top;
                float l = 0.0f;
                float4 o = make_float4(0, 0, 0, 0);
#pragma unroll
                for (int v = 0; v < kWarps; ++v) {
                    const float f = fast_exp2(sm.m[v][r] - base);
                    const float4 x =
                        *reinterpret_cast<const float4*>(s_join + (v * JR + rj) * DP + d);
                    l += f * sm.l[v][r];
                    o.x += f * x.x;
                    o.y += f * x.y;
                    o.z += f * x.z;
                    o.w += f * x.w;
                }
                if (whole) {
                    const uint32_t ct = r / in_block;
                    const uint64_t row = (uint64_t)(w.t + ct) * a.Hq + head0 + (r - ct * in_block);
                    const float inv = l == 0.0f ? 0.0f : a.v_scale / l;
                    uint2 y;
                    y.x = pack_bf16x2(o.x * inv, o.y * inv);
                    y.y = pack_bf16x2(o.z * inv, o.w * inv);
                    *reinterpret_cast<uint2*>(a.out + row * a.D + d) = y;
                    if (d == 0 && a.lse)
                        a.lse[row] = l == 0.0f ? -INFINITY : (top + log2f(l)) * kLn2;
                } else {
                    *reinterpret_cast<float4*>(part + r * DP + d) = o;
                    if (d == 0) {
                        part[kRows * DP + r] = top;
                        part[kRows * DP + kRows + r] = l;
                    }
                }
            }
            alive = meet();
            if (!alive) break;
        }
        if (!alive) break;
        if (shared_by && tid == 0) {
            OpenPiece x;
            x.n = shared_by;
            x.t = w.t;
            x.tokens = w.span.tokens;
            x.block = block;
            *open = x;
        }
        w.next(a.split);
    }
    if (!alive && lane == 0) flag(a.err_flags, KVW_ERR_TIMEOUT);
}

template <int DP, bool FP8, bool MODS, bool HIGH, Hook HOOK>
cudaError_t launch_as(GqaArgs& a, const CacheMaps& maps, cudaStream_t stream) {
    constexpr size_t smem = sizeof(Smem<DP, FP8>);
    static_assert(smem <= 113 * 1024, "two CTAs per SM");
    uint64_t wave = 0;
    cudaError_t e = wave_ctas<&gqa_decode_kernel<DP, FP8, MODS, HIGH, HOOK>>(kThreads, smem, wave);
    if (e != cudaSuccess) return e;
    if (wave == 0) return cudaErrorInvalidConfiguration;
    const uint32_t ctas = side_by_side(a, wave);
    e = launch_early(&gqa_decode_kernel<DP, FP8, MODS, HIGH, HOOK>, dim3(ctas), kThreads, smem,
                     stream, a, maps);
    if (e != cudaSuccess) return e;
    return launch_join<DP>(a, ctas, stream);
}

template <int DP, bool FP8, Hook HOOK>
int launch(GqaArgs& a, const kvw_paged_cache_t* cache, uint32_t layer_idx, cudaStream_t stream) {
    CacheMaps maps;
    const int st = encode_cache_maps(&maps, cache, layer_idx, 2);
    if (st != KVW_OK) return st;
    const bool mods = a.softcap > 0.0f || a.slopes, high = (a.per_token << a.split.log_c) > 8;
    const cudaError_t e = mods ? (high ? launch_as<DP, FP8, true, true, HOOK>(a, maps, stream)
                                       : launch_as<DP, FP8, true, false, HOOK>(a, maps, stream))
                          : high ? launch_as<DP, FP8, false, true, HOOK>(a, maps, stream)
                                 : launch_as<DP, FP8, false, false, HOOK>(a, maps, stream);
    return e == cudaSuccess ? KVW_OK : KVW_ECUDA;
}

int gqa_entry(void* out, float* lse, const void* q, int64_t q_row_stride,
              const uint32_t* input_row_offsets, uint32_t num_batches, uint32_t tot_seq_len,
              uint32_t num_q_heads, const kvw_paged_cache_t* cache, float v_scale,
              uint32_t layer_idx, float sm_scale, float softcap, uint32_t window,
              const float* alibi_slopes, void* workspace, uint64_t workspace_bytes,
              uint32_t* err_flags, cudaStream_t stream, Hook hook, uint64_t wait_ns) {
    const int st = check_cache(cache, layer_idx, 2);
    if (st != KVW_OK) return st;
    GqaArgs a = {};
    const int bad = gqa_arguments(a, out, lse, q, q_row_stride, input_row_offsets, num_batches,
                                  tot_seq_len, num_q_heads, cache, sm_scale, softcap, window,
                                  alibi_slopes, workspace, workspace_bytes, err_flags,
                                  tma_sizes_ok(cache), value_scale_ok(cache, v_scale),
                                  tma_strides_ok(cache, 2));
    if (bad != KVW_OK || tot_seq_len == 0) return bad;
    const bool fp8 = cache->dtype == KVW_DTYPE_FP8_E4M3;
    a.k_scale = fp8 ? cache->scale : 1.0f;
    a.v_scale = fp8 ? v_scale : 1.0f;
    a.wait_limit = wait_cycles(wait_ns);
    auto run = [&](auto dp, auto f8) {
#ifdef KVW_TEST_HOOKS
        if (hook == Hook::kWithheld)
            return launch<decltype(dp)::value, decltype(f8)::value, Hook::kWithheld>(
                a, cache, layer_idx, stream);
        if (hook == Hook::kAbandoned)
            return launch<decltype(dp)::value, decltype(f8)::value, Hook::kAbandoned>(
                a, cache, layer_idx, stream);
#else
        if (hook != Hook::kNone) return (int)KVW_EUNSUPPORTED;
#endif
        return launch<decltype(dp)::value, decltype(f8)::value, Hook::kNone>(a, cache, layer_idx,
                                                                            stream);
    };
    using D64 = std::integral_constant<int, 64>;
    using D128 = std::integral_constant<int, 128>;
    using D256 = std::integral_constant<int, 256>;
    switch (padded_head(a.D)) {
        case 64: return fp8 ? run(D64{}, std::true_type{}) : run(D64{}, std::false_type{});
        case 128: return fp8 ? run(D128{}, std::true_type{}) : run(D128{}, std::false_type{});
        default: return fp8 ? run(D256{}, std::true_type{}) : run(D256{}, std::false_type{});
    }
}

}  // namespace
}  // namespace kvw

extern "C" int kva_gqa_decode_workspace(uint32_t num_q_heads, uint32_t num_kv_heads,
                                        uint32_t head_size, uint64_t* bytes) {
    return kvw::workspace_bytes_for(num_q_heads, num_kv_heads, head_size, bytes);
}

extern "C" int kva_gqa_decode_paged(void* out, float* lse, const void* q, int64_t q_row_stride,
                                    const uint32_t* input_row_offsets, uint32_t num_batches,
                                    uint32_t tot_seq_len, uint32_t num_q_heads,
                                    const kvw_paged_cache_t* cache, float v_scale,
                                    uint32_t layer_idx, float sm_scale, float softcap,
                                    uint32_t window, const float* alibi_slopes, void* workspace,
                                    uint64_t workspace_bytes, uint32_t* err_flags,
                                    cudaStream_t stream) {
    return kvw::gqa_entry(out, lse, q, q_row_stride, input_row_offsets, num_batches, tot_seq_len,
                          num_q_heads, cache, v_scale, layer_idx, sm_scale, softcap, window,
                          alibi_slopes, workspace, workspace_bytes, err_flags, stream,
                          kvw::Hook::kNone, kvw::kWaitLimitNs);
}

#ifdef KVW_TEST_HOOKS
// Test builds only (a separate library; the product has no such symbol): the
// first half tile of every CTA is announced on its barrier but never copied,
// and every wait is bounded by `wait_ns`, so the consumers' wait runs out,
// KVW_ERR_TIMEOUT is set and the kernel returns.
extern "C" int kva_test_gqa_decode_withheld(
    void* out, const void* q, int64_t q_row_stride, const uint32_t* input_row_offsets,
    uint32_t num_batches, uint32_t tot_seq_len, uint32_t num_q_heads,
    const kvw_paged_cache_t* cache, uint32_t layer_idx, void* workspace, uint64_t workspace_bytes,
    uint32_t* err_flags, cudaStream_t stream, uint64_t wait_ns) {
    return kvw::gqa_entry(out, nullptr, q, q_row_stride, input_row_offsets, num_batches,
                          tot_seq_len, num_q_heads, cache, 1.0f, layer_idx, 0.1f, 0.0f, 0, nullptr,
                          workspace, workspace_bytes, err_flags, stream, kvw::Hook::kWithheld,
                          wait_ns);
}

// The consumers leave at once, so nobody waits for the copies; err_flags[1]
// counts places whose last copy had not landed when the feeding warp left.
extern "C" int kva_test_gqa_decode_abandoned(
    void* out, const void* q, int64_t q_row_stride, const uint32_t* input_row_offsets,
    uint32_t num_batches, uint32_t tot_seq_len, uint32_t num_q_heads,
    const kvw_paged_cache_t* cache, uint32_t layer_idx, void* workspace, uint64_t workspace_bytes,
    uint32_t* err_flags, cudaStream_t stream, uint64_t wait_ns) {
    return kvw::gqa_entry(out, nullptr, q, q_row_stride, input_row_offsets, num_batches,
                          tot_seq_len, num_q_heads, cache, 1.0f, layer_idx, 0.1f, 0.0f, 0, nullptr,
                          workspace, workspace_bytes, err_flags, stream, kvw::Hook::kAbandoned,
                          wait_ns);
}
#endif
