// Attention of new tokens over the paged MLA latent cache.
//
// Mathematics, for one token and a block of up to 64 heads: every head reads
// the same rows (576 wide: 512 latent, 64 rotated), so one tile of 64
// positions serves all of them.  S = Q K^T (64 heads x 64 positions, 576
// deep); with the running maximum m and sum l of a softmax per head, P =
// 2^(S - m); and, turned around so that the 512 output columns fill the matrix
// unit's lanes, O^T += V^T P^T (512 x 64, 64 positions deep), V being the
// first 512 columns of the same tile in shared memory.  m follows the maximum
// only when that has risen by more than 2^6, so O^T is rescaled seldom, and
// stays 2^9 below it for the fp16 weights of an E4M3 cache (kva_attention.cuh).
//
// Bound: 64 heads do 121 flops per byte of a bf16 row (242 with both blocks
// of 128 heads, whose two CTAs read the same piece at the same time and meet
// in L2), close to the ridge of the card: both HBM and the matrix unit's
// operand bandwidth matter.  The products are tcgen05 MMAs on tiles that the
// copy engine writes in the operands' own swizzled layout, page by page, so a
// bf16 row goes from HBM to the matrix unit without passing a register.
//
// An E4M3 cache keeps its codes for S: the query row, scaled by a power of
// two, is the sum of two E4M3 numbers (4 + 4 significant bits are bf16's 8),
// x = q1 + q2 / 16, so q1 fills rows 32w .. 32w + 15 and q2 rows 32w + 16 ..
// 32w + 31 of one 128-row operand and S = S1 + S2 / 16; products of two E4M3
// numbers are exact in fp32.  The sum is exact down to 2^-21 of the row's
// largest value.  Weights need more than E4M3 has, so four warps turn the
// value columns into fp16 (exactly) for O^T.
//
// Shared memory (227 KB) decides the rest.  bf16: Q 72 KB and two tiles of 72
// KB, each in three groups of panels that are filled one by one and freed as
// the row blocks of O^T complete.  E4M3: Q's two parts 72 KB, two tiles of
// codes 80 KB, one fp16 tile of values 64 KB in two halves.  P 8 KB.  O^T
// fills 256 of the 512 columns of tensor memory, two S tiles 128.  What is
// ready goes first, the next S or the next O^T, so that neither a late tile nor
// a late softmax holds up the other.
//
// Measured, contexts of up to 8192 positions: 256 requests, 128 heads, bf16
// 408 us (720 TF/s, 39 % of the card's matrix rate), E4M3 456 us; 64 heads,
// bf16 225 us (5.6 TB/s, 82 % of its copy rate), E4M3 250; 16 heads 204 and 220;
// one token, 16 heads, 1501 positions 14.7 us.  A tile of 64 positions takes some 3700 cycles, of which
// the products fill 1900: with 64 rows a 16-deep step of S reads 2 KB of Q and
// 2 KB of K from shared memory at 128 bytes a cycle, and a step of O^T 4 KB
// and 2 KB.  The rest is the round of a tile's place (copy 1600 cycles, S 1400,
// softmax 1250, O^T 900, two places), and for E4M3 the round of the values'
// (conversion 1900, O^T 1200, one place).  Steps of 32 positions, four places,
// took 581 and 658 us: S costs as much for 32 as for 64.
//
// Warps: 0-3 softmax, rescaling, results; 5 issues the MMAs; 4 and (several)
// the last ones feed; 6-9 (E4M3) convert values.  Every wait is bounded.
#include <cstdint>
#include <type_traits>

#include "kva_attention.cuh"
#include "kva_split.cuh"
#include "kva_tcgen05.cuh"
#include "kva_tma.cuh"

namespace kvw {
namespace {

constexpr uint32_t kHeads = 64;               // rows of a row block
constexpr uint32_t kLatent = 512, kRow = 576;
constexpr uint32_t kPanel = kTile * 128;      // 64 columns of a 16-bit tile, or 128 codes
constexpr uint32_t kGroups = 3;               // of a bf16 tile: three of its nine panels each
constexpr uint32_t kCodePanels = 5;           // of an E4M3 tile: 64 rotated columns, 4 x 128 latent ones
constexpr uint32_t kCodeGroups = 2;           // panels 0 - 2 and 3, 4
constexpr uint32_t kMaxCtas = 192;
constexpr uint32_t kTmemColumns = 512, kScoreColumn = 256;
constexpr int kSoftmaxThreads = 128;

struct MlaArgs {
    SplitArgs split;
    uint16_t* out;
    float* lse;
    const uint16_t *q_latent, *q_rope;
    int64_t q_latent_stride, q_rope_stride;
    const uint32_t* page_table;
    uint32_t* err_flags;
    unsigned char* workspace;
    float scale;      // sm_scale * log2(e) * row_scale
    float row_scale;  // what a cache element stands for: its code times this
    uint32_t H, HB, slot_rows;  // heads, row blocks, rows of a workspace slot
    uint32_t num_pages, max_pages, pieces;
    FastDiv ps;
    int64_t wait_limit;  // cycles
};

struct QMaps {
    CUtensorMap latent, rope, panels;
};

// WHOLE: a tile lies in one page (64 divides the page size).
// Feeding warps: small pages make many copies, and issuing them was most of a
// tile's time (256 requests, 128 heads, pages of 16: bf16 with three warps 441
// us, two 535, one 772; E4M3 with two 491, one 540).  Of whole tiles two (bf16)
// or one (E4M3) are enough, and more warps cost (bf16: three 413 us, two 407).
template <bool FP8, bool WHOLE>
constexpr uint32_t feeders_of() {
    return FP8 ? (WHOLE ? 1 : 2) : WHOLE ? 2 : 3;
}
template <bool FP8, bool WHOLE>
constexpr int threads_of() {
    return 32 * ((FP8 ? 9 : 5) + feeders_of<FP8, WHOLE>());
}

template <bool FP8, bool WHOLE>
struct Smem {
    // bf16: Q as nine panels, rotated columns last.  E4M3: four panels of 128
    // rows x 128 codes, then 128 rows x 64 rotated columns in 64-byte lines.
    unsigned char q[9 * kPanel];
    unsigned char p[kPanel];
    // two tiles as they come: nine panels each, or five of codes
    unsigned char kv[2 * (FP8 ? kCodePanels : 9) * kPanel];
    unsigned char values[FP8 ? 8 * kPanel : 16];  // E4M3: the value columns in fp16
    uint64_t full[2 * kGroups], empty[2 * kGroups];  // groups of the two tiles
    uint64_t v_full[2], v_empty[2];                  // halves of `values`
    uint64_t q_full, q_ready, q_free;
    uint64_t s_full[2], p_full, pv_done, o_free, drained;
    uint64_t there[8];  // of a tile: positions that are there
    float alpha[kHeads], m[kHeads], l[kHeads], q_scale[kHeads];
    SplitShared<threads_of<FP8, WHOLE>()> split;
    uint32_t tmem, stop;
};

// The panels of a tile: eight of the latent columns, then the rotated ones;
// of codes the rotated columns, then four of the latent ones.  Group g: its
// first panel and their number.
template <bool FP8>
__device__ __forceinline__ uint32_t group_start(uint32_t g) { return 3u * g; }
template <bool FP8>
__device__ __forceinline__ uint32_t group_panels(uint32_t g) { return FP8 && g ? 2u : 3u; }

// Do any of the softmax threads say yes?
__device__ __forceinline__ bool any_softmax(bool mine) {
    uint32_t all;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, 1, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(all)
        : "r"((uint32_t)mine)
        : "memory");
    return all != 0;
}

// A workspace slot: `rows` x 512 sums, then their maxima and sums of weights,
// in whole 16-byte vectors.
__host__ __device__ __forceinline__ uint32_t slot_floats(uint32_t rows) {
    return (rows * (kLatent + 2) + 3u) & ~3u;
}
__device__ __forceinline__ float* slot_of(const MlaArgs& a, uint32_t cta, uint32_t s) {
    return reinterpret_cast<float*>(a.workspace + kMaxCtas * sizeof(OpenPiece)) +
           (uint64_t)(2 * cta + s) * slot_floats(a.slot_rows);
}

// ---------------------------------------------------------------- feeding

// Of pages of whole tiles a group is one copy of three panels; three copies of
// one panel each took 433 us instead of 411 when it was changed.
template <bool FP8, bool WHOLE, Hook HOOK, uint32_t WHICH>
__device__ __forceinline__ void feed(const MlaArgs& a, const CacheMaps& maps, const QMaps& qm,
                                     Smem<FP8, WHOLE>& sm) {
    constexpr uint32_t kTileGroups = FP8 ? kCodeGroups : kGroups;
    constexpr uint32_t kTilePanels = FP8 ? kCodePanels : 9;
    constexpr int kUnroll = FP8 ? 8 : 1;
    // of one warp all groups, of as many as groups one each, of two for three
    // groups the first two and the last
    constexpr uint32_t kWarps = feeders_of<FP8, WHOLE>();
    constexpr uint32_t kFrom = WHICH == 0 ? 0 : WHICH + kTileGroups - kWarps;
    constexpr uint32_t kTo = WHICH + 1 + kTileGroups - kWarps;
    const uint32_t lane = threadIdx.x & 31u, hb = blockIdx.x % a.HB;
    auto column = [](uint32_t panel) {
        return FP8 ? (panel == 0 ? kLatent : (panel - 1) * 128u) : panel * 64u;
    };
    Walk w;
    w.begin(a.split, sm.split.start);
    uint32_t bad_page = 0, tile = 0, segment = 0;
    uint32_t stopped_at = kFrom;  // the group whose place was not free in time
    bool ok = true;
    while (ok && !w.done()) {
        prefetch_page(maps, a.page_table, a.max_pages, a.ps, w.b,
                      (int64_t)(w.span.tile0 + w.first) * kTile, lane);
        if constexpr (!FP8 && WHICH == kWarps - 1) {
            ok = wait_phase(&sm.q_free, (segment & 1u) ^ 1u, &sm.stop, a.wait_limit);
            if (!ok) break;
            if (elect_one()) {
                const uint32_t bar = smem_addr(&sm.q_full);
                mbar_arrive_expect_tx(&sm.q_full, 9 * kPanel);
                tma_3d(smem_addr(sm.q + 8 * kPanel), &qm.rope, 0, hb * kHeads, w.t, bar);
#pragma unroll kUnroll
                for (uint32_t x = 0; x < 8; ++x)
                    tma_3d(smem_addr(sm.q + x * kPanel), &qm.latent, x * 64, hb * kHeads, w.t,
                           bar);
            }
            __syncwarp();
            ++segment;
        }
        TilePlan t;
        uint32_t row = 0, page = 0;  // of a tile that is one copy
        auto plan = [&](uint32_t i) {
            plan_tile(maps, a.page_table, a.max_pages, a.num_pages, a.ps, w.b,
                      (int64_t)(w.span.tile0 + i) * kTile, w.span.start, w.span.hi, t, bad_page);
            row = __shfl_sync(0xffffffffu, t.copy[0].row, 0);
            page = __shfl_sync(0xffffffffu, t.copy[0].page, 0);
        };
        plan(w.first);
        for (uint32_t i = w.first; ok && i < w.last; ++i) {
#pragma unroll kUnroll
            for (uint32_t g = kFrom; g < kTo; ++g) {
                uint64_t* full = &sm.full[(tile & 1u) * kTileGroups + g];
                if (ok) {
                    stopped_at = g;
                    ok = wait_phase(&sm.empty[(tile & 1u) * kTileGroups + g],
                                    ((tile >> 1) & 1u) ^ 1u, &sm.stop, a.wait_limit);
                }
                if (!ok) continue;
                const uint32_t bytes = (t.n << maps.log_rows) * 128u * group_panels<FP8>(g);
                const uint32_t bar = smem_addr(full);
                const uint32_t base = smem_addr(
                    sm.kv + ((tile & 1u) * kTilePanels + group_start<FP8>(g)) * kPanel);
                const bool withheld = HOOK == Hook::kWithheld && tile == 0 && g == 0;
                if constexpr (WHOLE) {
                    if (elect_one()) {
                        if (g == 0) sm.there[tile & 7u] = ((uint64_t)t.t_hi << 32) | t.t_lo;
                        mbar_arrive_expect_tx(full, bytes);
                        if (t.n && !withheld) {
                            if constexpr (!FP8) {
                                tma_4d(base, &qm.panels, 0, row, 3 * g, page, bar);
                            } else {
                                if (g == 0)
                                    tma_rows(base, &maps.map[0], kLatent, 0, row, page, 0, bar);
                                tma_4d(base + (g == 0 ? kPanel : 0), &qm.panels, 0, row, 2 * g,
                                       page, bar);
                            }
                        }
                    }
                    __syncwarp();
                } else {
                    if (lane == 0) {
                        if (g == 0) sm.there[tile & 7u] = ((uint64_t)t.t_hi << 32) | t.t_lo;
                        mbar_arrive_expect_tx(full, bytes);
                    }
                    __syncwarp();
                    if (!withheld)
                        each_copy(maps, t, [&](uint32_t unit, uint32_t r, uint32_t id,
                                                  const CUtensorMap* map) {
#pragma unroll kUnroll
                            for (uint32_t x = 0; x < group_panels<FP8>(g); ++x)
                                tma_rows(base + x * kPanel + (unit << maps.log_rows) * 128u, map,
                                         column(group_start<FP8>(g) + x), 0, r, id, 0, bar);
                        });
                }
            }
            if (!ok) break;
            ++tile;
            stopped_at = kFrom;
            if (i + 1 < w.last) {
                // The next tile's place is taken for a while yet: into L2 with
                // it (256 requests, 128 heads, when it was added: bf16 472 ->
                // 453 us; a tile of codes by whole panels 470 -> 465, panel by
                // panel no gain; two tiles ahead is no better than one).
                plan(i + 1);
                if ((i & 1u) == hb || a.HB == 1) {
                    if constexpr (WHOLE) {
                        if (t.n && elect_one()) {
#pragma unroll 1
                            for (uint32_t g = kFrom; g < kTo; ++g)
                                tma_4d_prefetch(&qm.panels, 0, row, (FP8 ? 2 : 3) * g, page);
                            if constexpr (FP8)
                                tma_prefetch(&maps.map[0], kLatent, 0, row, page, 0);
                        }
                        __syncwarp();
                    } else {
                        each_copy(maps, t, [&](uint32_t, uint32_t r, uint32_t id,
                                                  const CUtensorMap* map) {
#pragma unroll 1
                            for (uint32_t x = group_start<FP8>(kFrom);
                                 x < group_start<FP8>(kTo - 1) + group_panels<FP8>(kTo - 1); ++x)
                                tma_prefetch(map, column(x), 0, r, id, 0);
                        });
                    }
                }
            }
        }
        if (ok) w.next(a.split);
    }
    if (bad_page) flag(a.err_flags, KVW_ERR_PAGE);
    if (!ok && lane == 0) flag(a.err_flags, KVW_ERR_TIMEOUT);
    // Whether or not this warp had to wait in vain: it leaves when the last copy
    // into each place has landed, or after a bounded time.
#pragma unroll 1
    for (uint32_t buf = 0; buf < 2; ++buf)
#pragma unroll 1
        for (uint32_t g = kFrom; g < kTo; ++g) {
            const uint32_t issued = (tile + (g < stopped_at) + 1 - buf) >> 1;  // into this place
            if (issued)
                leave_phase<HOOK>(&sm.full[buf * kTileGroups + g], (issued - 1) & 1u,
                                  a.wait_limit, a.err_flags);
        }
    if (!FP8 && segment)
        leave_phase<HOOK>(&sm.q_full, (segment - 1) & 1u, a.wait_limit, a.err_flags);
}

// ---------------------------------------------------------------- converting

// Codes of the value columns -> fp16 panels in the operands' layout; positions
// that are not there become zeros.
template <bool WHOLE>
__device__ __forceinline__ void convert(const MlaArgs& a, Smem<true, WHOLE>& sm) {
    const uint32_t lane = threadIdx.x & 31u, i0 = threadIdx.x - 192u, c = i0 & 7u;
    Walk w;
    w.begin(a.split, sm.split.start);
    uint32_t tile = 0;
    bool ok = true;
    while (ok && !w.done()) {
        for (uint32_t i = w.first; ok && i < w.last; ++i, ++tile) {
            const uint32_t buf = tile & 1u;
#pragma unroll 1
            for (uint32_t g = 0; g < 4; ++g) {  // 128 columns each
                const uint32_t slot = buf * kCodeGroups + (g >> 1);
                if (!(g & 1u))
                    ok = wait_phase(&sm.full[slot], (tile >> 1) & 1u, &sm.stop, a.wait_limit);
                if (!ok) break;
                const uint64_t there = sm.there[tile & 7u];
                const unsigned char* src = sm.kv + (buf * kCodePanels + 1 + g) * kPanel;
                uint4 v[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint32_t r = (i0 >> 3) + 16u * k;
                    v[k] = *reinterpret_cast<const uint4*>(src + r * 128u + (((c ^ r) & 7u) << 4));
                }
                if (!(g & 1u))
                    ok = wait_phase(&sm.v_empty[g >> 1], (tile & 1u) ^ 1u, &sm.stop, a.wait_limit);
                if (!ok) break;
                unsigned char* dst = sm.values + 2 * g * kPanel;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint32_t r = (i0 >> 3) + 16u * k;
                    if (!((there >> r) & 1ull)) v[k] = make_uint4(0, 0, 0, 0);
                    uint4 x, y;
                    codes_to_f16(v[k].x, x.x, x.y);
                    codes_to_f16(v[k].y, x.z, x.w);
                    codes_to_f16(v[k].z, y.x, y.y);
                    codes_to_f16(v[k].w, y.z, y.w);
                    // 16 codes are two chunks of the row's line; chunks 4-7 of
                    // the codes go to the second panel and store their odd
                    // chunk first, so that the eight lanes of a row hit
                    // distinct banks
                    const uint32_t o = 2u * (c & 3u), odd = c >> 2;
                    unsigned char* line = dst + (c >> 2) * kPanel + r * 128u;
                    *reinterpret_cast<uint4*>(line + (((o + odd) ^ (r & 7u)) << 4)) = odd ? y : x;
                    *reinterpret_cast<uint4*>(line + (((o + (odd ^ 1u)) ^ (r & 7u)) << 4)) =
                        odd ? x : y;
                }
                if (g & 1u) {
                    fence_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(&sm.v_full[g >> 1]);
                        mbar_arrive(&sm.empty[slot]);
                    }
                }
            }
        }
        if (ok) w.next(a.split);
    }
}

// ---------------------------------------------------------------- products

// What the issuing thread of a bf16 cache keeps of its place: the next
// group of S and the next O^T.  O^T goes first: it frees a tile's place, S only
// takes one.  S runs at most two tiles ahead of O^T (its two buffers).  One
// loop with one copy of either product: with the MMAs of a tile unrolled, and
// more so with several copies of O^T, the loop's time was that of fetching its
// instructions.
struct Products {
    Walk w;
    uint32_t s_tile = 0, o_tile = 0, group = 0, i = 0, s_segment = 0;
    // of the tiles between S and O^T, by the parity of the tile: is it the
    // first of its segment, and the parity of that
    uint32_t firsts = 0, odd_segments = 0;

    __device__ __forceinline__ bool more(const MlaArgs&) const {
        return !w.done() || o_tile < s_tile;
    }
    __device__ __forceinline__ bool s_next() const { return !w.done() && s_tile - o_tile < 2; }
    __device__ __forceinline__ bool last_of_segment() const { return i + 1 == w.last - w.first; }
    __device__ __forceinline__ void s_done(const MlaArgs& a) {
        const uint32_t bit = 1u << (s_tile & 1u);
        firsts = i == 0 ? firsts | bit : firsts & ~bit;
        odd_segments = s_segment & 1u ? odd_segments | bit : odd_segments & ~bit;
        ++s_tile;
        group = 0;
        if (last_of_segment()) {
            i = 0;
            ++s_segment;
            w.next(a.split);
        } else {
            ++i;
        }
    }
    __device__ __forceinline__ bool first() const { return (firsts >> (o_tile & 1u)) & 1u; }
    __device__ __forceinline__ uint32_t odd() const { return (odd_segments >> (o_tile & 1u)) & 1u; }
};

// The products of a bf16 cache: one thread issues every MMA.  (Fences only
// where tensor memory passes between threads: operands in shared memory come
// with their barriers.)
template <bool WHOLE>
__device__ __forceinline__ void multiply(const MlaArgs& a, Smem<false, WHOLE>& sm) {
    const uint32_t hb = blockIdx.x % a.HB, tmem = sm.tmem;
    const uint32_t rows = a.H - hb * kHeads < kHeads ? a.H - hb * kHeads : kHeads;
    const uint32_t cols = (rows + 15u) & ~15u;  // of O^T
    constexpr uint32_t qk_instr = f16_instr(true, 0, 0, kHeads, kTile);
    const uint32_t pv_instr = f16_instr(true, 1, 0, 128, cols);
    const uint32_t q_op = operand_low(smem_addr(sm.q), 0);
    const uint32_t k_op = operand_low(smem_addr(sm.kv), 0);
    const uint32_t v_op = operand_low(smem_addr(sm.kv), kPanel);
    const uint32_t p_op = operand_low(smem_addr(sm.p), 0);
    if (elect_one()) {
        Products x;
        x.w.begin(a.split, sm.split.start);
        bool ok = true;
        int64_t t0 = 0;
        uint32_t tries = 0;
        while (ok && x.more(a)) {
            if (x.o_tile < x.s_tile && phase_done(&sm.p_full, x.o_tile & 1u)) {
                // O^T (+)= V^T P^T
                const uint32_t buf = x.o_tile & 1u;
                if (x.first())
                    ok = wait_one(&sm.o_free, x.odd() ^ 1u, &sm.stop, a.wait_limit);
                fence_after_sync();
                uint32_t d = tmem, v = v_op + ((buf * 9 * kPanel) >> 4);
                uint64_t* empty = &sm.empty[buf * kGroups];
                const bool add = !x.first();
#pragma unroll 1
                for (uint32_t j = 0; ok && j < 4; ++j) {
#pragma unroll
                    for (uint32_t ks = 0; ks < 4; ++ks)
                        mma_f16_ss(d, v + ((ks * 2048u) >> 4), p_op + ((ks * 32u) >> 4), pv_instr,
                                   add || ks > 0);
                    // panels 0-2, 3-5, 6-8: block j takes 2j and 2j + 1
                    if (j > 0) mma_commit(empty++);
                    d += kHeads;
                    v += (2 * kPanel) >> 4;
                }
                mma_commit(&sm.pv_done);
                ++x.o_tile;
                tries = 0;
            } else if (x.s_next() &&
                       phase_done(&sm.full[(x.s_tile & 1u) * kGroups + x.group],
                                  (x.s_tile >> 1) & 1u) &&
                       (x.i > 0 || phase_done(&sm.q_full, x.s_segment & 1u))) {
                // a group of S.  Its buffer is free: S of tile n - 2 was read
                // before the weights of that tile were written, and those have
                // been waited for.
                const uint32_t buf = x.s_tile & 1u, d = tmem + kScoreColumn + buf * kTile;
                uint32_t at = (group_start<false>(x.group) * kPanel) >> 4;
                const uint32_t k = k_op + ((buf * 9 * kPanel) >> 4);
                const uint32_t end = at + ((group_panels<false>(x.group) * kPanel) >> 4);
#pragma unroll 1
                for (; at < end; at += kPanel >> 4)
#pragma unroll
                    for (uint32_t ks = 0; ks < 4; ++ks)
                        mma_f16_ss(d, q_op + at + ks * 2u, k + at + ks * 2u, qk_instr,
                                   at > 0 || ks > 0);
                if (++x.group == kGroups) {
                    mma_commit(&sm.s_full[buf]);
                    if (x.last_of_segment()) mma_commit(&sm.q_free);
                    x.s_done(a);
                }
                tries = 0;
            } else if ((++tries & 63u) == 0) {
                if (tries == 64u) t0 = clock64();
                if (clock64() - t0 > a.wait_limit)
                    *reinterpret_cast<volatile uint32_t*>(&sm.stop) = 1;
                if (*reinterpret_cast<volatile uint32_t*>(&sm.stop)) ok = false;
            }
        }
        if (!ok) flag(a.err_flags, KVW_ERR_TIMEOUT);
        // what was issued finishes before tensor and shared memory go, also where
        // the softmax warps, who wait for it, gave up
        mma_commit(&sm.drained);
        drain_phase(&sm.drained, 0, a.wait_limit);
    }
    __syncwarp();
}

// The products of an E4M3 cache: a warp whose elected thread issues.
template <bool WHOLE>
__device__ __forceinline__ void multiply_codes(const MlaArgs& a, Smem<true, WHOLE>& sm) {
    const uint32_t hb = blockIdx.x % a.HB, tmem = sm.tmem;
    const uint32_t rows = a.H - hb * kHeads < kHeads ? a.H - hb * kHeads : kHeads;
    const uint32_t cols = (rows + 15u) & ~15u;  // of O^T
    constexpr uint32_t qk_instr = e4m3_instr(128, kTile);
    const uint32_t pv_instr = f16_instr(false, 1, 0, 128, cols);
    const uint32_t q_op = operand_low(smem_addr(sm.q), 0);
    const uint32_t k_op = operand_low(smem_addr(sm.kv), 0);
    const uint32_t v_op = operand_low(smem_addr(sm.values), kPanel);
    const uint32_t p_op = operand_low(smem_addr(sm.p), 0);
    Walk w;
    w.begin(a.split, sm.split.start);
    bool ok = true;

    auto all_done = [&](uint64_t* bar, uint32_t parity) {
        return __all_sync(0xffffffffu, phase_done(bar, parity)) != 0;
    };
    // S of tile n (its buffer is free as in multiply)
    auto scores = [&](uint32_t n) {
        const uint32_t buf = n & 1u;
        const uint32_t k_tile = k_op + ((buf * kCodePanels * kPanel) >> 4);
        const uint32_t d = tmem + kScoreColumn + buf * kTile;
#pragma unroll
        for (uint32_t g = 0; g < kCodeGroups; ++g) {
            const uint32_t slot = buf * kCodeGroups + g;
            if (!wait_phase(&sm.full[slot], (n >> 1) & 1u, &sm.stop, a.wait_limit)) return false;
            if (elect_one()) {
                if (g == 0) {  // rotated columns: 64-byte lines of Q behind its panels
#pragma unroll
                    for (uint32_t ks = 0; ks < 2; ++ks)
                        mma_e4m3_ss<kOperandHigh64>(d, q_op + ((8 * kPanel + ks * 32u) >> 4),
                                                    k_tile + ((ks * 32u) >> 4), qk_instr, ks > 0);
                }
#pragma unroll
                for (uint32_t x = 0; x < 2; ++x)
#pragma unroll
                    for (uint32_t ks = 0; ks < 4; ++ks)
                        mma_e4m3_ss<kOperandHigh>(
                            d, q_op + (((2 * g + x) * 2 * kPanel + ks * 32u) >> 4),
                            k_tile + (((1 + 2 * g + x) * kPanel + ks * 32u) >> 4), qk_instr, true);
                mma_commit(&sm.empty[slot]);
                if (g == kCodeGroups - 1) mma_commit(&sm.s_full[buf]);
            }
            __syncwarp();
        }
        return true;
    };
    // O^T (+)= V^T P^T of tile n, the `first` of a segment or not; `odd`: the
    // segment's parity
    auto values = [&](uint32_t n, bool first, uint32_t odd) {
        if (first && !wait_phase(&sm.o_free, odd ^ 1u, &sm.stop, a.wait_limit)) return false;
        if (!wait_phase(&sm.p_full, n & 1u, &sm.stop, a.wait_limit)) return false;
        fence_after_sync();
#pragma unroll
        for (uint32_t j = 0; j < 4; ++j) {
            if (!(j & 1u) &&
                !wait_phase(&sm.v_full[j >> 1], n & 1u, &sm.stop, a.wait_limit))
                return false;
            if (elect_one()) {
#pragma unroll
                for (uint32_t ks = 0; ks < 4; ++ks)
                    mma_f16_ss(tmem + j * kHeads, v_op + ((2 * j * kPanel + ks * 2048u) >> 4),
                               p_op + ((ks * 32u) >> 4), pv_instr, !first || ks > 0);
                if (j & 1u) mma_commit(&sm.v_empty[j >> 1]);
                if (j == 3) mma_commit(&sm.pv_done);
            }
            __syncwarp();
        }
        return true;
    };

    // S runs at most two tiles ahead of O^T (its two buffers).  Whichever is
    // ready goes first.
    uint32_t s_tile = 0, o_tile = 0, s_segment = 0, i = 0;
    // of the tiles between S and O^T, by the parity of the tile: is it the
    // first of its segment, and the parity of that
    uint32_t firsts = 0, odd_segments = 0;
    while (ok && (!w.done() || o_tile < s_tile)) {
        const uint32_t pending = s_tile - o_tile;
        bool take_s = !w.done() && pending < 2;
        if (take_s && pending > 0) {
            // both are possible: wait for either
            const uint32_t slot = (s_tile & 1u) * kCodeGroups + kCodeGroups - 1;
            const int64_t t0 = clock64();
            while (true) {
                if (all_done(&sm.p_full, o_tile & 1u)) {
                    take_s = false;
                    break;
                }
                if (all_done(&sm.full[slot], (s_tile >> 1) & 1u) &&
                    (i > 0 || all_done(&sm.q_ready, s_segment & 1u)))
                    break;
                bool give_up = *reinterpret_cast<volatile uint32_t*>(&sm.stop) != 0;
                if (clock64() - t0 > a.wait_limit) {
                    *reinterpret_cast<volatile uint32_t*>(&sm.stop) = 1;
                    give_up = true;
                }
                if (__any_sync(0xffffffffu, give_up)) {
                    ok = false;
                    break;
                }
            }
            if (!ok) break;
        }
        if (take_s) {
            if (i == 0) ok = wait_phase(&sm.q_ready, s_segment & 1u, &sm.stop, a.wait_limit);
            if (!ok) break;
            ok = scores(s_tile);
            const uint32_t bit = 1u << (s_tile & 1u);
            firsts = i == 0 ? firsts | bit : firsts & ~bit;
            odd_segments = s_segment & 1u ? odd_segments | bit : odd_segments & ~bit;
            ++s_tile;
            if (++i == w.last - w.first) {
                i = 0;
                ++s_segment;
                w.next(a.split);
            }
        } else {
            ok = values(o_tile, (firsts >> (o_tile & 1u)) & 1u, (odd_segments >> (o_tile & 1u)) & 1u);
            ++o_tile;
        }
    }
    // what was issued finishes before tensor and shared memory go, also where the
    // softmax warps, who wait for it, gave up
    if (elect_one()) {
        if (!ok) flag(a.err_flags, KVW_ERR_TIMEOUT);
        mma_commit(&sm.drained);
    }
    __syncwarp();
    drain_phase(&sm.drained, 0, a.wait_limit);
}

// ---------------------------------------------------------------- softmax

// Two scaled bf16 values in fp16 -> their E4M3 parts, two codes each: x = q1 +
// q2 / 16.  In fp16 all of it is exact but the two roundings to E4M3.
__device__ __forceinline__ void split_pair(uint32_t x, uint32_t& q1, uint32_t& q2) {
    asm("{\n\t.reg .b16 a, b;\n\t.reg .b32 y, z;\n\t"
        "cvt.rn.satfinite.e4m3x2.f16x2 a, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 y, a;\n\t"
        "mul.rn.f16x2 z, %2, %3;\n\t"
        "fma.rn.f16x2 z, y, %4, z;\n\t"
        "cvt.rn.satfinite.e4m3x2.f16x2 b, z;\n\t"
        "cvt.u32.u16 %0, a;\n\tcvt.u32.u16 %1, b;\n\t}"
        : "=r"(q1), "=r"(q2)
        : "r"(x), "r"(0x4c004c00u), "r"(0xcc00cc00u));  // 16, -16
}

// The queries of a segment as two E4M3 parts: row h scaled by a power of two
// so that its largest value lies in [128, 256), x = q1 + q2 / 16 with q1 the
// nearest E4M3 number and q2 the remainder, exact while q1's step is not
// below E4M3's smallest (2^-9).  A row with an infinity or a NaN becomes NaN
// (E4M3 has no infinity; its scores are not finite either way).  The heads go
// round the warps, a warp taking four of them at a time with the next four on
// their way, its lanes the 72 chunks of 8 values of a row.
template <bool WHOLE>
__device__ __forceinline__ void split_queries(const MlaArgs& a, Smem<true, WHOLE>& sm, uint32_t t,
                                              uint32_t head0, uint32_t rows) {
    const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31u;
    constexpr int kAtOnce = 4;
    auto load = [&](uint32_t h0, uint4(&v)[kAtOnce][3]) {
#pragma unroll
        for (int n = 0; n < kAtOnce; ++n) {
            const uint32_t h = h0 + n;
            const uint16_t* ql = a.q_latent + (int64_t)t * a.q_latent_stride +
                                 (int64_t)(head0 + h) * kLatent;
            const uint16_t* qr = a.q_rope + (int64_t)t * a.q_rope_stride + (int64_t)(head0 + h) * 64;
#pragma unroll
            for (int k = 0; k < 3; ++k) {
                const uint32_t c = lane + 32u * k;
                v[n][k] = make_uint4(0, 0, 0, 0);
                if (h < rows && c < 72)
                    v[n][k] = __ldg(reinterpret_cast<const uint4*>(c < 64 ? ql + c * 8
                                                                          : qr + (c - 64) * 8));
            }
        }
    };
    uint4 ahead[kAtOnce][3];
    load(warp * kAtOnce, ahead);
#pragma unroll 1
    for (uint32_t h0 = warp * kAtOnce; h0 < rows; h0 += 4 * kAtOnce) {
        uint4 v[kAtOnce][3];
#pragma unroll
        for (int n = 0; n < kAtOnce; ++n)
#pragma unroll
            for (int k = 0; k < 3; ++k) v[n][k] = ahead[n][k];
        load(h0 + 4 * kAtOnce, ahead);
#pragma unroll
        for (int n = 0; n < kAtOnce; ++n) {
            uint32_t top = 0;
#pragma unroll
            for (int k = 0; k < 3; ++k)
                top = __vmaxu2(top, __vmaxu2(__vmaxu2(v[n][k].x & 0x7fff7fffu, v[n][k].y & 0x7fff7fffu),
                                             __vmaxu2(v[n][k].z & 0x7fff7fffu, v[n][k].w & 0x7fff7fffu)));
            top = max(top & 0xffffu, top >> 16);
            top = __reduce_max_sync(0xffffffffu, top);
            float up, down;
            row_power(top, up, down);  // to [2^14, 2^15)
            up = (top >> 7) == 255u ? __int_as_float(0x7fffffff) : up * 0x1p-7f;
            down *= 0x1p7f;
            const uint32_t h = h0 + n;  // below 64: rows past the last head are zeros
            const uint32_t r1 = 32u * (h >> 4) + (h & 15u), r2 = r1 + 16u;
            if (lane == 0) sm.q_scale[h] = down;
#pragma unroll
            for (int k = 0; k < 3; ++k) {
                const uint32_t c = lane + 32u * k;
                if (c >= 72) continue;
                auto part = [&](uint32_t x, uint32_t& q1, uint32_t& q2) {
                    split_pair(pack2<true>(bf16_lo(x) * up, bf16_hi(x) * up), q1, q2);
                };
                uint32_t lo1, lo2, hi1, hi2;
                uint2 q1, q2;
                part(v[n][k].x, lo1, lo2);
                part(v[n][k].y, hi1, hi2);
                q1.x = lo1 | (hi1 << 16);
                q2.x = lo2 | (hi2 << 16);
                part(v[n][k].z, lo1, lo2);
                part(v[n][k].w, hi1, hi2);
                q1.y = lo1 | (hi1 << 16);
                q2.y = lo2 | (hi2 << 16);
                // 8 codes: half of a 16-byte chunk
                if (c < 64) {
                    unsigned char* at = sm.q + (c >> 4) * 2 * kPanel;
                    const uint32_t chunk = (c >> 1) & 7u, half = (c & 1u) * 8u;
                    *reinterpret_cast<uint2*>(at + r1 * 128u + ((chunk ^ (r1 & 7u)) << 4) + half) = q1;
                    *reinterpret_cast<uint2*>(at + r2 * 128u + ((chunk ^ (r2 & 7u)) << 4) + half) = q2;
                } else {
                    unsigned char* at = sm.q + 8 * kPanel;
                    const uint32_t chunk = (c - 64) >> 1, half = (c & 1u) * 8u;
                    *reinterpret_cast<uint2*>(at + r1 * 64u + ((chunk ^ ((r1 >> 1) & 3u)) << 4) + half) = q1;
                    *reinterpret_cast<uint2*>(at + r2 * 64u + ((chunk ^ ((r2 >> 1) & 3u)) << 4) + half) = q2;
                }
            }
        }
    }
}

template <bool FP8, bool WHOLE>
__device__ __forceinline__ void soften(const MlaArgs& a, Smem<FP8, WHOLE>& sm) {
    const uint32_t tid = threadIdx.x, warp = tid >> 5, lane = tid & 31u;
    const uint32_t quad = lane >> 2, in_quad = lane & 3u, hb = blockIdx.x % a.HB;
    const uint32_t rows = a.H - hb * kHeads < kHeads ? a.H - hb * kHeads : kHeads;
    const uint32_t head0 = hb * kHeads, tmem = sm.tmem + ((warp * 32u) << 16);
    // this thread's rows of S: heads h0 and h0 + 8, 16 positions of each
    const uint32_t h0 = warp * 16u + quad;
    OpenPiece* open = reinterpret_cast<OpenPiece*>(a.workspace) + blockIdx.x;
    Walk w;
    w.begin(a.split, sm.split.start);
    bool ok = true;
    uint32_t tile = 0, segment = 0;
    if constexpr (FP8) {
        // rows of Q past the last head stay zeros
        for (uint32_t i = tid; i < sizeof(sm.q) / 16; i += kSoftmaxThreads)
            reinterpret_cast<uint4*>(sm.q)[i] = make_uint4(0, 0, 0, 0);
        if (tid < kHeads) sm.q_scale[tid] = 1.0f;
        any_softmax(false);
    }
    while (!w.done()) {
        if ((int64_t)w.len0 + w.k + 1 > a.split.cap && tid == 0) flag(a.err_flags, KVW_ERR_PAGE);
        const uint32_t shared_by = w.first == 0 && !w.whole()
                                       ? sharers(a.split, sm.split.start, w, blockIdx.x / a.HB)
                                       : 0;
        float qs0 = a.scale, qs1 = a.scale;
        if constexpr (FP8) {
            // the last S of the segment before has been read: Q is free
            split_queries(a, sm, w.t, head0, rows);
            fence_async_smem();
            any_softmax(false);  // q_scale is written
            qs0 = fmaxf(a.scale * sm.q_scale[h0], 1.17549435e-38f);
            qs1 = fmaxf(a.scale * sm.q_scale[h0 + 8], 1.17549435e-38f);
            if (lane == 0) mbar_arrive(&sm.q_ready);
        }
        float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.0f, l1 = 0.0f;
        const uint32_t count = w.last - w.first;
        bool stopped = false;
        for (uint32_t i = 0; i < count; ++i, ++tile) {
            const uint32_t buf = tile & 1u;
            float s[32];
            ok = ok && wait_phase(&sm.s_full[buf], (tile >> 1) & 1u, &sm.stop, a.wait_limit);
            if (ok) {
                fence_after_sync();
                tmem_ld_16x64(s, tmem + kScoreColumn + buf * kTile);
                if constexpr (FP8) {
                    float s2[32];
                    tmem_ld_16x64(s2, tmem + (16u << 16) + kScoreColumn + buf * kTile);
#pragma unroll
                    for (int e = 0; e < 32; ++e) s[e] = fmaf(s2[e], 0.0625f, s[e]);
                }
            } else {
#pragma unroll
                for (int e = 0; e < 32; ++e) s[e] = 0.0f;
            }
            const uint64_t there = sm.there[tile & 7u];
            if (there != ~0ull) {
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                    const uint32_t j = 8u * (e >> 2) + 2u * in_quad + (e & 1);
                    if (!((there >> j) & 1ull)) s[e] = -INFINITY;
                }
            }
            float top0 = -INFINITY, top1 = -INFINITY;
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
                top0 = fmaxf(top0, fmaxf(s[e], s[e + 1]));
                top1 = fmaxf(top1, fmaxf(s[e + 2], s[e + 3]));
            }
#pragma unroll
            for (int o = 1; o < 4; o <<= 1) {
                top0 = fmaxf(top0, __shfl_xor_sync(0xffffffffu, top0, o));
                top1 = fmaxf(top1, __shfl_xor_sync(0xffffffffu, top1, o));
            }
            top0 *= qs0;
            top1 *= qs1;
            constexpr float kLift = weight_lift<FP8>();
            if (any_softmax(!ok || top0 > m0 + (kSlack + kLift) ||
                            top1 > m1 + (kSlack + kLift))) {
                const float n0 = fmaxf(m0, top0 - kLift), n1 = fmaxf(m1, top1 - kLift);
                const float f0 = n0 == m0 ? 1.0f : fast_exp2(m0 - n0);
                const float f1 = n1 == m1 ? 1.0f : fast_exp2(m1 - n1);
                m0 = n0;
                m1 = n1;
                l0 *= f0;
                l1 *= f1;
                if (in_quad == 0) {
                    sm.alpha[h0] = f0;
                    sm.alpha[h0 + 8] = f1;
                }
                if (i > 0)
                    ok = ok && wait_phase(&sm.pv_done, (tile - 1) & 1u, &sm.stop, a.wait_limit);
                if (any_softmax(!ok)) {  // the alphas are written
                    stopped = true;
                    break;
                }
                if (i > 0) {
                    fence_after_sync();
                    for (uint32_t c = 0; c < rows; c += 16) {
                        float f[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e) f[e] = sm.alpha[c + e];
#pragma unroll
                        for (uint32_t j = 0; j < 4; ++j) {
                            float o[16];
                            tmem_ld_32x16(o, tmem + j * kHeads + c);
#pragma unroll
                            for (int e = 0; e < 16; ++e) o[e] *= f[e];
                            tmem_st_32x16(tmem + j * kHeads + c, o);
                        }
                    }
                    tmem_st_wait();
                }
            }
            // a row that has seen no position keeps m = -inf: subtract 0
            const float b0 = m0 == -INFINITY ? 0.0f : m0, b1 = m1 == -INFINITY ? 0.0f : m1;
            uint32_t p[16];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float x0 = fast_exp2(fmaf(s[4 * e], qs0, -b0));
                const float x1 = fast_exp2(fmaf(s[4 * e + 1], qs0, -b0));
                const float y0 = fast_exp2(fmaf(s[4 * e + 2], qs1, -b1));
                const float y1 = fast_exp2(fmaf(s[4 * e + 3], qs1, -b1));
                l0 += x0 + x1;
                l1 += y0 + y1;
                p[2 * e] = pack2<FP8>(x0, x1);
                p[2 * e + 1] = pack2<FP8>(y0, y1);
            }
            if (tile > 0)  // P's memory is free
                ok = ok && wait_phase(&sm.pv_done, (tile - 1) & 1u, &sm.stop, a.wait_limit);
            if (ok) {
#pragma unroll
                for (uint32_t e = 0; e < 8; ++e) {
                    const uint32_t chunk = ((e ^ (h0 & 7u)) << 4) + in_quad * 4u;
                    *reinterpret_cast<uint32_t*>(sm.p + h0 * 128u + chunk) = p[2 * e];
                    *reinterpret_cast<uint32_t*>(sm.p + (h0 + 8u) * 128u + chunk) = p[2 * e + 1];
                }
                if constexpr (!FP8) {
                    // a weight of 0 does not keep out what a row that is not
                    // there may hold
                    if (there != ~0ull) {
                        unsigned char* kv = sm.kv + (tile & 1u) * 9 * kPanel;
                        for (uint32_t x = tid; x < 64 * 64; x += kSoftmaxThreads) {
                            const uint32_t r = x >> 6, c = x & 63u;
                            if (!((there >> r) & 1ull))
                                *reinterpret_cast<uint4*>(kv + (c >> 3) * kPanel + r * 128u +
                                                          (c & 7u) * 16u) = make_uint4(0, 0, 0, 0);
                        }
                    }
                }
                fence_async_smem();
                fence_before_sync();  // S has been read, O^T may have been rescaled
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.p_full);
            }
        }
        if (stopped) break;
        // ---- the segment's results
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
            l0 += __shfl_xor_sync(0xffffffffu, l0, o);
            l1 += __shfl_xor_sync(0xffffffffu, l1, o);
        }
        if (in_quad == 0) {
            sm.m[h0] = m0;
            sm.m[h0 + 8] = m1;
            sm.l[h0] = l0;
            sm.l[h0 + 8] = l1;
        }
        const bool whole = w.whole();
        ok = ok && wait_phase(&sm.pv_done, (tile - 1) & 1u, &sm.stop, a.wait_limit);
        // What the sums are multiplied by.  Not before the wait: a warp behind
        // this one may still rescale by the alphas of the last tile, which it
        // has read when it arrives on p_full, and pv_done follows all four.
        // The vote makes the new ones visible.
        if (ok && in_quad == 0) {
            sm.alpha[h0] = l0 == 0.0f ? 0.0f : whole ? a.row_scale / l0 : 1.0f;
            sm.alpha[h0 + 8] = l1 == 0.0f ? 0.0f : whole ? a.row_scale / l1 : 1.0f;
        }
        if (any_softmax(!ok)) break;
        fence_after_sync();
        float* part = slot_of(a, blockIdx.x, w.first == 0 ? 1 : 0);
        uint16_t* out = a.out + ((uint64_t)w.t * a.H + head0) * kLatent;
        // A lane has one column (its own) of 16 heads at a time: neighbours
        // swap, so that each has two columns of every other head.
        const uint32_t odd = lane & 1u;
        uint16_t* out_at = out + (uint64_t)odd * kLatent + (tid & ~1u);
        float* part_at = part + (uint64_t)odd * kLatent + (tid & ~1u);
        auto store = [&](auto whole_const, uint32_t c) {
            float f[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) f[e] = sm.alpha[c + e];
#pragma unroll
            for (uint32_t j = 0; j < 4; ++j) {
                float o[16];
                tmem_ld_32x16(o, tmem + j * kHeads + c);
#pragma unroll
                for (uint32_t e = 0; e < 16; e += 2) {
                    const float x = o[e] * f[e], y = o[e + 1] * f[e + 1];
                    const float got = __shfl_xor_sync(0xffffffffu, odd ? x : y, 1);
                    const float lo = odd ? got : x, hi = odd ? y : got;
                    if (c + e + odd < rows) {
                        const uint64_t at = (uint64_t)(c + e) * kLatent + j * 128u;
                        if constexpr (decltype(whole_const)::value)
                            *reinterpret_cast<uint32_t*>(out_at + at) = pack_bf16x2(lo, hi);
                        else
                            *reinterpret_cast<float2*>(part_at + at) = make_float2(lo, hi);
                    }
                }
            }
        };
#pragma unroll 1
        for (uint32_t c = 0; c < rows; c += 16) {
            if (whole)
                store(std::true_type{}, c);
            else
                store(std::false_type{}, c);
        }
        fence_before_sync();
        if (tid < rows) {
            const float l = sm.l[tid], m = sm.m[tid];
            if (whole) {
                if (a.lse)
                    a.lse[(uint64_t)w.t * a.H + head0 + tid] =
                        l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2;
            } else {
                part[(uint64_t)a.slot_rows * kLatent + tid] = m;
                part[(uint64_t)a.slot_rows * (kLatent + 1) + tid] = l;
            }
        }
        if (shared_by && tid == 0) {
            OpenPiece x;
            x.n = shared_by;
            x.t = w.t;
            x.tokens = 1;
            x.block = hb;
            *open = x;
        }
        any_softmax(false);  // sm.m, sm.l are read
        if (lane == 0) mbar_arrive(&sm.o_free);
        ++segment;
        w.next(a.split);
    }
    if (!ok && lane == 0) flag(a.err_flags, KVW_ERR_TIMEOUT);
}

template <bool FP8, bool WHOLE, Hook HOOK>
__global__ void __launch_bounds__((threads_of<FP8, WHOLE>()), 1)
    mla_decode_kernel(const MlaArgs a, const __grid_constant__ CacheMaps maps,
                      const __grid_constant__ QMaps qm) {
    extern __shared__ __align__(1024) unsigned char dyn[];
    Smem<FP8, WHOLE>& sm = *reinterpret_cast<Smem<FP8, WHOLE>*>(dyn);
    const uint32_t tid = threadIdx.x, warp = tid >> 5;
    // the join of the pieces may be scheduled; it waits for this grid's end
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (tid == 128) {  // not a thread that the division of the work waits for
        for (uint32_t i = 0; i < 2 * kGroups; ++i) {
            mbar_init(&sm.full[i], 1);
            // E4M3: codes go to the matrix unit and to four warps
            mbar_init(&sm.empty[i], FP8 ? 5 : 1);
        }
        for (uint32_t i = 0; i < 2; ++i) {
            mbar_init(&sm.v_full[i], 4);
            mbar_init(&sm.v_empty[i], 1);
        }
        mbar_init(&sm.q_full, 1);
        mbar_init(&sm.q_ready, 4);
        mbar_init(&sm.q_free, 1);
        for (int i = 0; i < 2; ++i) mbar_init(&sm.s_full[i], 1);
        mbar_init(&sm.p_full, 4);
        mbar_init(&sm.pv_done, 1);
        mbar_init(&sm.o_free, 4);
        mbar_init(&sm.drained, 1);
        sm.stop = 0;
        mbar_init_fence();
        prefetch_map(&maps.map[0]);
        prefetch_map(&qm.latent);
        prefetch_map(&qm.rope);
        prefetch_map(&qm.panels);
    }
    if (warp == 5) tmem_alloc(&sm.tmem, kTmemColumns);
    // All that touches global memory comes after the kernel before this one in
    // the stream; its launch and the lines above do not (calls in a row,
    // one token, 16 heads, 1501 positions 18.5 -> 15.5 us).
    wait_for_stream();
    const bool ok = find_piece(a.split, a.pieces, blockIdx.x / a.HB, sm.split);
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    if (tid == 0) reinterpret_cast<OpenPiece*>(a.workspace)[blockIdx.x].n = 0;
    if (!ok) {
        if (blockIdx.x == 0 && tid == 0) flag(a.err_flags, KVW_ERR_OFFSETS);
    } else if (warp < 4) {
        if constexpr (HOOK == Hook::kAbandoned)
            *reinterpret_cast<volatile uint32_t*>(&sm.stop) = 1;
        else
            soften<FP8, WHOLE>(a, sm);
    } else if (warp == 4) {
        feed<FP8, WHOLE, HOOK, 0>(a, maps, qm, sm);
    } else if (warp == 5) {
        if constexpr (FP8)
            multiply_codes(a, sm);
        else
            multiply(a, sm);
    } else if (FP8 && warp < 10) {
        if constexpr (FP8) convert(a, sm);
    } else if (warp == (FP8 ? 10 : 6)) {
        if constexpr (feeders_of<FP8, WHOLE>() > 1) feed<FP8, WHOLE, HOOK, 1>(a, maps, qm, sm);
    } else {
        if constexpr (feeders_of<FP8, WHOLE>() > 2) feed<FP8, WHOLE, HOOK, 2>(a, maps, qm, sm);
    }
    fence_before_sync();
    __syncthreads();
    if (warp == 5) {
        fence_after_sync();
        tmem_free(sm.tmem, kTmemColumns);
    }
}

// Joins what piece blockIdx.x / HB left open, four rows a block: weights
// 2^(m_i - M) of the pieces, then one weighted sum in their order.  Of up to
// AT_ONCE pieces each thread loads all that it needs at once, of more AT_ONCE
// at a time.  With many requests every piece has a join of a few neighbours,
// and what counts is blocks per SM (3 loads, four blocks: 64 requests 118 us,
// with 8 loads and two blocks 127); with few requests it is loads in flight
// (one context of 24598 positions 43 and 38 us).
constexpr int kJoinThreads = 512;
constexpr uint32_t kJoinRows = 4;

template <uint32_t AT_ONCE>
__global__ void __launch_bounds__(kJoinThreads, AT_ONCE > 4 ? 2 : 4)
    mla_join_kernel(const MlaArgs a) {
    __shared__ float s_w[kJoinRows][kMaxCtas];
    __shared__ float s_top[kJoinRows], s_sum[kJoinRows];
    wait_for_stream();
    const OpenPiece open = reinterpret_cast<const OpenPiece*>(a.workspace)[blockIdx.x];
    if (open.n == 0) return;
    const uint32_t rows = a.H - open.block * kHeads < kHeads ? a.H - open.block * kHeads : kHeads;
    const uint32_t r0 = blockIdx.y * kJoinRows;
    if (r0 >= rows) return;
    const uint32_t here = rows - r0 < kJoinRows ? rows - r0 : kJoinRows;
    const uint32_t piece = blockIdx.x / a.HB, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31u;
    const uint32_t n = open.n;
    auto part = [&](uint32_t i) {
        return slot_of(a, (piece + i) * a.HB + open.block, i == 0 ? 1 : 0);
    };
    const uint64_t tops = (uint64_t)a.slot_rows * kLatent, sums = tops + a.slot_rows;
    const uint32_t rj = tid >> 7, d = (tid & 127u) * 4u;  // 128 threads a row
    float4 o = make_float4(0, 0, 0, 0);
    float top = -INFINITY, l = 0.0f;
    auto add = [&](float f, const float4& x) {
        o.x += f * x.x;
        o.y += f * x.y;
        o.z += f * x.z;
        o.w += f * x.w;
    };
    if (n <= AT_ONCE) {
        if (rj >= here) return;
        float4 x[AT_ONCE];
        float m[AT_ONCE], s[AT_ONCE];
#pragma unroll
        for (uint32_t k = 0; k < AT_ONCE; ++k) {
            m[k] = -INFINITY;
            s[k] = 0.0f;
            if (k < n) {
                const float* p = part(k);
                x[k] = load_part(p + (uint64_t)(r0 + rj) * kLatent + d);
                m[k] = p[tops + r0 + rj];
                s[k] = p[sums + r0 + rj];
                top = fmaxf(top, m[k]);
            }
        }
        const float base = top == -INFINITY ? 0.0f : top;
#pragma unroll
        for (uint32_t k = 0; k < AT_ONCE; ++k)
            if (k < n) {
                const float f = fast_exp2(m[k] - base);
                l += f * s[k];
                add(f, x[k]);
            }
    } else {
        if (warp < here) {
            const uint32_t r = r0 + warp;
            float s_first = 0.0f;  // of the lane's first piece
            if (lane < n) s_first = part(lane)[sums + r];
            for (uint32_t i = lane; i < n; i += 32) {
                const float m = part(i)[tops + r];
                s_w[warp][i] = m;
                top = fmaxf(top, m);
            }
#pragma unroll
            for (int k = 16; k > 0; k >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, k));
            const float base = top == -INFINITY ? 0.0f : top;
            for (uint32_t i = lane; i < n; i += 32) {
                const float f = fast_exp2(s_w[warp][i] - base);
                s_w[warp][i] = f;
                l += f * (i == lane ? s_first : part(i)[sums + r]);
            }
#pragma unroll
            for (int k = 16; k > 0; k >>= 1) l += __shfl_xor_sync(0xffffffffu, l, k);
            if (lane == 0) {
                s_top[warp] = top;
                s_sum[warp] = l;
            }
        }
        __syncthreads();
        if (rj >= here) return;
        top = s_top[rj];
        l = s_sum[rj];
        for (uint32_t i0 = 0; i0 < n; i0 += AT_ONCE) {
            float4 x[AT_ONCE];
#pragma unroll
            for (uint32_t k = 0; k < AT_ONCE; ++k)
                if (i0 + k < n) x[k] = load_part(part(i0 + k) + (uint64_t)(r0 + rj) * kLatent + d);
#pragma unroll
            for (uint32_t k = 0; k < AT_ONCE; ++k)
                if (i0 + k < n) add(s_w[rj][i0 + k], x[k]);
        }
    }
    const uint64_t row = (uint64_t)open.t * a.H + open.block * kHeads + r0 + rj;
    const float inv = l == 0.0f ? 0.0f : a.row_scale / l;
    uint2 y;
    y.x = pack_bf16x2(o.x * inv, o.y * inv);
    y.y = pack_bf16x2(o.z * inv, o.w * inv);
    *reinterpret_cast<uint2*>(a.out + row * kLatent + d) = y;
    if (d == 0 && a.lse) a.lse[row] = l == 0.0f ? -INFINITY : (top + log2f(l)) * kLn2;
}

int workspace_bytes_for(uint32_t num_heads, uint64_t* bytes) {
    if (!bytes || !num_heads) return KVW_EINVAL;
    if (num_heads > 1024) return KVW_EUNSUPPORTED;
    const uint32_t rows = num_heads < kHeads ? num_heads : kHeads;
    *bytes = kMaxCtas * (sizeof(OpenPiece) + 2ull * slot_floats(rows) * sizeof(float));
    return KVW_OK;
}

template <bool FP8, bool WHOLE, Hook HOOK>
cudaError_t launch(MlaArgs& a, const CacheMaps& maps, const QMaps& qm, cudaStream_t stream) {
    constexpr size_t smem = sizeof(Smem<FP8, WHOLE>);
    static_assert(smem <= 227 * 1024, "shared memory of a CTA");
    cudaError_t e = prepare_smem<&mla_decode_kernel<FP8, WHOLE, HOOK>>(smem);
    if (e != cudaSuccess) return e;
    int sms = 0;
    if ((e = sm_count(sms)) != cudaSuccess) return e;
    uint32_t ctas = (uint32_t)sms < kMaxCtas ? (uint32_t)sms : kMaxCtas;
    a.pieces = ctas / a.HB > 0 ? ctas / a.HB : 1;
    ctas = a.pieces * a.HB;
    e = launch_early(&mla_decode_kernel<FP8, WHOLE, HOOK>, dim3(ctas), threads_of<FP8, WHOLE>(), smem, stream,
                     a, maps, qm);
    if (e != cudaSuccess) return e;
    // few tokens: many pieces each
    const dim3 joins(ctas, (a.slot_rows + kJoinRows - 1) / kJoinRows);
    return a.pieces > 4 * a.split.T
               ? launch_early(&mla_join_kernel<8>, joins, kJoinThreads, 0, stream, a)
               : launch_early(&mla_join_kernel<3>, joins, kJoinThreads, 0, stream, a);
}

int mla_entry(void* out, float* lse, const void* q_latent, int64_t q_latent_row_stride,
              const void* q_rope, int64_t q_rope_row_stride, const uint32_t* input_row_offsets,
              uint32_t num_batches, uint32_t tot_seq_len, uint32_t num_heads,
              const kvw_paged_cache_t* cache, uint32_t layer_idx, float sm_scale, void* workspace,
              uint64_t workspace_bytes, uint32_t* err_flags, cudaStream_t stream, Hook hook,
              uint64_t wait_ns) {
    const int st = check_cache(cache, layer_idx, 1);
    if (st != KVW_OK) return st;
    uint64_t need = 0;
    const int ws = workspace_bytes_for(num_heads, &need);
    if (ws != KVW_OK) return ws;
    if (cache->num_heads != 1 || cache->head_size != kRow) return KVW_EUNSUPPORTED;
    if (num_batches > KVW_MAX_BATCHES || tot_seq_len > (1u << 20) || !tma_sizes_ok(cache))
        return KVW_EUNSUPPORTED;
    if (!out || !q_latent || !q_rope || !input_row_offsets || num_batches == 0 || !workspace ||
        workspace_bytes < need)
        return KVW_EINVAL;
    if (!aligned16(out) || !aligned16(q_latent) || !aligned16(q_rope) || !aligned16(workspace) ||
        !aligned4(lse) || !aligned4(input_row_offsets) || !aligned4(err_flags))
        return KVW_EINVAL;
    if (!tma_strides_ok(cache, 1)) return KVW_EINVAL;
    const int64_t top = 1ll << 39;  // bytes below 2^40
    if (q_latent_row_stride < (int64_t)num_heads * kLatent || q_latent_row_stride % 8 ||
        q_latent_row_stride >= top || q_rope_row_stride < (int64_t)num_heads * 64 ||
        q_rope_row_stride % 8 || q_rope_row_stride >= top)
        return KVW_EINVAL;
    if (!(sm_scale > 0.0f) || !std::isfinite(sm_scale)) return KVW_EINVAL;
    if (tot_seq_len == 0) return KVW_OK;

    const bool fp8 = cache->dtype == KVW_DTYPE_FP8_E4M3;
    MlaArgs a = {};
    a.split.offsets = input_row_offsets;
    a.split.cache_lengths = cache->cache_lengths;
    a.split.B = num_batches;
    a.split.T = tot_seq_len;
    a.split.blocks = 1;  // the row blocks of a token are CTAs of the same piece
    a.split.min_units = 1;
    // What a segment costs beside its tiles, in tiles: with E4M3 the queries are
    // split (2, 4, 6: 174 requests of up to 1266 positions, 64 heads 74, 71, 68
    // us; 206 of up to 2249, 16 heads 73, 72, 75); bf16 168 requests of 2 tokens,
    // 8 heads 47, 52, 56 us.
    a.split.overhead = fp8 ? 5 : 2;
    const uint64_t reach = (uint64_t)cache->max_pages_per_seq * cache->page_size;
    a.split.cap = reach > kMaxReach ? (int64_t)kMaxReach : (int64_t)reach;
    a.split.window = 1ll << 40;
    a.out = static_cast<uint16_t*>(out);
    a.lse = lse;
    a.q_latent = static_cast<const uint16_t*>(q_latent);
    a.q_rope = static_cast<const uint16_t*>(q_rope);
    a.q_latent_stride = q_latent_row_stride;
    a.q_rope_stride = q_rope_row_stride;
    a.page_table = cache->page_table;
    a.err_flags = err_flags;
    a.workspace = static_cast<unsigned char*>(workspace);
    a.row_scale = fp8 ? cache->scale : 1.0f;
    a.scale = sm_scale * kLog2e * a.row_scale;
    a.H = num_heads;
    a.HB = (num_heads + kHeads - 1) / kHeads;
    a.slot_rows = num_heads < kHeads ? num_heads : kHeads;
    a.num_pages = cache->num_pages;
    a.max_pages = cache->max_pages_per_seq;
    a.ps = make_fast_div(cache->page_size);
    a.wait_limit = wait_cycles(wait_ns);
    CacheMaps maps;
    QMaps qm;
    int e = encode_cache_maps(&maps, cache, layer_idx, 1);
    if (e == KVW_OK)
        e = encode_query_map(&qm.latent, q_latent, kLatent, num_heads, tot_seq_len,
                             q_latent_row_stride);
    if (e == KVW_OK)
        e = encode_query_map(&qm.rope, q_rope, 64, num_heads, tot_seq_len, q_rope_row_stride);
    qm.panels = qm.rope;
    if (e == KVW_OK && maps.log_rows == 6)
        e = encode_panel_map(&qm.panels, cache, layer_idx, fp8 ? 2 : 3);
    if (e != KVW_OK) return e;
    cudaError_t r;
    auto run = [&](auto with) {
        constexpr Hook kHook = decltype(with)::value;
        if (maps.log_rows == 6)
            return fp8 ? launch<true, true, kHook>(a, maps, qm, stream)
                       : launch<false, true, kHook>(a, maps, qm, stream);
        return fp8 ? launch<true, false, kHook>(a, maps, qm, stream)
                   : launch<false, false, kHook>(a, maps, qm, stream);
    };
#ifdef KVW_TEST_HOOKS
    r = hook == Hook::kWithheld    ? run(std::integral_constant<Hook, Hook::kWithheld>{})
        : hook == Hook::kAbandoned ? run(std::integral_constant<Hook, Hook::kAbandoned>{})
                                   : run(std::integral_constant<Hook, Hook::kNone>{});
#else
    if (hook != Hook::kNone) return KVW_EUNSUPPORTED;
    r = run(std::integral_constant<Hook, Hook::kNone>{});
#endif
    return r == cudaSuccess ? KVW_OK : KVW_ECUDA;
}

}  // namespace
}  // namespace kvw

extern "C" int kva_mla_decode_workspace(uint32_t num_heads, uint64_t* bytes) {
    return kvw::workspace_bytes_for(num_heads, bytes);
}

extern "C" int kva_mla_decode_paged(void* out, float* lse, const void* q_latent,
                                    int64_t q_latent_row_stride, const void* q_rope,
                                    int64_t q_rope_row_stride, const uint32_t* input_row_offsets,
                                    uint32_t num_batches, uint32_t tot_seq_len, uint32_t num_heads,
                                    const kvw_paged_cache_t* cache, uint32_t layer_idx,
                                    float sm_scale, void* workspace, uint64_t workspace_bytes,
                                    uint32_t* err_flags, cudaStream_t stream) {
    return kvw::mla_entry(out, lse, q_latent, q_latent_row_stride, q_rope, q_rope_row_stride,
                          input_row_offsets, num_batches, tot_seq_len, num_heads, cache, layer_idx,
                          sm_scale, workspace, workspace_bytes, err_flags, stream,
                          kvw::Hook::kNone, kvw::kWaitLimitNs);
}

#ifdef KVW_TEST_HOOKS
// Test builds only (a separate library; the product has no such symbol): the
// first copies of every CTA are announced on their barrier but never made, and
// every wait is bounded by `wait_ns`, so the waits for them run out,
// KVW_ERR_TIMEOUT is set and the kernel returns.
extern "C" int kva_test_mla_decode_withheld(
    void* out, const void* q_latent, int64_t q_latent_row_stride, const void* q_rope,
    int64_t q_rope_row_stride, const uint32_t* input_row_offsets, uint32_t num_batches,
    uint32_t tot_seq_len, uint32_t num_heads, const kvw_paged_cache_t* cache, uint32_t layer_idx,
    void* workspace, uint64_t workspace_bytes, uint32_t* err_flags, cudaStream_t stream,
    uint64_t wait_ns) {
    return kvw::mla_entry(out, nullptr, q_latent, q_latent_row_stride, q_rope, q_rope_row_stride,
                          input_row_offsets, num_batches, tot_seq_len, num_heads, cache, layer_idx,
                          0.1f, workspace, workspace_bytes, err_flags, stream, kvw::Hook::kWithheld,
                          wait_ns);
}

// The softmax warps leave at once, so nobody waits for the last copies;
// err_flags[1] counts places whose last copy had not landed when their feeding
// warp left.
extern "C" int kva_test_mla_decode_abandoned(
    void* out, const void* q_latent, int64_t q_latent_row_stride, const void* q_rope,
    int64_t q_rope_row_stride, const uint32_t* input_row_offsets, uint32_t num_batches,
    uint32_t tot_seq_len, uint32_t num_heads, const kvw_paged_cache_t* cache, uint32_t layer_idx,
    void* workspace, uint64_t workspace_bytes, uint32_t* err_flags, cudaStream_t stream,
    uint64_t wait_ns) {
    return kvw::mla_entry(out, nullptr, q_latent, q_latent_row_stride, q_rope, q_rope_row_stride,
                          input_row_offsets, num_batches, tot_seq_len, num_heads, cache, layer_idx,
                          0.1f, workspace, workspace_bytes, err_flags, stream,
                          kvw::Hook::kAbandoned, wait_ns);
}
#endif
