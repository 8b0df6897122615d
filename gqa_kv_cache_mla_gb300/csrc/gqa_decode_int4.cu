// Attention of new tokens over a paged GQA key-value cache held in 4 bits.
//
// Mathematics: the pass of gqa_decode_paged.cu over K = s_k (u - 8) and V =
// s_v (u - 8), with a scale s for each position and group of 64 columns:
//   S_j  = sum_g s_k[j, g] (sum_{d in g} q_d u_jd - 8 sum_{d in g} q_d)
//   O_d  = sum_j (P_j s_v[j, g]) u_jd - 8 sum_j (P_j s_v[j, g])
// Both offsets are sums over what the matrix instructions see, so they come
// from the same instructions with a constant operand: 8 sum q once for a
// segment, where it is the products' first accumulator, and 8 sum (P s_v) as
// one product per group and 16 positions.
//
// Codes as operands: the pattern of a code u in the lowest 4 bits of an fp16
// number is u 2^-24, and in the next 4 it is 16 u 2^-24, both exact.  Four codes
// lie in 16 bits, so an AND takes a pair of them out of 32 bits and one shift
// serves two pairs: 5 instructions for 8 codes, against 11 to bring them to
// exact bf16 numbers (and with the bf16 patterns 128 + u alone the offset to
// cancel would be 136).  Queries that meet codes 16 times as large are 16 times
// smaller, and output columns of such codes 16 times as large until the end.
// The price: these numbers lie below fp16's smallest normal one, 2^-14, and the
// instruction lines its products up as if each were that large, so it may cut a
// product at 2^-13 of a code (in units of its other factor).  That is a 2000th
// of the half code that the cache itself may be off, and less than the fp16
// rounding of a weight costs a code of +-4.  Codes moved to bits 4 to 7 are cut
// at 2^-17 and cost two more instructions in eight: 256 requests 217 us against
// 201.
//
// Both products have the row block's 8 rows as the instruction's columns: S^T =
// K Q^T and O^T = V^T P^T.  Codes are then the operand of 16 rows, no half of an
// instruction is idle, and P^T passes from the order of one's result to the
// other's operand by transposing 8 x 8 blocks (movmatrix).  Row i of an operand's
// upper and lower half are positions 2 i and 2 i + 1, whose scales are one word.
// (Queries as the operand of 16 rows, half of them zeros: 364 us instead of 292
// at that step.  Two row blocks in a pass, for 9 to 16 rows, lack the registers:
// 64 query over 4 key-value heads 124 us, as two passes side by side 119.  Scores
// by E4M3 products, whose operand is one AND for 4 codes: 299 us instead of 252;
// with operands that change they run at half the rate of the fp16 ones.)
//
// Weights times scales are fp16.  Their reference m follows the row's largest
// P s_v, not its largest score: raised when a product passes 2^15, to where
// the largest is 2^9 (weight_lift).  The sum of weights is fp32.  A position whose
// values are all zero takes part in it alone, with any weight: so a scale counts as
// kLeastScale at least in the row's largest, and the reference rises as well when
// weights or their sum pass kMostSum.  (By the products alone, zero values 80 above
// the rest made the sum infinite, and with it every other position's share 0; the
// look at the sums costs 198 -> 201 us of 256 requests, 128 -> 131 of heads of 64.)
//
// Bound: a tile of 64 positions is 8.7 KB for heads of 128, and what a consumer
// does for it (S, softmax, O^T for 16 positions each of four warps) some 250
// instructions a slice, half of an SM's issue slots at the full rate of HBM; the
// warps wait for each other's results rather than for tiles (feeding alone: 178
// us of the 201 below).  So: three CTAs of four consumer warps per SM, two tiles
// at a time, all that can be known once per segment worked out by the feeding
// warp, queries' operands in shared memory.
//
// Measured, 32 query and 8 key-value heads of 128: 256 requests of up to 8192
// positions 201 us (5.7 TB/s, 86 % of the card's copy rate; with 198 at that step,
// one tile at a time 236, two CTAs per SM 217), with a cap 228 (the instance for
// heads of 128 spills 16 bytes a thread), with a distance bias 205, pages of 16 235,
// heads of 64 131, of 96 176, of 256 (128 requests) 207; 64 query heads, 8 requests
// of up to 131072 97 us; 32 of up to 4096 24 us (some 9 of it before the first and
// after the last byte); one token over 901 positions 9.7 us, over 65536 24.  A prompt
// is right and slow, its context converted for every 8 rows: 8 requests of 512 new
// tokens after up to 4096 940 us, of which the products need 75.
//
// Division of the work, workspace and join are those of gqa_decode_paged.cu.
#include <cstdint>
#include <type_traits>

#include "kva_gqa.cuh"
#include "kva_int4.cuh"
#include "kva_tma.cuh"

namespace kvw {
namespace {

// A value's scale as the weights' reference sees it, at least; weights that raise
// the reference, at a time or in all; the sum of a row that has no reference.
constexpr float kLeastScale = 0x1p-40f, kMostSum = 0x1p100f, kUnset = 0x1p126f;

// What happens to scores: nothing, a distance bias, or a cap and perhaps a bias.
enum class Mods { kNone, kBias, kCap };

// One layer's codes and scales.  A copy takes both planes of some rows of one
// head and page: the codes as lines of 128 bytes in the 128-byte swizzle
// (chunk c of line l lies at c ^ (l & 7)), the scales as they lie, group by
// group.
struct Int4Maps {
    CacheMaps codes;  // one map: copies of R rows, R = 16, 32 or 64
    CUtensorMap scales;
};

inline int encode_int4_maps(Int4Maps* m, const kvw_paged_cache_t* c, const kva_group_scales_t* s,
                            uint32_t layer_idx) {
    const auto encode = tensor_map_encoder();
    if (!encode) return KVW_ECUDA;
    const uint32_t rows = rows_per_copy(c->page_size), line_rows = c->head_size / 2;
    m->codes.levels = 1;
    m->codes.log_rows = rows == 64 ? 6 : rows == 32 ? 5 : 4;
    const cuuint32_t ones[5] = {1, 1, 1, 1, 1};
    // a dimension of one index takes any legal stride
    auto bytes = [](int64_t s, uint64_t n) { return n > 1 ? (cuuint64_t)s : (cuuint64_t)16; };
    {
        const cuuint64_t dims[5] = {128, (cuuint64_t)c->page_size * line_rows / 128, c->num_heads,
                                    c->num_pages, 2};
        const cuuint64_t strides[4] = {128, bytes(c->stride_head / 2, c->num_heads),
                                       bytes(c->stride_page / 2, c->num_pages),
                                       (cuuint64_t)(c->stride_kv / 2)};
        const cuuint32_t box[5] = {128, rows * line_rows / 128, 1, 1, 2};
        if (encode(&m->codes.map[0], CU_TENSOR_MAP_DATA_TYPE_UINT8, 5, int4_codes(c, layer_idx, 0),
                   dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                   CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return KVW_EINVAL;
    }
    {
        const uint32_t groups = groups_of(c->head_size);
        const cuuint64_t dims[5] = {c->page_size, groups, c->num_heads, c->num_pages, 2};
        const cuuint64_t strides[4] = {(cuuint64_t)c->page_size * 2,
                                       bytes(s->stride_head * 2, c->num_heads),
                                       bytes(s->stride_page * 2, c->num_pages),
                                       (cuuint64_t)(s->stride_kv * 2)};
        const cuuint32_t box[5] = {rows, groups, 1, 1, 2};
        if (encode(&m->scales, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5,
                   int4_scales(c, s, layer_idx, 0), dims, strides, box, ones,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return KVW_EINVAL;
    }
    return KVW_OK;
}

// D: head size.
template <int D>
struct Shape4 {
    static constexpr int kChunks = D / 32;          // 16-byte chunks of a row of codes
    static constexpr int kGroups = (D + 63) / 64;
    // Four consumer warps, a slice of 16 positions of a tile each, and a feeding
    // warp.
    static constexpr int kWarps = 4, kThreads = 32 * (kWarps + 1);
    static constexpr int kCtas = D <= 128 ? 3 : 2;  // of an SM
    // Tiles of a place of the ring, which arrive and are taken together.
    static constexpr int kTiles = D <= 128 ? 2 : 1;
    static constexpr int kCodes = 2 * kTile * D / 2;             // bytes of a tile, both planes
    static constexpr int kScales = 256 * (kGroups < 2 ? 2 : kGroups);  // and of its scales
    static constexpr int kRing = (D == 64 ? 56 : kCtas == 3 ? 54 : 88) * 1024 / (kTiles * (kCodes + kScales));
    static constexpr int kSlots = kRing > 12 ? 12 : kRing;
    static constexpr int kPadded = D <= 64 ? 64 : D <= 128 ? 128 : 256;  // of a workspace row
    static constexpr int kQPitch = D * 2 + 16;  // eight rows on distinct banks
    // 256-wide heads: what can be worked out again or fetched leaves the registers
    // to the sums (128 requests of up to 8192: 223 -> 206 us; three CTAs 235, spills)
    static constexpr bool kLean = D == 256;
    static constexpr int kBlock = 8, kQBufs = 2;  // rows of a row block; places for queries
    // rows that join at a time, four rows' stores on distinct banks
    static constexpr int kJoinPitch = D + 8;
    static constexpr int kJoinRows = D == 256 ? 2 : 4;
    static_assert(kSlots >= 3, "shared memory");
};

// What the consumers need of a segment, from the feeding warp that walks the
// piece: they would else keep the walk in registers that its tiles need.
struct Segment {
    int64_t p_first, pos0;    // position of its first tile, and of the chunk's first token
    uint32_t count;           // tiles; 0 ends the piece
    uint32_t t, tokens, rows, in_block, head0, block;
    uint32_t shared_by;       // pieces that share it, where this one begins it; else 0
    bool whole, slot1, past;  // a segment of its own; workspace place; past the page table
};

template <int D>
struct Smem4 {
    using Sh = Shape4<D>;
    unsigned char codes[Sh::kSlots][Sh::kTiles][Sh::kCodes];    // units of [K rows][V rows]
    unsigned char scales[Sh::kSlots][Sh::kTiles][Sh::kScales];  // units of [K][V][group][row]
    unsigned char q_raw[Sh::kQBufs][Sh::kBlock * Sh::kQPitch];
    uint4 q[Sh::kChunks][32];  // the queries as operands
    // where kLean: -8 sum of a group's queries for rows 2 i and 2 i + 1
    float2 off[Sh::kWarps][Sh::kLean ? Sh::kGroups : 1][4];
    float join[Sh::kWarps][Sh::kJoinRows][Sh::kJoinPitch];
    uint64_t full[Sh::kSlots], empty[Sh::kSlots], q_full[Sh::kQBufs], q_empty[Sh::kQBufs], meet;
    Segment segment[Sh::kQBufs];
    uint64_t there[Sh::kSlots][Sh::kTiles];  // positions of the tiles that are there
    uint32_t even[Sh::kSlots];  // all positions are there, and every row sees them
    float m[Sh::kWarps][kRows], l[Sh::kWarps][kRows];
    SplitShared<Sh::kThreads> split;
    uint32_t stop;  // a wait ran out
};

// Bytes of shared memory that the scales of a unit of R rows take: copies land
// on multiples of 128.
__host__ __device__ __forceinline__ uint32_t scale_unit(uint32_t groups, uint32_t log_rows) {
    const uint32_t n = 4 * groups << log_rows;
    return n < 128 ? 128 : n;
}

// Where 16-byte chunk `c` of row r of a tile's plane lies among its codes.
template <int D>
__device__ __forceinline__ uint32_t code_at(uint32_t log_rows, uint32_t plane, uint32_t r,
                                            uint32_t c) {
    const uint32_t unit = r >> log_rows, in = r & ((1u << log_rows) - 1u);
    const uint32_t x = ((2 * unit + plane) << log_rows) * (D / 2) + in * (D / 2) + 16 * c;
    return x ^ ((x >> 3) & 0x70u);
}

// The feeding warp: walks the piece's tiles ahead of the arithmetic.
template <int D, Hook HOOK>
__device__ __forceinline__ void feed4(const GqaArgs& a, const Int4Maps& maps, Smem4<D>& sm) {
    using Sh = Shape4<D>;
    const uint32_t lane = threadIdx.x & 31u, log_rows = maps.codes.log_rows;
    const uint32_t row_bytes = D + 4 * Sh::kGroups, s_unit = scale_unit(Sh::kGroups, log_rows);
    Walk w;
    w.begin(a.split, sm.split.start);
    RingPos<Sh::kSlots> at;
    RingPos<Sh::kQBufs> q_at;
    uint32_t bad_page = 0, issued = 0;
    bool ok = true;
    while (ok) {
        ok = wait_phase(&sm.q_empty[q_at.slot], q_at.parity ^ 1u, &sm.stop, a.wait_limit);
        if (!ok) break;
        if (w.done()) {
            if (lane == 0) {
                sm.segment[q_at.slot].count = 0;
                mbar_arrive(&sm.q_full[q_at.slot]);
            }
            __syncwarp();
            q_at.step();
            break;
        }
        const uint32_t block = w.block * a.lanes + blockIdx.x % a.lanes;
        const uint32_t kvh = a.HB == 1 ? block : block / a.HB, hb = block - kvh * a.HB;
        const uint32_t in_block = a.G - hb * Sh::kBlock < a.per_token ? a.G - hb * Sh::kBlock : a.per_token;
        // The last tiles come first: with a distance bias their scores are the
        // largest, and a reference set by them stays (256 requests 243 -> 203 us).
        constexpr uint32_t T = Sh::kTiles;
        const uint32_t places = (w.last - w.first + T - 1) / T;
        const uint32_t final = w.first + (places - 1) * T;  // first tile of the last place
        prefetch_page(maps.codes, a.page_table, a.max_pages, a.ps, w.b,
                      (int64_t)(w.span.tile0 + final) * kTile, lane);
        // ---- the segment, and its queries: one copy per row
        const uint32_t rows = w.span.tokens * in_block;
        if (lane == 0) {
            Segment& x = sm.segment[q_at.slot];
            x.p_first = (int64_t)(w.span.tile0 + w.first) * kTile;
            x.pos0 = (int64_t)w.len0 + ((int64_t)w.k << a.split.log_c);
            x.count = w.last - w.first;
            x.t = w.t;
            x.tokens = w.span.tokens;
            x.rows = rows;
            x.in_block = in_block;
            x.head0 = kvh * a.G + hb * Sh::kBlock;
            x.block = block;
            x.whole = w.whole();
            x.slot1 = w.first == 0;
            x.past = x.pos0 + w.span.tokens > a.split.cap;
            x.shared_by = w.first == 0 && !x.whole
                              ? sharers(a.split, sm.split.start, w, blockIdx.x / a.lanes)
                              : 0;
            mbar_arrive_expect_tx(&sm.q_full[q_at.slot], rows * D * 2);
        }
        __syncwarp();
        if (lane < rows) {
            const uint32_t ct = w.span.tokens == 1 ? 0 : lane / in_block;
            bulk_load(sm.q_raw[q_at.slot] + lane * Sh::kQPitch,
                      a.q + (int64_t)(w.t + ct) * a.q_stride +
                          (int64_t)(kvh * a.G + hb * Sh::kBlock + (lane - ct * in_block)) * D,
                      D * 2, &sm.q_full[q_at.slot]);
        }
        q_at.step();
        // ---- the tiles
        auto copy = [&](uint32_t j, uint32_t unit, uint32_t row, uint32_t page) {
            const uint32_t bar = smem_addr(&sm.full[at.slot]);
            // (rows of a copy begin at multiples of 16; a row's bytes would pass 32 bits)
            tma_rows(smem_addr(sm.codes[at.slot][j]) + ((unit * D) << log_rows), &maps.codes.map[0],
                     0, row / 16 * (D / 16), kvh, page, 0, bar);
            tma_rows(smem_addr(sm.scales[at.slot][j]) + unit * s_unit, &maps.scales, row, 0, kvh,
                     page, 0, bar);
        };
        // positions that every row of the block sees
        const int64_t pos0 = (int64_t)w.len0 + ((int64_t)w.k << a.split.log_c);
        const int64_t all_lo = pos0 + w.span.tokens - a.split.window, all_hi = pos0;
        auto seen = [&](int64_t p, int n) { return p >= all_lo && p + n * kTile - 1 <= all_hi; };
        if (log_rows == 6) {
            // a tile lies in one page: two copies, the same in every lane
            auto plan = [&](uint32_t i) {
                return plan_page(a.page_table, a.max_pages, a.num_pages, a.ps, w.b,
                                 (w.span.tile0 + i) * kTile, w.span.start, w.span.hi);
            };
            PagePlan next[T];
#pragma unroll
            for (uint32_t j = 0; j < T; ++j)
                if (final + j < w.last) next[j] = plan(final + j);
            for (uint32_t place = places; ok && place-- > 0;) {
                const uint32_t i = w.first + place * T;
                PagePlan t[T];
                uint32_t bytes = 0;
                bool all = seen((int64_t)(w.span.tile0 + i) * kTile, T);
#pragma unroll
                for (uint32_t j = 0; j < T; ++j) {
                    t[j] = next[j];
                    if (i + j >= w.last) {
                        t[j].valid = false;
                        t[j].there = 0;
                    } else if (!t[j].valid) {
                        bad_page = 1;
                    }
                    bytes += t[j].valid ? kTile * row_bytes : 0;
                    all = all && t[j].there == ~0ull;
                    if (place > 0) next[j] = plan(i - T + j);
                }
                ok = wait_phase(&sm.empty[at.slot], at.parity ^ 1u, &sm.stop, a.wait_limit);
                if (!ok) break;
                if (elect_one()) {
                    sm.even[at.slot] = all;
#pragma unroll
                    for (uint32_t j = 0; j < T; ++j) sm.there[at.slot][j] = t[j].there;
                    mbar_arrive_expect_tx(&sm.full[at.slot], bytes);
                    if (!(HOOK == Hook::kWithheld && issued == 0)) {
#pragma unroll
                        for (uint32_t j = 0; j < T; ++j)
                            if (t[j].valid) copy(j, 0, t[j].row, t[j].page);
                    }
                }
                __syncwarp();
                at.step();
                ++issued;
            }
            if (ok) w.next(a.split);
            continue;
        }
        // Lane c takes unit c of a place: R rows of one page.  Page ids are looked
        // up one place ahead (256 requests, pages of 16, 281 -> 230 us; of 32, 200).
        const uint32_t per_tile = 64u >> log_rows, j = lane / per_tile, unit = lane % per_tile;
        // (positions that the page table reaches are below 2^32)
        auto begins = [&](uint32_t i) {
            return (w.span.tile0 + i) * kTile + (lane << log_rows);
        };
        auto page_id = [&](uint32_t i) {
            const uint32_t idx = fast_div(begins(i), a.ps);
            return j < T && i + j < w.last && idx < a.max_pages
                       ? __ldg(a.page_table + (uint64_t)w.b * a.max_pages + idx)
                       : (uint32_t)KVW_PAGE_UNMAPPED;
        };
        uint32_t next = page_id(final);
        for (uint32_t place = places; ok && place-- > 0;) {
            const uint32_t i = w.first + place * T;
            const uint32_t page = next, p = begins(i);
            if (place > 0) next = page_id(i - T);
            const int64_t p_tile = (int64_t)(w.span.tile0 + i) * kTile;
            bool used = j < T;
            uint64_t there = ((1ull << (1u << log_rows)) - 1) << (unit << log_rows);
            if (i + T > w.last || p_tile < w.span.start || p_tile + T * kTile > w.span.hi) {
                // the unit's positions that count
                const int64_t lo = p > w.span.start ? (int64_t)p : w.span.start;
                const int64_t end = p_tile + ((int64_t)(lane + 1) << log_rows);
                const int64_t hi = end < w.span.hi ? end : w.span.hi;
                used = used && i + j < w.last && lo < hi;
                there = used ? ((1ull << (uint32_t)(hi - lo)) - 1)
                                   << (uint32_t)(lo - p + (unit << log_rows))
                             : 0;
            }
            const bool valid = used && page < a.num_pages;
            if (used && !valid) bad_page = 1;
            const bool whole = valid && __popcll(there) == 1 << log_rows;
            const bool all =
                __all_sync(0xffffffffu, whole || j >= T) && seen(p_tile, T);
            const uint32_t units = __popc(__ballot_sync(0xffffffffu, valid));
            uint64_t words[T];
#pragma unroll
            for (uint32_t t = 0; t < T; ++t) {
                words[t] = ~0ull;
                if (!all) {
                    const uint64_t mine = valid && j == t ? there : 0;
                    words[t] = (uint64_t)__reduce_or_sync(0xffffffffu, (uint32_t)(mine >> 32)) << 32 |
                               __reduce_or_sync(0xffffffffu, (uint32_t)mine);
                }
            }
            ok = wait_phase(&sm.empty[at.slot], at.parity ^ 1u, &sm.stop, a.wait_limit);
            if (!ok) break;
            if (lane == 0) {
                sm.even[at.slot] = all;
#pragma unroll
                for (uint32_t t = 0; t < T; ++t) sm.there[at.slot][t] = words[t];
                mbar_arrive_expect_tx(&sm.full[at.slot], (units << log_rows) * row_bytes);
            }
            __syncwarp();
            if (valid && !(HOOK == Hook::kWithheld && issued == 0)) {
                const uint32_t idx = fast_div(p, a.ps);
                copy(j, unit, p - idx * a.ps.d, page);
            }
            __syncwarp();
            at.step();
            ++issued;
        }
        if (ok) w.next(a.split);
    }
    if (bad_page) flag(a.err_flags, KVW_ERR_PAGE);
    if (!ok && lane == 0) flag(a.err_flags, KVW_ERR_TIMEOUT);
    // Whether or not this warp had to wait in vain: it leaves when the last copy
    // into each place has landed, or after a bounded time.
    const uint32_t n = issued < (uint32_t)Sh::kSlots ? issued : (uint32_t)Sh::kSlots;
    for (uint32_t i = 0; i < n; ++i) {
        const uint32_t x = issued - 1 - i;
        leave_phase<HOOK>(&sm.full[x % Sh::kSlots], (x / Sh::kSlots) & 1u, a.wait_limit,
                          a.err_flags);
    }
    for (uint32_t i = 0; i < (uint32_t)Sh::kQBufs; ++i)
        leave_phase<HOOK>(&sm.q_full[i], q_at.parity ^ (i < q_at.slot ? 0u : 1u), a.wait_limit,
                          a.err_flags);
}

// D = A B + C, with C in registers of its own.
__device__ __forceinline__ void mma_from(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1, const float (&c)[4]) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%10,%11,%12,%13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]),
          "f"(c[2]), "f"(c[3]));
}

// The transpose of an 8 x 8 block of fp16 values.
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

template <int D, Mods MODS, Hook HOOK>
__global__ void __launch_bounds__(Shape4<D>::kThreads, Shape4<D>::kCtas)
    gqa_int4_kernel(const GqaArgs a, const __grid_constant__ Int4Maps maps) {
    using Sh = Shape4<D>;
    constexpr int CH = Sh::kChunks, NG = Sh::kGroups, W = Sh::kWarps;
    constexpr uint32_t kLow = 0x000f000fu, kHigh = 0x00f000f0u;  // pairs of codes
    constexpr uint32_t kEight = 0x00080008u, kEights = 0x00800080u;  // 8, as these are
    extern __shared__ __align__(1024) unsigned char dyn[];
    Smem4<D>& sm = *reinterpret_cast<Smem4<D>*>(dyn);

    const uint32_t tid = threadIdx.x, warp = tid >> 5, lane = tid & 31u;
    // the join of the pieces may be scheduled; it waits for this grid's end
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (tid == Sh::kThreads - 32) {
        for (int i = 0; i < Sh::kSlots; ++i) {
            mbar_init(&sm.full[i], 1);
            mbar_init(&sm.empty[i], W);
        }
        for (int i = 0; i < Sh::kQBufs; ++i) {
            mbar_init(&sm.q_full[i], 1);
            mbar_init(&sm.q_empty[i], W);
        }
        mbar_init(&sm.meet, W);
        sm.stop = 0;
        mbar_init_fence();
        prefetch_map(&maps.codes.map[0]);
        prefetch_map(&maps.scales);
    }
    wait_for_stream();
    const bool ok = find_piece(a.split, a.pieces, blockIdx.x / a.lanes, sm.split);
    OpenPiece* open = reinterpret_cast<OpenPiece*>(a.workspace) + blockIdx.x;
    if (tid == 0) open->n = 0;
    if (!ok) {
        if (blockIdx.x == 0 && tid == 0) flag(a.err_flags, KVW_ERR_OFFSETS);
        return;
    }
    if (warp == W) {
        feed4<D, HOOK>(a, maps, sm);
        return;
    }

    // `warp` is also the slice of 16 positions of every tile that the warp takes
    const uint32_t quad = lane >> 2, in_quad = lane & 3u;
    RingPos<Sh::kSlots> at;
    RingPos<Sh::kQBufs> q_at;
    uint32_t meet_parity = 0;
    // the consumers meet (bounded, so that one that gave up strands nobody)
    auto meet = [&]() {
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.meet);
        const bool met = wait_phase(&sm.meet, meet_parity, &sm.stop, a.wait_limit);
        meet_parity ^= 1u;
        return met;
    };
    // ---- places of this lane's operands in a tile, the same for every tile
    const uint32_t log_rows = maps.codes.log_rows;
    constexpr int kPlaces = Sh::kLean ? 1 : NG;
    uint32_t k_at[kPlaces], v_at[kPlaces];  // chunks 2 g and 2 g + 1
    {
        const uint32_t row = warp * 16 + 2 * (lane & 7u) + ((lane >> 3) & 1u);
#pragma unroll
        for (int g = 0; g < kPlaces; ++g) {
            const uint32_t c = 2 * g + (lane >> 4) < (uint32_t)CH ? 2 * g + (lane >> 4) : 2 * g;
            k_at[g] = code_at<D>(log_rows, 0, row, c);
            v_at[g] = code_at<D>(log_rows, 1, row, c);
        }
    }
    // (a row of 256 codes is a line: its chunks 2 g and 0 lie 32 g apart but for
    // the swizzle)
    auto place = [&](const uint32_t(&x)[kPlaces], int g) {
        return Sh::kLean ? x[0] ^ (32u * g) : x[Sh::kLean ? 0 : g];
    };
    // scales of positions 2 * quad and the next of the slice; groups 2R bytes apart
    const uint32_t s_group = 2u << log_rows;
    const uint32_t s_at = ((warp * 16) >> log_rows) * scale_unit(NG, log_rows) +
                          2 * (((warp * 16) & ((1u << log_rows) - 1u)) + 2 * quad);

    bool alive = true;
    if constexpr (HOOK == Hook::kAbandoned) {
        *reinterpret_cast<volatile uint32_t*>(&sm.stop) = 1;
        alive = false;
    }
    while (alive) {
        // ---- queries: B operands, fp16 rows brought into range by 2^x
        alive = wait_phase(&sm.q_full[q_at.slot], q_at.parity, &sm.stop, a.wait_limit);
        if (!alive) break;
        const Segment& seg = sm.segment[q_at.slot];
        const uint32_t count = seg.count, rows = seg.rows;
        if (count == 0) break;
        if (seg.past && tid == 0) flag(a.err_flags, KVW_ERR_PAGE);
        // Operands of chunk c come from warp c mod 4, for all warps: in registers
        // they would leave too few for the tiles.  (The last meeting of the segment
        // before this one lies behind all reads of the old ones.)
        float qs[2];         // factors of rows 2 * in_quad and the next, whose scores the lane has
        uint32_t token = 0;  // and their tokens in the chunk, 16 bits each
        {
            const unsigned char* q = sm.q_raw[q_at.slot] + quad * Sh::kQPitch + 16 * in_quad;
            auto raw = [&](uint32_t c) {  // eight columns of row quad
                const uint4 v = *reinterpret_cast<const uint4*>(q + 64 * c);
                return quad < rows ? v : make_uint4(0, 0, 0, 0);
            };
            uint32_t top = 0;
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                const uint4 v = raw(c);
                top = __vmaxu2(top, __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu),
                                             __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu)));
            }
#pragma unroll
            for (int o = 1; o < 4; o <<= 1)
                top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, o));
            float up, down;
            row_power(max(top & 0xffffu, top >> 16), up, down);
            // products are of codes 2^-24 as large; scores in units of log2 straight
            // from the product, or 2 log2(e) / cap of them
            float by = a.sm_scale * down * 0x1p24f;
            by *= MODS == Mods::kCap ? a.cap_factor : kLog2e;
            // never 0, a masked score is -inf times this, and never infinite
            by = fminf(fmaxf(by, 1.17549435e-38f), 3.4028234e38f);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                qs[e] = __shfl_sync(0xffffffffu, by, 8 * in_quad + 4 * e);
                if (seg.tokens > 1) token |= (2 * in_quad + e) / seg.in_block << (16 * e);
            }
            const float up16 = up * 0.0625f;
#pragma unroll 1
            for (uint32_t c = warp; c < (uint32_t)CH; c += W) {
                const uint4 v = raw(c);
                // columns i and i + 4 of the lane's eight, i = 0 .. 3
                sm.q[c][lane] =
                    make_uint4(pack2<true>(bf16_lo(v.x) * up, bf16_lo(v.z) * up),
                               pack2<true>(bf16_hi(v.x) * up16, bf16_hi(v.z) * up16),
                               pack2<true>(bf16_lo(v.y) * up, bf16_lo(v.w) * up),
                               pack2<true>(bf16_hi(v.y) * up16, bf16_hi(v.w) * up16));
            }
        }
        alive = meet();
        if (!alive) break;
        const uint32_t eights_k[4] = {kEight, kEight, kEights, kEights};
        const uint32_t eights_v[4] = {kEight, kEights, kEight, kEights};
        // -8 sum of a group's queries, in units of the products
        [[maybe_unused]] float off[NG][4];
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            float x[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int c = 2 * g; c < 2 * g + 2 && c < CH; ++c) {
                const uint4 q = sm.q[c][lane];
                mma16816<true>(x, eights_k, q.x, q.y);
                mma16816<true>(x, eights_k, q.z, q.w);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) off[g][e] = -x[e];
            if (Sh::kLean && quad == 0) sm.off[warp][g][in_quad] = make_float2(-x[0], -x[1]);
        }
        if constexpr (Sh::kLean) __syncwarp();
        auto token_of = [&](int e) { return (token >> (16 * e)) & 0xffffu; };
        // distance biases of the lane's rows, and the rows' distances from its first
        // position in tile 0 (those of positions that a row sees fit 32 bits)
        [[maybe_unused]] float slope[2];
        [[maybe_unused]] uint32_t far[2];
        if constexpr (MODS != Mods::kNone) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const uint32_t r = 2 * in_quad + e;
                far[e] = (uint32_t)(seg.pos0 + token_of(e) - seg.p_first) - warp * 16 - 2 * quad;
                slope[e] = a.slopes && r < rows
                               ? kLog2e * __ldg(a.slopes + seg.head0 + (r - token_of(e) * seg.in_block))
                               : 0.0f;
            }
        }

        float acc[CH][2][4], less[NG][4];  // O^T, and 8 sum (P s_v) in its units
        // the rows' references and sums; a row that has seen no position has m =
        // -inf, subtracts 0 and has a sum that asks for a reference
        float m[2] = {-INFINITY, -INFINITY}, ref[2] = {0.0f, 0.0f}, l[2] = {kUnset, kUnset};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
#pragma unroll
            for (int c = 0; c < CH; ++c) acc[c][0][e] = acc[c][1][e] = 0.0f;
#pragma unroll
            for (int g = 0; g < NG; ++g) less[g][e] = 0.0f;
        }

        // The warp's slices of N tiles of the place at `at`, from its tile j on,
        // tile k of the segment; EDGE: positions may be missing, or seen by some
        // rows only.
        auto tiles = [&](uint32_t j, uint32_t k, bool release, auto n_const, auto edge_const) {
            constexpr int N = decltype(n_const)::value;
            constexpr bool EDGE = decltype(edge_const)::value;
            static_assert(N == 1 || !EDGE, "edge tiles are taken one by one");
            const uint32_t codes = smem_addr(sm.codes[at.slot][j]);
            const unsigned char* sc = sm.scales[at.slot][j] + s_at;
            auto scales_of = [&](int i, int g) {  // of both positions; values' after the keys'
                return *reinterpret_cast<const uint32_t*>(sc + i * Sh::kScales + g * s_group);
            };
            // ---- S^T = K Q^T; score e: row 2 * in_quad + e % 2, position 2 * quad + e / 2
            float s[N][4];
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                float x[N][4];
                uint32_t kw[N][4];
#pragma unroll
                for (int i = 0; i < N; ++i) ldsm4(kw[i], codes + i * Sh::kCodes + place(k_at, g));
#pragma unroll
                for (int c = 0; c < 2 && 2 * g + c < CH; ++c) {
                    const uint4 q = sm.q[2 * g + c][lane];
#pragma unroll
                    for (int i = 0; i < N; ++i) {
                        const uint32_t u = kw[i][2 * c], v = kw[i][2 * c + 1];
                        const uint32_t u8 = u >> 8, v8 = v >> 8;
                        const uint32_t f0[4] = {u & kLow, v & kLow, u & kHigh, v & kHigh};
                        const uint32_t f1[4] = {u8 & kLow, v8 & kLow, u8 & kHigh, v8 & kHigh};
                        if (c > 0) {
                            mma16816<true>(x[i], f0, q.x, q.y);
                        } else if constexpr (Sh::kLean) {
                            const float none[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                            mma_from(x[i], f0, q.x, q.y, none);
                        } else {
                            mma_from(x[i], f0, q.x, q.y, off[g]);
                        }
                        mma16816<true>(x[i], f1, q.z, q.w);
                    }
                }
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    const uint32_t by = scales_of(i, g);
                    if constexpr (Sh::kLean) {
                        const float2 o = sm.off[warp][g][in_quad];
#pragma unroll
                        for (int e = 0; e < 4; ++e) x[i][e] += e & 1 ? o.y : o.x;
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float f = e < 2 ? bf16_lo(by) : bf16_hi(by);
                        s[i][e] = g == 0 ? f * x[i][e] : fmaf(f, x[i][e], s[i][e]);
                    }
                }
            }
            // ---- cap, distance bias, mask
            // (scores of kNone are brought into units of log2 with the weights)
            if constexpr (MODS == Mods::kCap) {
                // tanh as in gqa_decode_paged.cu: 1 - 2 / (2^u + 1), its odd series
                // where that loses small scores
#pragma unroll
                for (int x = 0; x < 4 * N; ++x) {
                    float& y = s[x / 4][x % 4];
                    const float u = y * qs[x & 1], v = u * u;
                    const float near = a.cap_half * u *
                                       fmaf(v, fmaf(v, fmaf(v, -kTanh7, kTanh5), -kTanh3), 1.0f);
                    const float far = a.softcap - __fdividef(2.0f * a.softcap, fast_exp2(u) + 1.0f);
                    y = fabsf(u) < kTanhNear ? near : far;
                }
            }
            if (MODS == Mods::kBias || (MODS == Mods::kCap && a.slopes)) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float f = MODS == Mods::kCap ? 1.0f : qs[e];
                    const float bias = -slope[e] * (float)(far[e] - k * kTile);
#pragma unroll
                    for (int i = 0; i < N; ++i) {
                        const float nearer = i == 0 ? bias : fmaf(slope[e], (float)(kTile * i), bias);
                        s[i][e] = fmaf(s[i][e], f, nearer);
                        s[i][2 + e] = fmaf(s[i][2 + e], f, nearer + slope[e]);
                    }
                }
            }
            [[maybe_unused]] uint32_t seen = 0;  // bit e: score e counts
            if constexpr (EDGE) {
                const int64_t p0 = seg.p_first + (int64_t)k * kTile + warp * 16 + 2 * quad;
                const uint32_t there = (uint32_t)(sm.there[at.slot][j] >> (warp * 16 + 2 * quad));
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int64_t p = p0 + e / 2, last = seg.pos0 + token_of(e & 1);
                    if (((there >> (e / 2)) & 1u) && p <= last && p > last - a.split.window)
                        seen |= 1u << e;
                    else
                        s[0][e] = -INFINITY;
                }
            }
            auto kept = [&](int e) { return !EDGE || ((seen >> e) & 1u); };
            // ---- weights, and weights times scales of the values
            float sum[N][2];       // of the rows' weights
            uint32_t b[N][NG][2];  // rows 2 * in_quad and the next, of either position
            auto weights = [&]() {
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    float p[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        p[e] = fast_exp2(MODS == Mods::kNone
                                             ? fmaf(s[i][e], qs[e & 1], -ref[e & 1])
                                             : s[i][e] - ref[e & 1]);
                    sum[i][0] = p[0] + p[2];
                    sum[i][1] = p[1] + p[3];
#pragma unroll
                    for (int g = 0; g < NG; ++g) {
                        const uint32_t by = scales_of(i, NG + g);
                        float x[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            x[e] = p[e] * (e < 2 ? bf16_lo(by) : bf16_hi(by));
                            if (!kept(e)) x[e] = 0.0f;  // whatever its scale holds
                        }
                        b[i][g][0] = pack2<true>(x[0], x[1]);
                        b[i][g][1] = pack2<true>(x[2], x[3]);
                    }
                }
            };
            uint32_t vw[N][4];  // the first group's values are on their way meanwhile
#pragma unroll
            for (int i = 0; i < N; ++i) ldsm4_trans(vw[i], codes + i * Sh::kCodes + place(v_at, 0));
            weights();
            // Does a row's reference have to rise?  (The patterns are those of
            // numbers that are not negative; a NaN's, and those of negative
            // scales, are above 2^15's.)
            uint32_t top = 0;
            float most_sum = fmaxf(l[0], l[1]);
#pragma unroll
            for (int i = 0; i < N; ++i) {
#pragma unroll
                for (int g = 0; g < NG; ++g)
                    top = __vmaxu2(top, __vmaxu2(b[i][g][0], b[i][g][1]));
                most_sum = fmaxf(most_sum, fmaxf(sum[i][0], sum[i][1]));
            }
            if (__any_sync(0xffffffffu,
                           most_sum > kMostSum || __vcmpgtu2(top, 0x78007800u) != 0)) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    // the row's largest weight times scale, in log2, its sum so far as
                    // a position of zero values
                    float most = m[e] + __log2f(l[e] * kLeastScale);
#pragma unroll
                    for (int y = 0; y < 2 * N; ++y) {
                        const int i = y / 2, h = y % 2;
                        float by = kLeastScale;
#pragma unroll
                        for (int g = 0; g < NG; ++g) {
                            const uint32_t x = scales_of(i, NG + g);
                            by = fmaxf(by, fabsf(h ? bf16_hi(x) : bf16_lo(x)));
                        }
                        const float x = s[i][2 * h + e] * (MODS == Mods::kNone ? qs[e] : 1.0f);
                        if (kept(2 * h + e)) most = fmaxf(most, x + __log2f(by));
                    }
#pragma unroll
                    for (int o = 4; o < 32; o <<= 1)
                        most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
                    const float next = fmaxf(m[e], most - weight_lift<true>());
                    const float f = next == m[e] ? 1.0f : fast_exp2(m[e] - next);
                    m[e] = next;
                    ref[e] = next == -INFINITY ? 0.0f : next;
                    l[e] *= f;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
#pragma unroll
                        for (int c = 0; c < CH; ++c) {
                            acc[c][0][2 * h + e] *= f;
                            acc[c][1][2 * h + e] *= f;
                        }
#pragma unroll
                        for (int g = 0; g < NG; ++g) less[g][2 * h + e] *= f;
                    }
                }
                weights();
            }
#pragma unroll
            for (int i = 0; i < N; ++i) {
                l[0] += sum[i][0];
                l[1] += sum[i][1];
            }
            // ---- O^T += V^T (P s_v)^T
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                if (g > 0) {
#pragma unroll
                    for (int i = 0; i < N; ++i)
                        ldsm4_trans(vw[i], codes + i * Sh::kCodes + place(v_at, g));
                }
                if (g == NG - 1 && release) {
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sm.empty[at.slot]);
                }
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    const uint32_t b0 = transposed(b[i][g][0]), b1 = transposed(b[i][g][1]);
                    mma16816<true>(less[g], eights_v, b0, b1);
#pragma unroll
                    for (int c = 0; c < 2 && 2 * g + c < CH; ++c) {
                        const uint32_t x = vw[i][2 * c], y = vw[i][2 * c + 1];
                        const uint32_t x8 = x >> 8, y8 = y >> 8;
                        const uint32_t f0[4] = {x & kLow, x & kHigh, y & kLow, y & kHigh};
                        const uint32_t f1[4] = {x8 & kLow, x8 & kHigh, y8 & kLow, y8 & kHigh};
                        mma16816<true>(acc[2 * g + c][0], f0, b0, b1);
                        mma16816<true>(acc[2 * g + c][1], f1, b0, b1);
                    }
                }
            }
        };
        using One = std::integral_constant<int, 1>;
        using All = std::integral_constant<int, Sh::kTiles>;
        for (uint32_t place = (count + Sh::kTiles - 1) / Sh::kTiles; place-- > 0;) {
            const uint32_t k = place * Sh::kTiles;
            alive = wait_phase(&sm.full[at.slot], at.parity, &sm.stop, a.wait_limit);
            if (!alive) break;
            if (sm.even[at.slot]) {
                tiles(0, k, true, All{}, std::false_type{});
            } else {
                const uint32_t n = count - k < Sh::kTiles ? count - k : Sh::kTiles;
#pragma unroll 1
                for (uint32_t j = 0; j < n; ++j)
                    tiles(j, k + j, j + 1 == n, One{}, std::true_type{});
            }
            at.step();
        }
        if (!alive) break;

        // ---- the warps join, a few rows at a time
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            if (m[e] == -INFINITY) l[e] -= kUnset;  // 0, or NaN
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) l[e] += __shfl_xor_sync(0xffffffffu, l[e], o);
            if (quad == 0) {
                sm.m[warp][2 * in_quad + e] = m[e];
                sm.l[warp][2 * in_quad + e] = l[e];
            }
        }
        float* part = slot_of<Sh::kPadded>(a.workspace, blockIdx.x, seg.slot1 ? 1 : 0);
        constexpr uint32_t JR = Sh::kJoinRows, quads = D / 4;
#pragma unroll
        for (uint32_t round = 0; round < Sh::kBlock / JR; ++round) {
            if (round * JR >= rows) break;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const uint32_t r = 2 * in_quad + e;
                if (r / JR != round) continue;
                float* mine = sm.join[warp][r % JR] + 4 * quad;
#pragma unroll
                for (int c = 0; c < CH; ++c) {
                    const float lo = less[c / 2][e], hi = less[c / 2][2 + e];
                    *reinterpret_cast<float4*>(mine + 32 * c) = make_float4(
                        (acc[c][0][e] - lo) * 0x1p24f, (acc[c][0][2 + e] - hi) * 0x1p20f,
                        (acc[c][1][e] - lo) * 0x1p24f, (acc[c][1][2 + e] - hi) * 0x1p20f);
                }
            }
            alive = meet();
            if (!alive) break;
            const uint32_t here = rows - round * JR < JR ? rows - round * JR : JR;
            for (uint32_t x = tid; x < here * quads; x += 32 * W) {
                const uint32_t rj = x / quads, d = (x - rj * quads) * 4, r = round * JR + rj;
                float top = sm.m[0][r];
#pragma unroll
                for (int v = 1; v < W; ++v) top = fmaxf(top, sm.m[v][r]);
                const float base = top == -INFINITY ? 0.0f : top;
                float sum = 0.0f;
                float4 o = make_float4(0, 0, 0, 0);
#pragma unroll
                for (int v = 0; v < W; ++v) {
                    const float f = fast_exp2(sm.m[v][r] - base);
                    const float4 y = *reinterpret_cast<const float4*>(sm.join[v][rj] + d);
                    sum += f * sm.l[v][r];
                    o.x += f * y.x;
                    o.y += f * y.y;
                    o.z += f * y.z;
                    o.w += f * y.w;
                }
                if (seg.whole) {
                    const uint32_t ct = r / seg.in_block;
                    const uint64_t row =
                        (uint64_t)(seg.t + ct) * a.Hq + seg.head0 + (r - ct * seg.in_block);
                    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
                    uint2 y;
                    y.x = pack_bf16x2(o.x * inv, o.y * inv);
                    y.y = pack_bf16x2(o.z * inv, o.w * inv);
                    *reinterpret_cast<uint2*>(a.out + row * D + d) = y;
                    if (d == 0 && a.lse)
                        a.lse[row] = sum == 0.0f ? -INFINITY : (top + log2f(sum)) * kLn2;
                } else {
                    *reinterpret_cast<float4*>(part + r * Sh::kPadded + d) = o;
                    if (d == 0) {
                        part[kRows * Sh::kPadded + r] = top;
                        part[kRows * Sh::kPadded + kRows + r] = sum;
                    }
                }
            }
            alive = meet();
            if (!alive) break;
        }
        if (!alive) break;
        if (seg.shared_by && tid == 0) {
            OpenPiece x;
            x.n = seg.shared_by;
            x.t = seg.t;
            x.tokens = seg.tokens;
            x.block = seg.block;
            *open = x;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.q_empty[q_at.slot]);
        q_at.step();
    }
    if (!alive && lane == 0) flag(a.err_flags, KVW_ERR_TIMEOUT);
}

template <int D, Mods MODS, Hook HOOK>
cudaError_t launch_as(GqaArgs& a, const Int4Maps& maps, cudaStream_t stream) {
    using Sh = Shape4<D>;
    constexpr size_t smem = sizeof(Smem4<D>);
    static_assert(smem <= (Sh::kCtas == 3 ? 75 : 113) * 1024, "shared memory of an SM");
    uint64_t wave = 0;
    cudaError_t e = wave_ctas<&gqa_int4_kernel<D, MODS, HOOK>>(Sh::kThreads, smem, wave);
    if (e != cudaSuccess) return e;
    if (wave == 0) return cudaErrorInvalidConfiguration;
    // Where two CTAs per SM would have a tile each at most, as far as the page table
    // reaches, two leave the join's blocks room to wait beside them (one token over
    // 901 positions 10.4 -> 9.7 us).  Longer contexts want all three: one token over
    // 4096 positions 12.1 us against 12.7, 32768 17.6 against 19.1, 131072 34.4 against
    // 37.5 (heads of 64, two requests: 28.5, 31.9); two requests of 32768 20.8, 19.6.
    const uint64_t two = wave - wave / 3;
    const uint64_t tiles = (uint64_t)(a.split.cap + kTile - 1) / kTile;
    if (Sh::kCtas == 3 && tiles * a.split.T * a.split.blocks <= two) wave = two;
    const uint32_t ctas = side_by_side(a, wave);
    e = launch_early(&gqa_int4_kernel<D, MODS, HOOK>, dim3(ctas), Sh::kThreads, smem, stream, a,
                     maps);
    if (e != cudaSuccess) return e;
    return launch_join<Sh::kPadded, Sh::kBlock>(a, ctas, stream);
}

template <int D, Hook HOOK>
int launch(GqaArgs& a, const kvw_paged_cache_t* cache, const kva_group_scales_t* scales,
           uint32_t layer_idx, cudaStream_t stream) {
    Int4Maps maps;
    const int st = encode_int4_maps(&maps, cache, scales, layer_idx);
    if (st != KVW_OK) return st;
    const cudaError_t e = a.softcap > 0.0f ? launch_as<D, Mods::kCap, HOOK>(a, maps, stream)
                          : a.slopes       ? launch_as<D, Mods::kBias, HOOK>(a, maps, stream)
                                           : launch_as<D, Mods::kNone, HOOK>(a, maps, stream);
    return e == cudaSuccess ? KVW_OK : KVW_ECUDA;
}

// Strides that a tensor map takes (see tma_strides_ok), of codes and scales that
// check_int4 has found positive.
bool int4_strides_ok(const kvw_paged_cache_t* c, const kva_group_scales_t* s) {
    auto ok = [](int64_t codes, int64_t scales, uint64_t n) {
        return n <= 1 || (codes / 2 < (1ll << 40) && scales < (1ll << 39));
    };
    return ok(c->stride_head, s->stride_head, c->num_heads) &&
           ok(c->stride_page, s->stride_page, c->num_pages) && ok(c->stride_kv, s->stride_kv, 2);
}

int int4_entry(void* out, float* lse, const void* q, int64_t q_row_stride,
               const uint32_t* input_row_offsets, uint32_t num_batches, uint32_t tot_seq_len,
               uint32_t num_q_heads, const kvw_paged_cache_t* cache,
               const kva_group_scales_t* scales, uint32_t layer_idx, float sm_scale, float softcap,
               uint32_t window, const float* alibi_slopes, void* workspace,
               uint64_t workspace_bytes, uint32_t* err_flags, cudaStream_t stream, Hook hook,
               uint64_t wait_ns) {
    const int st = check_int4(cache, scales, layer_idx);
    if (st != KVW_OK) return st;
    GqaArgs a = {};
    const int bad = gqa_arguments(a, out, lse, q, q_row_stride, input_row_offsets, num_batches,
                                  tot_seq_len, num_q_heads, cache, sm_scale, softcap, window,
                                  alibi_slopes, workspace, workspace_bytes, err_flags,
                                  tma_sizes_ok(cache), true, int4_strides_ok(cache, scales),
                                  Shape4<64>::kBlock);
    if (bad != KVW_OK || tot_seq_len == 0) return bad;
    a.k_scale = a.v_scale = 1.0f;
    // a segment's cost beside its tiles, in tiles (64 requests of 4 tokens with 1: 115
    // us, 3: 109, 5: 107, 8: 111; one token each, up to 512: 38, 36, 35, 36)
    a.split.overhead = 5;
    a.wait_limit = wait_cycles(wait_ns);
    auto run = [&](auto d) {
        constexpr int D = decltype(d)::value;
#ifdef KVW_TEST_HOOKS
        if (hook == Hook::kWithheld)
            return launch<D, Hook::kWithheld>(a, cache, scales, layer_idx, stream);
        if (hook == Hook::kAbandoned)
            return launch<D, Hook::kAbandoned>(a, cache, scales, layer_idx, stream);
#else
        if (hook != Hook::kNone) return (int)KVW_EUNSUPPORTED;
#endif
        return launch<D, Hook::kNone>(a, cache, scales, layer_idx, stream);
    };
    switch (a.D) {
        case 64: return run(std::integral_constant<int, 64>{});
        case 96: return run(std::integral_constant<int, 96>{});
        case 128: return run(std::integral_constant<int, 128>{});
        default: return run(std::integral_constant<int, 256>{});
    }
}

}  // namespace
}  // namespace kvw

extern "C" int kva_gqa_decode_int4(void* out, float* lse, const void* q, int64_t q_row_stride,
                                   const uint32_t* input_row_offsets, uint32_t num_batches,
                                   uint32_t tot_seq_len, uint32_t num_q_heads,
                                   const kvw_paged_cache_t* cache,
                                   const kva_group_scales_t* scales, uint32_t layer_idx,
                                   float sm_scale, float softcap, uint32_t window,
                                   const float* alibi_slopes, void* workspace,
                                   uint64_t workspace_bytes, uint32_t* err_flags,
                                   cudaStream_t stream) {
    return kvw::int4_entry(out, lse, q, q_row_stride, input_row_offsets, num_batches, tot_seq_len,
                           num_q_heads, cache, scales, layer_idx, sm_scale, softcap, window,
                           alibi_slopes, workspace, workspace_bytes, err_flags, stream,
                           kvw::Hook::kNone, kvw::kWaitLimitNs);
}

#ifdef KVW_TEST_HOOKS
// Test builds only: as in gqa_decode_paged.cu, the first tile of every CTA is
// announced but never copied, or the consumers leave at once.
extern "C" int kva_test_gqa_int4(void* out, const void* q, int64_t q_row_stride,
                                 const uint32_t* input_row_offsets, uint32_t num_batches,
                                 uint32_t tot_seq_len, uint32_t num_q_heads,
                                 const kvw_paged_cache_t* cache, const kva_group_scales_t* scales,
                                 uint32_t layer_idx, void* workspace, uint64_t workspace_bytes,
                                 uint32_t* err_flags, cudaStream_t stream, uint64_t wait_ns,
                                 int abandoned) {
    return kvw::int4_entry(out, nullptr, q, q_row_stride, input_row_offsets, num_batches,
                           tot_seq_len, num_q_heads, cache, scales, layer_idx, 0.1f, 0.0f, 0,
                           nullptr, workspace, workspace_bytes, err_flags, stream,
                           abandoned ? kvw::Hook::kAbandoned : kvw::Hook::kWithheld, wait_ns);
}
#endif
