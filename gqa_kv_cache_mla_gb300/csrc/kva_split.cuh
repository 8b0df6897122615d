// How the attention calls of kva.h divide their work, and how the pieces
// meet again.
//
// Work is counted in units: one unit is one tile of kTile cache positions for
// one row block (a group of query heads that read the same rows) of one
// token.  The units of all tokens in order - token, row block, tile - form
// one long axis, cut into G pieces of equal length, one for each CTA (or CTA
// pair).  So every CTA reads the same amount of cache whatever the lengths, a
// CTA crosses from one token to the next where its piece does, and at most
// two of its segments are parts of a (token, row block) that other CTAs
// share: its first (slot 0) and its last (slot 1).  Those write their
// unnormalised sums with their running maximum and sum to a workspace whose
// size depends on G alone, and a second kernel joins them in order, so the
// result depends on nothing but the lengths and G.
//
// The number of tiles of one token's context is needed as a prefix sum over
// tokens.  A request's tokens have consecutive lengths, so its total is a
// difference of two closed forms (tiles_upto), one evaluation for each
// request; a CTA finds its start by one block-wide scan over requests and a
// search within one request.
#pragma once

#include "kva_common.cuh"

namespace kvw {

constexpr uint32_t kTile = 64;        // cache positions of one unit
constexpr uint32_t kMaxPieces = 512;  // G, and so the workspace, is bounded by this

struct SplitArgs {
    const uint32_t* offsets;
    const uint32_t* cache_lengths;
    uint32_t B, T;
    uint32_t blocks;  // row blocks per token
    uint32_t min_units;  // a piece is at least this long (fewer pieces for little work)
    uint64_t cap;     // positions the page tables can hold
    uint64_t window;  // positions seen, own included (a huge number for no window)
};

// Positions a token at length `len` (its own position + 1) reads: [start, hi),
// tiles [start / kTile, ceil(hi / kTile)).  Positions past the page table's
// reach are left out; at least one tile is kept so that every token has an
// owner for its output row.
struct TokenSpan {
    uint64_t start, hi;
    uint32_t tile0, tiles;
};

__device__ __forceinline__ TokenSpan token_span(const SplitArgs& a, uint64_t len) {
    TokenSpan s;
    s.start = len > a.window ? len - a.window : 0;
    s.hi = len < a.cap ? len : a.cap;
    const uint64_t first = s.start < s.hi ? s.start : s.hi - 1;
    s.tile0 = (uint32_t)(first / kTile);
    s.tiles = (uint32_t)((s.hi + kTile - 1) / kTile) - s.tile0;
    return s;
}

// Sum of token_span(l).tiles over lengths l = 1 .. x.
__device__ __forceinline__ uint64_t tiles_upto(const SplitArgs& a, uint64_t x) {
    // sum of ceil(min(l, cap) / kTile)
    const uint64_t u = x < a.cap ? x : a.cap;
    const uint64_t uq = u / kTile, ur = u % kTile;
    uint64_t n = kTile * (uq * (uq + 1) / 2) + ur * (uq + 1);
    n += (x - u) * ((a.cap + kTile - 1) / kTile);
    // minus the sum of floor(min(l - window, cap - 1) / kTile) over l > window
    if (x > a.window) {
        const uint64_t y = x - a.window, v = y < a.cap - 1 ? y : a.cap - 1;
        const uint64_t vq = v / kTile, vr = v % kTile;
        n -= (vq ? kTile * (vq * (vq - 1) / 2) : 0) + vq * (vr + 1);
        n -= (y - v) * ((a.cap - 1) / kTile);
    }
    return n;
}

// First unit of piece c of `pieces` over `units` units (even to one unit).
__host__ __device__ __forceinline__ uint64_t piece_start(uint64_t units, uint32_t pieces,
                                                         uint32_t c) {
    const uint64_t q = units / pieces, r = units % pieces;
    return q * c + (c < r ? c : r);
}

// Pieces in use: never more than `most`, and none shorter than min_units
// unless there is only one.
__device__ __forceinline__ uint32_t pieces_of(const SplitArgs& a, uint64_t units, uint32_t most) {
    const uint64_t p = units / a.min_units;
    return p == 0 ? 1u : p < most ? (uint32_t)p : most;
}

// Where a piece starts.
struct PieceStart {
    uint64_t units;       // of the whole call
    uint64_t u0, u1;      // the piece
    uint64_t token_base;  // first unit of the token u0 lies in
    uint32_t pieces;
    uint32_t b, i;        // that token: request and index in it
};

// All threads of the CTA call this.  Returns false (uniformly) for malformed
// offsets.  `shared` needs THREADS / 32 + 1 uint64 and one PieceStart.
template <int THREADS>
struct SplitShared {
    uint64_t warp_sum[THREADS / 32];
    PieceStart start;
};

template <int THREADS>
__device__ __forceinline__ bool find_piece(const SplitArgs& a, uint32_t most, uint32_t c,
                                           SplitShared<THREADS>& sh, PieceStart& out) {
    const uint32_t tid = threadIdx.x, lane = tid & 31u, warp = tid >> 5;
    const uint32_t per = (a.B + THREADS - 1) / THREADS;
    const uint32_t lo = tid * per < a.B ? tid * per : a.B;
    const uint32_t hi = lo + per < a.B ? lo + per : a.B;
    uint64_t mine = 0;
    int ok = 1;
    for (uint32_t r = lo; r < hi; ++r) {
        const uint32_t o0 = __ldg(a.offsets + r), o1 = __ldg(a.offsets + r + 1);
        const uint64_t len = __ldg(a.cache_lengths + r);
        if (o1 < o0 || o1 > a.T || (r == 0 && o0 != 0) || (r == a.B - 1 && o1 != a.T))
            ok = 0;
        else
            mine += tiles_upto(a, len + (o1 - o0)) - tiles_upto(a, len);
    }
    uint64_t scan = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint64_t v = __shfl_up_sync(0xffffffffu, scan, o);
        if (lane >= (uint32_t)o) scan += v;
    }
    if (lane == 31) sh.warp_sum[warp] = scan;
    if (!__syncthreads_and(ok)) return false;
    uint64_t before = scan - mine, total = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
        if ((uint32_t)w < warp) before += sh.warp_sum[w];
        total += sh.warp_sum[w];
    }
    PieceStart s;
    s.units = total * a.blocks;
    s.pieces = pieces_of(a, s.units, most);
    const bool used = c < s.pieces;
    s.u0 = used ? piece_start(s.units, s.pieces, c) : s.units;
    s.u1 = used ? piece_start(s.units, s.pieces, c + 1) : s.units;
    s.token_base = 0;
    s.b = s.i = 0;
    // the one thread whose requests hold u0 walks them
    if (s.u0 < s.u1 && s.u0 >= before * a.blocks && s.u0 < (before + mine) * a.blocks) {
        uint64_t base = before;
        for (uint32_t r = lo; r < hi; ++r) {
            const uint64_t len = __ldg(a.cache_lengths + r);
            const uint32_t n = __ldg(a.offsets + r + 1) - __ldg(a.offsets + r);
            const uint64_t at = tiles_upto(a, len);
            const uint64_t tiles = tiles_upto(a, len + n) - at;
            if (s.u0 < (base + tiles) * a.blocks) {
                // largest i whose tokens before it end at or before u0
                uint32_t i0 = 0, i1 = n;
                while (i1 - i0 > 1u) {
                    const uint32_t mid = i0 + (i1 - i0) / 2;
                    if ((base + tiles_upto(a, len + mid) - at) * a.blocks <= s.u0)
                        i0 = mid;
                    else
                        i1 = mid;
                }
                s.b = r;
                s.i = i0;
                s.token_base = (base + tiles_upto(a, len + i0) - at) * a.blocks;
                break;
            }
            base += tiles;
        }
        sh.start = s;
    }
    __syncthreads();
    if (s.u0 < s.u1) s = sh.start;
    out = s;
    return true;
}

// A CTA's place on the axis of units; every thread keeps one, they agree.
struct Walk {
    uint64_t u, u1, token_base;
    uint32_t b, i, t, n;  // request, index in it, token, tokens of the request
    uint64_t len0;        // cache_lengths[b]
    TokenSpan span;

    __device__ __forceinline__ void load_request(const SplitArgs& a) {
        const uint32_t o = __ldg(a.offsets + b);
        n = __ldg(a.offsets + b + 1) - o;
        t = o + i;
        len0 = __ldg(a.cache_lengths + b);
    }
    __device__ __forceinline__ void begin(const SplitArgs& a, const PieceStart& s) {
        u = s.u0;
        u1 = s.u1;
        token_base = s.token_base;
        b = s.b;
        i = s.i;
        if (u < u1) {
            load_request(a);
            span = token_span(a, len0 + i + 1);
        }
    }
    // The segment at u: row block, first and last + 1 tile (counted from the
    // token's tile0), and the unit where the (token, row block) ends.
    __device__ __forceinline__ void segment(uint32_t& block, uint32_t& first, uint32_t& last,
                                            uint64_t& end) const {
        const uint64_t in = u - token_base;
        block = (uint32_t)(in / span.tiles);
        first = (uint32_t)(in - (uint64_t)block * span.tiles);
        end = token_base + (uint64_t)(block + 1) * span.tiles;
        const uint64_t stop = end < u1 ? end : u1;
        last = first + (uint32_t)(stop - u);
    }
    __device__ __forceinline__ void advance(const SplitArgs& a, uint32_t count) {
        u += count;
        if (u >= u1 || u < token_base + (uint64_t)a.blocks * span.tiles) return;
        token_base += (uint64_t)a.blocks * span.tiles;
        if (++i < n) {
            ++t;
        } else {
            i = 0;
            do {
                ++b;
                load_request(a);
            } while (n == 0);  // u < u1: a later request has tokens
        }
        span = token_span(a, len0 + i + 1);
    }
};

// What piece c left open: a (token, row block) that it began (slot 1) and
// that pieces c + 1 .. go on with (their slot 0).  `units` 0: nothing.
struct OpenPiece {
    uint64_t units, end;
    uint32_t pieces, t, block, pad;
};

static_assert(sizeof(OpenPiece) == 32, "workspace layout");

}  // namespace kvw
