// How the attention calls of kva.h divide their work, and how the pieces
// meet again.
//
// A chunk is up to C consecutive new tokens of one request (C a power of two;
// their query rows share a row block, so a cache row is read once for all of
// them).  Work is counted in units: one unit is one tile of kTile cache
// positions for one row block of one chunk; `overhead` further units stand
// before the tiles of every (chunk, row block) for what it costs to begin and
// end one.  The units of all chunks in order - chunk, row block, tile - form
// one long axis, cut into equal pieces, one for each CTA (or for each of
// several CTAs that take row blocks side by side; those are then not part of
// the axis).  So every CTA has the same work whatever the lengths, a CTA
// crosses from one chunk to the next where its piece does, and at most two of
// its segments are parts of a (chunk, row block) that other CTAs share: its
// first (slot 0) and its last (slot 1).  Those write their unnormalised sums
// with their running maximum and sum to a workspace whose size depends on the
// number of pieces alone, and a second kernel joins them in order: the result
// depends on the lengths and the device only.
//
// Finding a piece needs the number of tiles before a chunk, a prefix sum over
// chunks.  Within a request the chunks' lengths rise by C, so a request's
// prefix has a closed form (tiles_before); a CTA finds its start by one
// block-wide scan over requests and a binary search within one.
#pragma once

#include "kva_common.cuh"

namespace kvw {

constexpr uint32_t kTile = 64;        // cache positions of one unit
constexpr uint32_t kMaxPieces = 512;  // bounds the workspace
constexpr uint64_t kMaxReach = 0xffffff00ull;  // positions, all 32-bit, tiles included

struct SplitArgs {
    const uint32_t* offsets;
    const uint32_t* cache_lengths;
    uint32_t B, T;
    uint32_t blocks;     // row blocks per chunk
    uint32_t log_c;      // log2 of the tokens per chunk, <= 6
    uint32_t min_units;  // a piece is at least this long (fewer pieces for little work)
    uint32_t overhead;   // what beginning a (chunk, row block) costs, in units
    int64_t cap;         // positions the page tables can hold
    int64_t window;      // positions seen, own included (a huge number for no window)
};

// What a chunk reads: positions [start, hi), tiles tile0 .. tile0 + tiles - 1
// (its last token's length bounds hi, its first token's window start).
// Positions past the page tables' reach are left out; at least one tile is
// kept so that every token has an owner for its output row.
struct ChunkSpan {
    int64_t start, hi;
    uint32_t tile0, tiles, tokens;
};

// Chunk k of a request with n new tokens after len cached ones.
__host__ __device__ __forceinline__ ChunkSpan chunk_span(const SplitArgs& a, int64_t len,
                                                         uint32_t n, uint32_t k) {
    ChunkSpan s;
    const uint32_t first = k << a.log_c, left = n - first, c = 1u << a.log_c;
    s.tokens = left < c ? left : c;
    const int64_t begin = len + first + 1 - a.window, end = len + first + s.tokens;
    s.start = begin > 0 ? begin : 0;
    s.hi = end < a.cap ? end : a.cap;
    const int64_t at = s.start < s.hi ? s.start : s.hi - 1;
    s.tile0 = (uint32_t)(at / kTile);
    s.tiles = (uint32_t)((s.hi + kTile - 1) / kTile) - s.tile0;
    return s;
}

// Sum of min(ceil(l / m), top) over l = 1 .. x, m = 1 << log_m.
__host__ __device__ __forceinline__ int64_t sum_ceil(int64_t x, uint32_t log_m, int64_t top) {
    const int64_t flat = top << log_m, u = x < flat ? x : flat;
    const int64_t q = u >> log_m, r = u - (q << log_m);
    return ((q * (q + 1) / 2) << log_m) + r * (q + 1) + (x - u) * top;
}

// Sum of min(floor(l / m), top) over l = 0 .. x - 1 (nothing for x <= 0).
__host__ __device__ __forceinline__ int64_t sum_floor(int64_t x, uint32_t log_m, int64_t top) {
    if (x <= 0) return 0;
    const int64_t flat = top << log_m, u = x < flat ? x : flat;
    const int64_t q = u >> log_m, r = u - (q << log_m);
    return (q * (q - 1) / 2) * (1ll << log_m) + r * q + (x - u) * top;
}

// Tiles of the first k chunks of a request, all of them full ones: with c =
// 1 << log_c and m = kTile / c, chunk j ends in tile ceil((e + j + 1) / m),
// e = ceil(len / c), and starts in tile floor((f + j) / m), f = floor((len +
// 1 - window) / c), both cut at the page tables' reach.
__host__ __device__ __forceinline__ int64_t tiles_before(const SplitArgs& a, int64_t len,
                                                         uint32_t k) {
    if (k == 0) return 0;  // single tokens, the usual case
    const uint32_t log_m = 6 - a.log_c;
    const int64_t e = (len + (1ll << a.log_c) - 1) >> a.log_c;
    const int64_t f = (len + 1 - a.window) >> a.log_c;  // floor, also of a negative number
    const int64_t last = (a.cap + kTile - 1) / kTile, from = (a.cap - 1) / kTile;
    return sum_ceil(e + k, log_m, last) - sum_ceil(e, log_m, last) -
           sum_floor(f + k, log_m, from) + sum_floor(f, log_m, from);
}

// Units of one row block of the first k chunks.
__host__ __device__ __forceinline__ int64_t units_before(const SplitArgs& a, int64_t len,
                                                         uint32_t k) {
    return tiles_before(a, len, k) + (int64_t)k * a.overhead;
}

__host__ __device__ __forceinline__ uint32_t chunks_of(const SplitArgs& a, uint32_t n) {
    return (n >> a.log_c) + ((n & ((1u << a.log_c) - 1u)) ? 1u : 0u);
}

// Units of one row block of a whole request.
__host__ __device__ __forceinline__ int64_t request_units(const SplitArgs& a, int64_t len,
                                                          uint32_t n) {
    if (n == 0) return 0;
    const uint32_t k = chunks_of(a, n) - 1;
    return units_before(a, len, k) + chunk_span(a, len, n, k).tiles + a.overhead;
}

// Quotients of the axis, with the 32-bit division where it will do.
__host__ __device__ __forceinline__ uint64_t div_units(uint64_t x, uint64_t y) {
    return (x | y) >> 32 ? x / y : (uint32_t)x / (uint32_t)y;
}

// `units` units cut into `pieces` pieces, even to one unit: the first r pieces
// have q + 1, the others q.
struct Cut {
    uint64_t q, r;
    __host__ __device__ __forceinline__ Cut(uint64_t units, uint32_t pieces) {
        q = div_units(units, pieces);
        r = units - q * pieces;
    }
    // First unit of piece c, and the piece that holds unit u.
    __host__ __device__ __forceinline__ uint64_t start(uint32_t c) const {
        return q * c + (c < r ? c : r);
    }
    __host__ __device__ __forceinline__ uint32_t piece_of(uint64_t u) const {
        const uint64_t longer = (q + 1) * r;
        return (uint32_t)(u < longer ? div_units(u, q + 1) : r + div_units(u - longer, q));
    }
};

// Pieces in use: at most `most`, none shorter than min_units unless there is
// only one.
__host__ __device__ __forceinline__ uint32_t pieces_of(const SplitArgs& a, uint64_t units,
                                                       uint32_t most) {
    const uint64_t p = a.min_units == 1 ? units : div_units(units, a.min_units);
    return p == 0 ? 1u : p < most ? (uint32_t)p : most;
}

// Where a piece starts.
struct PieceStart {
    uint64_t units;       // of the whole call
    uint64_t u0, u1;      // the piece
    uint64_t chunk_base;  // first unit of the chunk u0 lies in
    uint32_t pieces;
    uint32_t b, k;        // that chunk: request and index in it
    uint32_t first, n, len;  // the request's first token, tokens and cache length
};

template <int THREADS>
struct SplitShared {
    int64_t warp_sum[THREADS / 32];
    PieceStart start;
};

// All threads of the CTA call this, with the same arguments.  Returns false
// (uniformly) for malformed offsets; else the piece is in sh.start.
template <int THREADS>
__device__ __forceinline__ bool find_piece(const SplitArgs& a, uint32_t most, uint32_t c,
                                           SplitShared<THREADS>& sh) {
    const uint32_t tid = threadIdx.x, lane = tid & 31u, warp = tid >> 5;
    const uint32_t per = (a.B + THREADS - 1) / THREADS;
    const uint32_t lo = tid * per < a.B ? tid * per : a.B;
    const uint32_t hi = lo + per < a.B ? lo + per : a.B;
    int64_t mine = 0;
    int ok = 1;
    uint32_t o0 = 0, o1 = 0, len = 0;  // of the thread's last request, usually its only one
    for (uint32_t r = lo; r < hi; ++r) {
        o0 = __ldg(a.offsets + r);
        o1 = __ldg(a.offsets + r + 1);
        len = __ldg(a.cache_lengths + r);
        if (o1 < o0 || o1 > a.T || (r == 0 && o0 != 0) || (r == a.B - 1 && o1 != a.T))
            ok = 0;
        else
            mine += request_units(a, len, o1 - o0);
    }
    int64_t scan = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, scan, o);
        if (lane >= (uint32_t)o) scan += v;
    }
    if (lane == 31) sh.warp_sum[warp] = scan;
    if (!__syncthreads_and(ok)) return false;
    int64_t before = scan - mine, total = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
        if ((uint32_t)w < warp) before += sh.warp_sum[w];
        total += sh.warp_sum[w];
    }
    PieceStart s;
    s.units = (uint64_t)total * a.blocks;
    s.pieces = pieces_of(a, s.units, most);
    const bool used = c < s.pieces;
    const Cut cut(s.units, s.pieces);
    s.u0 = used ? cut.start(c) : s.units;
    s.u1 = used ? cut.start(c + 1) : s.units;
    s.chunk_base = 0;
    s.b = s.k = s.first = s.n = s.len = 0;
    if (!used && tid == 0) sh.start = s;
    // the one thread whose requests hold u0 walks them
    if (used && s.u0 >= (uint64_t)before * a.blocks &&
        s.u0 < (uint64_t)(before + mine) * a.blocks) {
        int64_t base = before;
        uint32_t r = lo;
        if (hi - lo > 1) {
            for (;; ++r) {
                o0 = __ldg(a.offsets + r);
                o1 = __ldg(a.offsets + r + 1);
                len = __ldg(a.cache_lengths + r);
                const int64_t units = request_units(a, len, o1 - o0);
                if (r + 1 == hi || s.u0 < (uint64_t)(base + units) * a.blocks) break;
                base += units;
            }
        }
        // the last chunk that begins at or before u0
        uint32_t k0 = 0, k1 = chunks_of(a, o1 - o0);
        if (k1 > 1u) {
            const uint64_t at = div_units(s.u0, a.blocks);  // the chunk holds this unit of a row block
            while (k1 - k0 > 1u) {
                const uint32_t mid = k0 + (k1 - k0) / 2;
                if ((uint64_t)(base + units_before(a, len, mid)) <= at)
                    k0 = mid;
                else
                    k1 = mid;
            }
        }
        s.b = r;
        s.k = k0;
        s.first = o0;
        s.n = o1 - o0;
        s.len = len;
        s.chunk_base = (uint64_t)(base + units_before(a, len, k0)) * a.blocks;
        sh.start = s;
    }
    __syncthreads();
    return true;
}

// A place on the axis of units and the segment that begins there: the rest of
// a (chunk, row block), as far as the piece goes.
struct Walk {
    uint64_t u, u1, chunk_base;
    uint32_t b, k, t, n;  // request, chunk in it, the chunk's first token, tokens of the request
    uint32_t len0;        // cache_lengths[b]
    ChunkSpan span;
    // the segment: row block, units of the axis, tiles first .. last - 1 of
    // the span (at least one)
    uint32_t block, units, first, last;

    __device__ __forceinline__ void load_request(const SplitArgs& a) {
        const uint32_t o = __ldg(a.offsets + b);
        n = __ldg(a.offsets + b + 1) - o;
        t = o + (k << a.log_c);
        len0 = __ldg(a.cache_lengths + b);
    }
    __device__ __forceinline__ uint64_t chunk_units(const SplitArgs& a) const {
        return (uint64_t)a.blocks * (span.tiles + a.overhead);
    }
    __device__ __forceinline__ void find_segment(const SplitArgs& a) {
        const uint32_t per = span.tiles + a.overhead;
        const uint64_t in = u - chunk_base, left = u1 - u;
        block = in < per ? 0 : (uint32_t)div_units(in, per);
        const uint32_t from = (uint32_t)(in - (uint64_t)block * per);
        units = per - from < left ? per - from : (uint32_t)left;
        first = from > a.overhead ? from - a.overhead : 0;
        last = from + units > a.overhead ? from + units - a.overhead : 0;
    }
    __device__ __forceinline__ void step(const SplitArgs& a) {
        u += units;
        if (u >= u1) return;
        if (u >= chunk_base + chunk_units(a)) {
            chunk_base += chunk_units(a);
            if (++k < chunks_of(a, n)) {
                t += 1u << a.log_c;
            } else {
                k = 0;
                do {
                    ++b;
                    load_request(a);
                } while (n == 0);  // u < u1: a later request has tokens
            }
            span = chunk_span(a, len0, n, k);
        }
        find_segment(a);
    }
    __device__ __forceinline__ void begin(const SplitArgs& a, const PieceStart& s) {
        u = s.u0;
        u1 = s.u1;
        chunk_base = s.chunk_base;
        b = s.b;
        k = s.k;
        block = units = first = last = 0;
        if (u < u1) {
            n = s.n;
            t = s.first + (k << a.log_c);
            len0 = s.len;
            span = chunk_span(a, len0, n, k);
            find_segment(a);
            while (u < u1 && first == last) step(a);
        }
    }
    __device__ __forceinline__ bool done() const { return u >= u1; }
    // The unit where the segment's (chunk, row block) ends.
    __device__ __forceinline__ uint64_t end(const SplitArgs& a) const {
        return chunk_base + (uint64_t)(block + 1) * (span.tiles + a.overhead);
    }
    __device__ __forceinline__ bool whole() const { return first == 0 && last == span.tiles; }
    // On to the next segment that has tiles (a piece may end in units that
    // have none).
    __device__ __forceinline__ void next(const SplitArgs& a) {
        do step(a);
        while (u < u1 && first == last);
    }
};

// What a piece left open: a (chunk, row block) whose first tile it has (slot 1)
// and that the next n - 1 pieces go on with (their slot 0).  n 0: nothing.
struct __align__(16) OpenPiece {
    uint32_t n, t, tokens, block;
};
static_assert(sizeof(OpenPiece) == 16, "workspace layout");

// Pieces that share the segment at w, which piece c of s begins.
__device__ __forceinline__ uint32_t sharers(const SplitArgs& a, const PieceStart& s, const Walk& w,
                                            uint32_t c) {
    return Cut(s.units, s.pieces).piece_of(w.end(a) - 1) - c + 1;
}

}  // namespace kvw
