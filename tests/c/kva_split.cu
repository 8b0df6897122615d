// Host check of the closed forms that divide the attention calls' work:
// against sums taken chunk by chunk, and the pieces against an even cut.
#include <cstdio>
#include <cstdlib>

#include "kva_split.cuh"

using namespace kvw;

static uint64_t g_state = 88172645463325252ull;
static uint64_t rnd(uint64_t n) {
    g_state ^= g_state << 13;
    g_state ^= g_state >> 7;
    g_state ^= g_state << 17;
    return g_state % n;
}

int main() {
    long checks = 0;
    for (int it = 0; it < 60000; ++it) {
        SplitArgs a = {};
        a.log_c = (uint32_t)rnd(7);
        a.cap = 1 + (int64_t)rnd(it % 3 == 0 ? 90 : it % 3 == 1 ? 1000 : 1ull << 32);
        a.overhead = (uint32_t)rnd(4);
        a.window = rnd(3) ? 1 + (int64_t)rnd(it % 2 ? 70 : 2000) : 1ll << 40;
        const int64_t len = (int64_t)rnd(it % 5 == 0 ? 1ull << 32 : it % 2 ? 100 : 3000);
        const uint32_t n = (uint32_t)rnd(200);
        int64_t sum = 0;
        for (uint32_t k = 0; k < chunks_of(a, n); ++k) {
            if (tiles_before(a, len, k) != sum) {
                printf("tiles_before: it %d k %u: %lld, want %lld\n", it, k,
                       (long long)tiles_before(a, len, k), (long long)sum);
                return 1;
            }
            const ChunkSpan s = chunk_span(a, len, n, k);
            // the definition, token by token
            int64_t lo = 1ll << 62, hi = 0;
            for (uint32_t i = k << a.log_c; i < ((k + 1) << a.log_c) && i < n; ++i) {
                const int64_t pos = len + i;
                int64_t from = pos + 1 - a.window;
                if (from < 0) from = 0;
                if (from < lo) lo = from;
                if (pos + 1 > hi) hi = pos + 1;
            }
            if (hi > a.cap) hi = a.cap;
            const int64_t at = lo < hi ? lo : hi - 1;
            if (s.start != lo || s.hi != hi || s.tile0 != at / 64 || s.tiles < 1 ||
                (int64_t)s.tile0 + s.tiles != (hi + 63) / 64) {
                printf("chunk_span: it %d k %u\n", it, k);
                return 1;
            }
            sum += s.tiles;
            ++checks;
        }
        if (request_units(a, len, n) != sum + (int64_t)chunks_of(a, n) * a.overhead) {
            printf("request_units: it %d\n", it);
            return 1;
        }
    }
    for (int it = 0; it < 20000; ++it) {
        const uint64_t units = 1 + rnd(it % 2 ? 3000 : 1ull << 58);
        SplitArgs a = {};
        a.min_units = 1 + (uint32_t)rnd(8);
        const uint32_t most = 1 + (uint32_t)rnd(512), p = pieces_of(a, units, most);
        const Cut cut(units, p);
        if (p < 1 || p > most || p > units || cut.start(0) != 0 ||
            cut.start(p) != units)
            return printf("pieces\n"), 1;
        for (uint32_t c = 0; c < p; ++c) {
            const uint64_t size = cut.start(c + 1) - cut.start(c);
            if (size < 1 || size < units / p || size > units / p + 1) return printf("cut\n"), 1;
            if (p > 1 && size < a.min_units) return printf("short piece\n"), 1;
            const uint64_t u = cut.start(c);
            if (cut.piece_of(u) != c || cut.piece_of(u + size - 1) != c)
                return printf("piece_of\n"), 1;
        }
        ++checks;
    }
    printf("%ld checks, 0 mismatches\n", checks);
    return 0;
}
