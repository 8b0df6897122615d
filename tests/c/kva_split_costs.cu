// Host check of the division of the attention calls' work with segments that
// cost up to 8 tiles to begin and end: the units of a request are its chunks'
// tiles and costs, and every unit of the axis lies in one chunk.
#include <cstdio>

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
    for (int it = 0; it < 40000; ++it) {
        SplitArgs a = {};
        a.log_c = (uint32_t)rnd(7);
        a.cap = 1 + (int64_t)rnd(it % 3 == 0 ? 90 : it % 3 == 1 ? 1000 : 1ull << 32);
        a.overhead = (uint32_t)rnd(9);
        a.window = rnd(3) ? 1 + (int64_t)rnd(it % 2 ? 70 : 2000) : 1ll << 40;
        const int64_t len = (int64_t)rnd(it % 5 == 0 ? 1ull << 32 : it % 2 ? 100 : 3000);
        const uint32_t n = (uint32_t)rnd(200);
        int64_t sum = 0;
        for (uint32_t k = 0; k < chunks_of(a, n); ++k) {
            if (units_before(a, len, k) != sum) return printf("units_before: it %d\n", it), 1;
            // the binary search for the chunk of a unit ends at this one
            const int64_t mine = chunk_span(a, len, n, k).tiles + (int64_t)a.overhead;
            const int64_t u = sum + (int64_t)rnd((uint64_t)mine);
            uint32_t k0 = 0, k1 = chunks_of(a, n);
            while (k1 - k0 > 1u) {
                const uint32_t mid = k0 + (k1 - k0) / 2;
                (units_before(a, len, mid) <= u ? k0 : k1) = mid;
            }
            if (k0 != k) return printf("chunk of a unit: it %d\n", it), 1;
            sum += mine;
            ++checks;
        }
        if (request_units(a, len, n) != sum) return printf("request_units: it %d\n", it), 1;
    }
    printf("%ld checks, 0 mismatches\n", checks);
    return 0;
}
