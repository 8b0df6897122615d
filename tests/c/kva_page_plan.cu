// Host check of the plan of a tile that lies in one page: which of its 64
// positions are there, also where what is seen begins behind the tile (a window
// that starts past the end of the page table).
#include <cstdio>
#include <vector>

#include "kva_tma.cuh"

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
    for (int it = 0; it < 100000; ++it) {
        const uint32_t page_size = 64 * (1 + (uint32_t)rnd(4)), width = 1 + (uint32_t)rnd(40);
        const uint32_t num_pages = 1 + (uint32_t)rnd(100);
        std::vector<uint32_t> table(2 * width);
        for (auto& id : table) id = rnd(10) ? (uint32_t)rnd(num_pages) : KVW_PAGE_UNMAPPED;
        const uint32_t b = (uint32_t)rnd(2);
        const FastDiv ps = make_fast_div(page_size);
        const uint32_t p_tile = 64 * (uint32_t)rnd((uint64_t)width * page_size / 64 + 1);
        const int64_t hi = (int64_t)p_tile + 1 + (int64_t)rnd(rnd(2) ? 64 : 1000);
        // before the tile, in it, just behind it, and 2^32 and more behind it
        const uint64_t kind = rnd(4);
        const int64_t start = kind == 0   ? (int64_t)rnd((uint64_t)p_tile + 1)
                              : kind == 1 ? (int64_t)p_tile + (int64_t)rnd(64)
                              : kind == 2 ? (int64_t)p_tile + 64 + (int64_t)rnd(200)
                                          : (int64_t)p_tile + (1ll << 32) + (int64_t)rnd(1 << 20);
        const PagePlan t = plan_page(table.data(), width, num_pages, ps, b, p_tile, start, hi);
        const uint32_t idx = p_tile / page_size;
        const bool valid = idx < width && table[b * width + idx] < num_pages;
        bool same = t.valid == valid && t.row == p_tile % page_size &&
                    (!valid || t.page == table[b * width + idx]);
        for (uint32_t r = 0; r < 64; ++r) {
            const int64_t p = (int64_t)p_tile + r;
            same &= ((t.there >> r) & 1) == (uint64_t)(valid && p >= start && p < hi);
        }
        if (!same) {
            printf("it %d tile %u start %lld hi %lld: there %llx\n", it, p_tile, (long long)start,
                   (long long)hi, (unsigned long long)t.there);
            return 1;
        }
        ++checks;
    }
    printf("%ld checks, 0 mismatches\n", checks);
    return 0;
}
