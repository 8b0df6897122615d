// Host check of the copies that fill a tile of 64 positions: every position of
// the tile that has a valid page is copied once, no copy leaves its page or
// the tile, and the rows copied are the rows announced.
#include <cstdio>
#include <cstdlib>
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

#define NEED(x)                                                                        \
    if (!(x)) {                                                                        \
        printf("it %d page_size %u start %lld hi %lld tile %lld: %s\n", it, page_size, \
               (long long)start, (long long)hi, (long long)p_tile, #x);                \
        return 1;                                                                      \
    }

int main() {
    static const uint32_t sizes[] = {1, 2, 3, 4, 8, 12, 16, 20, 24, 32, 48, 64, 96, 100, 128, 192, 256};
    long checks = 0;
    for (int it = 0; it < 60000; ++it) {
        const uint32_t page_size = rnd(4) ? sizes[rnd(17)] : 1 + (uint32_t)rnd(300);
        CacheMaps m = {};
        const uint32_t rows = rows_per_copy(page_size);
        while ((1u << m.log_rows) < rows) ++m.log_rows;
        for (uint32_t r = rows; r <= 64 && r <= page_size; r *= 4) ++m.levels;
        const uint32_t width = 1 + (uint32_t)rnd(400), num_pages = 1 + (uint32_t)rnd(1000);
        std::vector<uint32_t> table(2 * width);
        for (auto& id : table) id = rnd(20) ? (uint32_t)rnd(num_pages) : (uint32_t)(num_pages + rnd(3));
        if (rnd(9) == 0) table[rnd(2 * width)] = KVW_PAGE_UNMAPPED;
        const uint32_t b = (uint32_t)rnd(2);
        // mostly within the table, now and then past its end
        const int64_t reach = (int64_t)width * page_size;
        const int64_t hi = 1 + (int64_t)rnd(rnd(8) ? reach : reach + 100);
        const int64_t start = rnd(2) ? 0 : (int64_t)rnd(hi);
        const int64_t p_tile = 64 * (start / 64 + (int64_t)rnd((hi - 1) / 64 - start / 64 + 1));
        const FastDiv ps = make_fast_div(page_size);

        uint32_t announced = 0, copied = 0, by[64] = {};
        uint64_t there = 0;
        bool bad = false;
        for (uint32_t c = 0; c < 64; ++c) {
            const UnitCopy u =
                plan_unit(m, table.data(), width, num_pages, ps, b, p_tile, start, hi, c);
            if (start <= p_tile && p_tile + 64 <= hi && rows > 1) {  // the short way agrees
                const UnitCopy x = plan_inner_unit(m, table.data(), width, num_pages, ps, b,
                                                   (uint32_t)p_tile, c);
                NEED(x.level == u.level && x.bad_page == u.bad_page);
                NEED(x.level == 4 || (x.page == u.page && x.row == u.row));
            }
            if (u.there) announced += rows;
            NEED(!(there & u.there));
            there |= u.there;
            bad |= u.bad_page;
            if (u.level == 4) continue;
            NEED(u.level < m.levels && !u.bad_page && u.page < num_pages);
            const uint32_t n = rows << (2 * u.level), first = c << m.log_rows;
            NEED(u.row + n <= page_size && first + n <= 64);
            copied += n;
            for (uint32_t r = 0; r < n; ++r) {
                const uint64_t p = (uint64_t)p_tile + first + r;
                NEED(by[first + r]++ == 0 && p / page_size < width);
                NEED(table[b * width + p / page_size] == u.page && p % page_size == u.row + r);
            }
        }
        NEED(announced == copied);
        bool lost = false;
        for (uint32_t r = 0; r < 64; ++r) {
            const int64_t p = p_tile + r;
            const bool used = p >= start && p < hi, page = used && p / page_size < width &&
                              table[b * width + p / page_size] < num_pages;
            lost |= used && !page;
            NEED(((there >> r) & 1) == page);
            NEED(!page || by[r] == 1);
        }
        NEED(bad == lost);
        ++checks;
    }
    printf("%ld checks, 0 mismatches\n", checks);
    return 0;
}
