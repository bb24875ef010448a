// Every tile of one or two products that share a launch, and every piece of its sum, comes up exactly once, and a
// worker's tiles end where tile_at first says so.  Exits with 1 and a line at the first difference.
#include <cstdio>
#include <cstdlib>
#include <random>
#include <vector>

#include "tile_order.h"

using namespace harts;

#define REQUIRE(x)                                              \
    do {                                                        \
        if (!(x)) { std::printf("line %d: %s\n", __LINE__, #x); std::exit(1); } \
    } while (0)

struct Product {
    int32_t m_tiles, n_tiles, splits, k_per, fast_n;
    uint32_t items, per_split;
};
struct Launch {
    Product prod[2];
    int32_t n_prod;
    uint32_t each0, over, extra;
};

static void check(Launch p, int64_t most) {
    for (Product &q : p.prod) q.fast_n = q.n_tiles <= q.m_tiles;
    const uint32_t workers = share_tiles(p, most);
    std::vector<int> seen[2];
    for (int i = 0; i < p.n_prod; ++i) seen[i].assign(p.prod[i].items, 0);
    for (uint32_t w = 0; w < workers; ++w) {
        TileId t;
        int which = 0;
        uint32_t n = 0;
        for (; tile_at(p, n, w, workers, t); ++n) {
            const Product &q = p.prod[t.which];
            REQUIRE(t.which >= which && t.which < p.n_prod);          // the first product's tiles come first
            which = t.which;
            REQUIRE(t.mt >= 0 && t.mt < q.m_tiles && t.nt >= 0 && t.nt < q.n_tiles && t.split >= 0 && t.split < q.splits);
            ++seen[which][(static_cast<size_t>(t.split) * q.m_tiles + t.mt) * q.n_tiles + t.nt];
        }
        for (uint32_t k = 1; k < 4; ++k) REQUIRE(!tile_at(p, n + k, w, workers, t));
    }
    for (int i = 0; i < p.n_prod; ++i)
        for (int k : seen[i]) REQUIRE(k == 1);
}

int main() {
    std::mt19937 r(1);
    auto any = [&](int most) { return 1 + static_cast<int>(r() % most); };
    for (int i = 0; i < 4000; ++i) {
        Launch p{};
        p.n_prod = any(2);
        for (Product &q : p.prod) {
            const int size = i % 3 == 0 ? 6 : i % 3 == 1 ? 20 : 70;
            q.m_tiles = any(size);
            q.n_tiles = any(size);
            q.splits = r() % 3 ? 1 : any(32);
            q.k_per = any(300);
        }
        for (int64_t most : {152, 76, any(200)}) check(p, most);
    }
    return 0;
}
