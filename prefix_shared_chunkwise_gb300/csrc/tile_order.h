// How the persistent tile kernels deal out the output tiles of one product or of two that share a launch.
// Plain C++ on both sides, so that the host can go through the same order.
#pragma once
#include <algorithm>
#include <cstdint>

#ifdef __CUDACC__
#define HARTS_BOTH_SIDES __host__ __device__ __forceinline__
#else
#define HARTS_BOTH_SIDES inline
#endif

namespace harts {

constexpr uint32_t kGroup = 16;         // tiles along the fast side that run together

struct TileId { int which, mt, nt, split; };

// A P has prod[2], n_prod and each0, over, extra; a product m_tiles, n_tiles, splits, k_per, fast_n and items, per_split.

// The n-th tile of worker `w` of `workers` (blocks or pairs).  Tiles of the first product go
// round the workers; those of the second follow, the workers that got one tile less of the
// first taking `extra` of them before the others join in.  32-bit arithmetic: the threads that
// feed the tensor cores come through here between two tiles.
template <typename P> HARTS_BOTH_SIDES bool tile_at(const P &p, uint32_t n, uint32_t w, uint32_t workers, TileId &t) {
    uint32_t idx = w + n * workers;
    t.which = 0;
    if (idx >= p.prod[0].items) {
        if (p.n_prod < 2) return false;
        t.which = 1;
        const uint32_t few = workers - p.over;                       // workers with a tile less, if any
        uint32_t m = n - p.each0 - (w < p.over ? 1 : 0);
        if (p.over == 0) {
            idx = w + m * workers;
        } else if (w >= p.over && m < p.extra) {
            idx = (w - p.over) + m * few;
        } else {
            if (w >= p.over) m -= p.extra;
            idx = few * p.extra + w + m * workers;
        }
        if (idx >= p.prod[1].items) return false;
    }
    const auto &q = p.prod[t.which];
    t.split = 0;
    if (q.splits > 1) {
        t.split = static_cast<int>(idx / q.per_split);
        idx -= t.split * q.per_split;
    }
    // groups of kGroup tiles along the fast side run against every tile of the other
    const uint32_t fast = q.fast_n ? q.n_tiles : q.m_tiles, slow = q.fast_n ? q.m_tiles : q.n_tiles;
    uint32_t base = 0, len = fast;
    if (fast > kGroup) {
        const uint32_t g = idx / (kGroup * slow);
        idx -= g * kGroup * slow;
        base = g * kGroup;
        len = fast - base < kGroup ? fast - base : kGroup;
    }
    const uint32_t s = idx / len, f = base + idx - s * len;
    t.mt = q.fast_n ? s : f;
    t.nt = q.fast_n ? f : s;
    return true;
}

// Fills in what tile_at goes by, for at most `most` workers; returns their number.
template <typename P> inline uint32_t share_tiles(P &p, int64_t most) {
    int64_t items = 0;
    for (int i = 0; i < p.n_prod; ++i) {
        auto &q = p.prod[i];
        q.per_split = static_cast<uint32_t>(q.m_tiles) * q.n_tiles;
        q.items = q.per_split * q.splits;
        items += q.items;
    }
    const uint32_t workers = static_cast<uint32_t>(std::min<int64_t>(items, most));
    p.each0 = p.prod[0].items / workers;
    p.over = p.prod[0].items % workers;
    p.extra = 0;
    if (p.n_prod == 2 && p.over) {
        // a tile costs its K steps and about three more for its ends
        const uint32_t a = p.prod[0].k_per + 3, b = p.prod[1].k_per + 3;
        p.extra = std::min((a + b / 2) / b, p.prod[1].items / (workers - p.over));
    }
    return workers;
}

}  // namespace harts
