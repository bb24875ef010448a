// The scan's tables of random forests, against the definition of its tiles, groups and orders: every group size that
// the kernels use reads the same tables, and what a tile waits for has to come before it in either order (a
// block that waited for a tile dealt out later would wait for ever).  Exits with 1 and a line at the first difference.
#include <algorithm>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <map>
#include <random>
#include <vector>

#include "harts.h"
#include "plan_internal.h"

using namespace harts;

#define REQUIRE(x)                                              \
    do {                                                        \
        if (!(x)) { std::printf("line %d: %s\n", __LINE__, #x); std::exit(1); } \
    } while (0)

static void check(const std::vector<int32_t> &parent, const std::vector<int64_t> &len, uint32_t flags) {
    const int n = static_cast<int>(parent.size());
    harts_plan *P = nullptr;
    REQUIRE(harts_plan_calls(n, parent.data(), len.data(), 64, flags, &P) == HARTS_OK);
    const PlanImage &I = P->image;
    const int N = I.n_scan;
    const ScanTile *fwd = reinterpret_cast<const ScanTile *>(&I.words[I.off_scan_fwd]);
    const ScanTile *bwd = reinterpret_cast<const ScanTile *>(&I.words[I.off_scan_bwd]);
    const int32_t *next = &I.words[I.off_scan_next];
    // two records a tile and a word for each segment that follows another: a plan that no scan uses pays for no more
    int children = 0;
    for (int p : parent) children += p >= 0;
    REQUIRE(static_cast<int64_t>(I.words.size()) - I.off_scan_next <= 24 * int64_t(N) + children + 80);

    std::vector<int> first(n + 1, 0), root(n, 0), seg, place;
    int roots = 0;
    for (int v = 0; v < n; ++v) {
        if (parent[v] < 0) root[v] = roots++;
        const int tiles = static_cast<int>((len[v] + kScanRows - 1) / kScanRows);
        for (int t = 0; t < tiles; ++t) { seg.push_back(v); place.push_back(t); }
        first[v + 1] = first[v] + tiles;
    }
    REQUIRE(N == first[n]);
    std::vector<int> at_fwd(N, -1), at_bwd(N, -1);      // ticket of a tile
    for (int i = 0; i < N; ++i) {
        REQUIRE(fwd[i].tile >= 0 && fwd[i].tile < N && at_fwd[fwd[i].tile] < 0);
        REQUIRE(bwd[i].tile >= 0 && bwd[i].tile < N && at_bwd[bwd[i].tile] < 0);
        at_fwd[fwd[i].tile] = i;
        at_bwd[bwd[i].tile] = i;
    }
    int64_t longest = 0;
    std::vector<int64_t> end(n);
    for (int v = 0; v < n; ++v) longest = std::max(longest, end[v] = len[v] + (parent[v] < 0 ? 0 : end[parent[v]]));
    REQUIRE(longest == I.scan_longest);

    for (const int group : kScanGroups) {
        std::vector<int> groups(n + 1, 0);
        for (int v = 0; v < n; ++v) groups[v + 1] = groups[v] + (first[v + 1] - first[v] + group - 1) / group;
        auto group_of = [&](int t) { return groups[seg[t]] + place[t] / group; };
        std::vector<ScanPlace> of(N);
        std::map<int, int> slots;                       // a group's slot is its own
        for (int i = 0; i < N; ++i) of[fwd[i].tile] = scan_place(fwd[i], group);
        for (int t = 0; t < N; ++t) {
            const ScanPlace back = scan_place(bwd[at_bwd[t]], group);
            REQUIRE(!std::memcmp(&back, &of[t], sizeof(back)));
            REQUIRE(of[t].slot >= 0 && of[t].slot < I.n_scan_slots);
            REQUIRE(slots.emplace(of[t].slot, group_of(t)).first->second == group_of(t));
        }
        REQUIRE(static_cast<int>(slots.size()) == groups[n]);
        for (int t = 0; t < N; ++t) {
            const ScanPlace &q = of[t];
            const int v = seg[t], u = parent[v], count = first[v + 1] - first[v], start = t - q.at;
            const bool last = group_of(t) == groups[v + 1] - 1;
            REQUIRE(q.tile == t && q.row0 == P->seg_offset[v] + int64_t(kScanRows) * place[t]);
            REQUIRE(q.rows == std::min<int64_t>(kScanRows, len[v] - int64_t(kScanRows) * place[t]));
            REQUIRE(q.at == place[t] % group && q.count == std::min(group, count - place[start]));
            REQUIRE(q.pred_row == (place[t] > 0 ? q.row0 - 1 : u < 0 ? -1 - root[v] : P->seg_offset[u] + len[u] - 1));
            REQUIRE(q.seq_end == (last && P->seg_ctop[v] < 0 ? P->seg_seq[v] : -1));
            for (int k = start; k < t; ++k) REQUIRE(at_fwd[k] < at_fwd[t] && at_bwd[k] > at_bwd[t]);
            if (place[t] < group && u < 0) {
                REQUIRE(q.pred == -1 - root[v]);
            } else {
                const int before = place[t] < group ? first[u + 1] - 1 : start - 1;
                REQUIRE(slots.at(q.pred) == group_of(before));
                REQUIRE(at_fwd[before] < at_fwd[t] && at_bwd[before] > at_bwd[t]);
            }
            if (!last) {
                REQUIRE(q.next_count == 1 && q.next_begin < 0 && slots.at(-1 - q.next_begin) == group_of(t) + 1);
                continue;
            }
            int k = 0;
            for (int w = v + 1; w < n; ++w)             // by ascending segment
                if (parent[w] == v) REQUIRE(slots.at(next[q.next_begin + k++]) == groups[w]);
            REQUIRE(k == q.next_count);
        }
    }
    harts_plan_free(P);
}

int main() {
    std::mt19937 r(1);
    for (int i = 0; i < 300; ++i) {
        const int n = 1 + r() % 60;
        std::vector<int32_t> parent(n);
        std::vector<int64_t> len(n);
        for (int v = 0; v < n; ++v) {
            parent[v] = v == 0 || r() % 5 == 0 ? -1 : r() % 2 ? v - 1 : static_cast<int>(r() % v);
            const int kind = r() % 4;
            len[v] = kind == 0 ? 1 + r() % 20 : kind == 1 ? 1 + r() % 300 : kind == 2 ? 1 + r() % 5000 : kScanRows * (1 + r() % 70);
        }
        check(parent, len, i % 3 == 1 ? HARTS_PLAN_NODEWISE : i % 3 == 2 ? HARTS_PLAN_NOREPLAY : 0);
    }
    check({-1}, {1}, 0);
    check({-1, 0, 0, 0}, {128 * 64, 1, 128 * 33 + 1, 128}, 0);
    return 0;
}
