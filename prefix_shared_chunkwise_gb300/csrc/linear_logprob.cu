// Log-probabilities straight from the hidden rows and the vocabulary weight, forward and
// backward, without keeping the C x V logits.
//
//   z[c][v] = scale x_c . w_v,  lse_c = log sum_v e^z[c][v],  logp[s] = z[c(s)][y_s] - lse_c(s)
//   dz[c][v] = sum_{s -> c, y_s = v} g_s - G_c e^(z[c][v] - lse_c),  G_c = sum_{s -> c} g_s
//   dx_c = scale sum_v dz[c][v] w_v,    dw_v = scale sum_c dz[c][v] x_c
// (the compact-to-semantic form of HARTS, page "HARTS ... 精读", section 4.4 and eq. 19, with
// the vocabulary projection taken into the operator).  Positions whose label lies outside the
// vocabulary carry no log-probability and no gradient.
//
// Forward: one product X W^T whose 128 x N tiles never leave the SM.  A tile's accumulators
// are reduced in place to one (max, sum of exponentials) per row and the maximum's column, 9
// bytes instead of N logits; a small kernel joins a row's pairs, and the positions' own logits,
// like each row's largest, are formed by dot products (S + C of them, against C V in the product).
// Backward, over pieces of the vocabulary: the product again, its epilogue turning logits
// into scale * dz in bf16; then dX += dZ W and dW = dZ^T X in one launch, with the same tiles.
// dz is rounded to bf16 because the tensor cores take bf16 operands next to bf16 W and X;
// every entry, labels' included, is formed in fp32 and rounded once (up to 32 rows it is kept
// in two bf16 terms).  Sums are fp32.  dX of several pieces or of a split vocabulary is summed
// in fp32 (one buffer per split, added to in piece order), so results do not depend on timing.
//
// Tile kernel: persistent blocks, one per SM, in pairs where there are rows for it; warps 0 and
// 3 fill a ring of shared-memory stages with A and B by TMA, warp 1 issues tcgen05.mma into one
// of two 256-column accumulators in TMEM, warps 4-11 empty the other one, two warps for each 32
// rows taking columns in turn (through shared memory and TMA stores of warps 12-13, where there
// is output).  All waits are bounded.
//
// Many rows are bound by the tensor cores, under the power limit: 4,096 x 157,184 x 2,048 takes
// 1.50 ms forward (1.76 PFLOP/s) and 4.65 ms backward (1.70), at 92 - 95 % of the tensor pipe's
// cycles.  Few rows are bound by reading W: 1 row takes 107 us (6.0 TB/s).
#include <algorithm>
#include <cmath>
#include <cstring>

#include "kda_common.cuh"
#include "launch_util.h"
#include "tc_primitives.cuh"
#include "tensor_map.h"
#include "tile_order.h"
#include "tile_pairs.cuh"

namespace harts {
namespace {

using namespace pairs;

constexpr int kTM = 128, kTK = 64, kTN = 256;       // a block's tile rows, K step (one 128-byte swizzle row), tile columns
constexpr int kTwin = 32;                            // most rows whose dZ is kept in two bf16 terms
constexpr uint32_t kABytes = kTM * kTK * 2;
constexpr uint32_t kSlotBytes = kTM * 128;           // 128 rows x 128 bytes of the output on their way out

constexpr int kThreads = 448, kEpiWarp0 = 4, kStoreWarp0 = 12;    // eight epilogue warps: two for each 32 TMEM lanes
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

enum Mode { kFwd = 0, kDz = 1, kGrad = 2 };

// Shared memory: stages of both operands and slots of the output.  A block of a pair holds
// half of the tile's columns: its stages are smaller, and there are more of them.  The forward
// has no output; dW of few rows is nothing but output, which needs bytes on their way.
template <int MODE, int G> struct Ring {
    static constexpr uint32_t slots = MODE == kFwd ? 0 : MODE == kDz ? 2 : 4;
    static constexpr uint32_t stages = G == 2 ? (MODE == kFwd ? 7 : MODE == kDz ? 6 : 5) : (MODE == kGrad ? 3 : 4);
    static constexpr uint32_t stage_bytes = kABytes + kTN / G * kTK * 2;
    static constexpr uint32_t smem = stages * stage_bytes + slots * kSlotBytes + 1024;
    static_assert(smem + kTM * 9 <= 227 * 1024 - 384, "shared memory of an SM");
    // barriers
    static constexpr uint32_t full = 0, empty = stages, acc_full = 2 * stages, acc_empty = acc_full + 2, drain = acc_empty + 2,
                              out_full = drain + 1, out_free = out_full + slots, pair_full = out_free + slots,
                              pair_free = pair_full + 4, count = pair_free + 4;
};

// One product D = op(A) op(B)^T cut into tiles and splits of its K range.
struct Prod {
    CUtensorMap a, b, out;
    CUtensorMap b_edge;             // B's last columns, where they do not fill a panel
    int32_t a_mn, b_mn;             // operand stored [K][rows] instead of [rows][K]
    int32_t a_panel;                // A is dZ, kept in panels of 64 columns
    int32_t b_whole;                // B stored [K][columns]: columns in whole panels of 64, one copy for a tile of them
    int32_t a_rows;                 // rows of A's box when stored [rows][K]
    int32_t m_tiles, n_tiles, splits, n;
    uint32_t items, per_split;      // tiles times splits, tiles
    int32_t k_blocks, k_per;        // steps of 64 in all, per split
    int32_t b_y0, out_y0;           // row offsets of this piece of the vocabulary in B and the output
    int32_t rows, cols;             // extent of the output (rows from out_y0 on)
    int32_t fast_n;                 // tiles that run together share A (walk n first) instead of B
    int32_t out_f32, out_add;
};

struct alignas(16) RowInfo { float neg_g, lse2; int32_t count, first; };   // -scale G, lse log2 e, labelled entries

struct Params {
    Prod prod[2];
    int32_t n_prod;
    uint32_t each0, over, extra;    // see tile_at: tiles of the first product per worker, and what is left
    int32_t *error;
    float c2;                       // scale * log2 e (logit_factor)
    float2 *part;                   // forward: [C][n_tiles] accumulator of the largest logit; the sum
    uint8_t *top;                   // forward: [C][n_tiles] column of the tile's maximum
    const RowInfo *rows;            // dz: per compact row
    const int32_t *ent_y;
    const float *ent_v;
    int32_t v0;                     // dz: first vocabulary entry of the piece
    int32_t twin;                   // dz: rows 32 .. 63 hold what rounding takes from rows 0 .. 31
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float y;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
    return y;
}
__device__ __forceinline__ float min3(float a, float b, float c) {
    float y;
    asm("min.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
    return y;
}

template <int MODE, int G>
__global__ void __launch_bounds__(kThreads, 1) head_tile_kernel(const __grid_constant__ Params p) {
    using B = Ring<MODE, G>;
    constexpr uint32_t kStages = B::stages, kStageBytes = B::stage_bytes, kSlots = B::slots;
    extern __shared__ uint8_t smraw[];
    uint8_t *sm = smraw + ((1024 - (tc::smem_addr(smraw) & 1023)) & 1023);
    __shared__ uint64_t bars[B::count];
    __shared__ uint32_t s_tmem;
    __shared__ int s_fail;
    __shared__ float2 s_pair[MODE == kFwd ? kTM : 1];
    __shared__ uint8_t s_top[MODE == kFwd ? kTM : 1];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = G == 2 ? static_cast<int>(cluster_rank()) : 0;
    const uint32_t worker = blockIdx.x / G, workers = gridDim.x / G;

    if (tid == 0) {
        for (uint32_t i = 0; i < kStages; ++i) { tc::mbar_init(&bars[B::full + i], 2); tc::mbar_init(&bars[B::empty + i], 1); }
        for (int i = 0; i < 2; ++i) { tc::mbar_init(&bars[B::acc_full + i], 1); tc::mbar_init(&bars[B::acc_empty + i], 8 * G); }
        for (int i = 0; i < static_cast<int>(kSlots); ++i) { tc::mbar_init(&bars[B::out_full + i], 4); tc::mbar_init(&bars[B::out_free + i], 1); }
        for (int i = 0; i < 4; ++i) { tc::mbar_init(&bars[B::pair_full + i], 1); tc::mbar_init(&bars[B::pair_free + i], 1); }
        tc::mbar_init(&bars[B::drain], 1);
        tc::fence_mbar_init();
        s_fail = 0;
    }
    if (warp == 3 && lane < 2 * p.n_prod) {             // the first copies find their descriptors fetched
        const Prod &q = p.prod[lane >> 1];
        prefetch_map(lane & 1 ? &q.b : &q.a);
    }
    if (warp == 2) { pair_alloc<G>(&s_tmem); tc::fence_before_sync(); }
    __syncthreads();
    if (G == 2) cluster_sync();                         // the other block's barriers exist
    tc::fence_after_sync();
    let_next_start();
    const uint32_t tm = s_tmem;
    // Bounded waits begin once the kernel before this one is done: its time is not theirs, and it
    // may be any.  dZ's first two tiles, one for each accumulator, are copied and multiplied beside
    // it where both operands are the call's own; nothing else waits for a barrier until then.
    const bool ahead = MODE == kDz && !p.prod[0].a_panel;

    if (warp == 0 || warp == 3) {
        // One warp each for A and B, whole like the issuing one: a copy by a lone thread, or both
        // operands' by one warp, could not keep up with the 512 cycles of a step's products.
        const bool is_b = warp == 3;
        const uint32_t on = elect_lane(), arms = rank == 0 ? on : 0;
        // dZ is complete; the aligned copy of X, where there is one (B fills its stages once before)
        if (MODE == kGrad || (!is_b && !ahead)) wait_previous();
        uint32_t it = 0;                                // stages filled so far
        uint32_t s = 0, round = 0;                      // next stage, times the ring went round
        const uint32_t own0 = tc::smem_addr(&bars[B::full]), full0 = G == 2 ? leader_addr(&bars[B::full]) : own0;
        const uint32_t dst0 = tc::smem_addr(sm) + (is_b ? kABytes : 0);
        TileId t;
        bool ok = true;
        for (uint32_t n = 0; ok && tile_at(p, n, worker, workers, t); ++n) {
            if (ahead && n == 2) wait_previous();
            // what the loop needs is taken out of the parameters once a tile
            const Prod &q = p.prod[t.which];
            const int32_t k0 = t.split * q.k_per, k1 = min(q.k_blocks, k0 + q.k_per);
            const int32_t nb = q.n / G;                 // columns that this block holds
            const int32_t m0 = (t.mt * G + rank) * kTM, n0 = t.nt * q.n + rank * nb, y0 = q.b_y0;
            enum { kRows, kPanelRows, kPanelCols, kBoxes };
            const int how = is_b ? (q.b_mn ? (n0 + nb <= q.b_whole ? kPanelCols : kBoxes) : kRows)
                                 : (q.a_panel ? (q.a_mn ? kPanelCols : kPanelRows) : kRows);
            const CUtensorMap *map = is_b ? (how == kBoxes ? &q.b_edge : &q.b) : &q.a;
            const int32_t row = is_b ? y0 + n0 : m0, panel = (is_b ? n0 : m0) / 64, ky = is_b ? y0 : 0;
            const uint32_t bytes = (is_b ? nb * 128u : q.a_mn ? kABytes : q.a_rows * 128u) * G;
            for (int32_t k = k0; k < k1; ++k, ++it) {
                if (it == kStages && !ahead) wait_previous();
                if (round > 0 && !warp_wait(&bars[B::empty + s], (round - 1) & 1, &s_fail)) { ok = false; break; }
                const uint32_t full = full0 + s * 8, dst = dst0 + s * kStageBytes;
                expect(arms, own0 + s * 8, bytes);
                const int32_t yk = ky + k * kTK;
                if (how == kRows) pair_load<G>(on, dst, map, k * kTK, row, full);
                else if (how == kPanelCols) pair_load3<G>(on, dst, map, 0, yk, panel, full);
                else if (how == kPanelRows) pair_load3<G>(on, dst, map, 0, row, k, full);
                else for (int j = 0; j < nb; j += 64) pair_load<G>(on, dst + j * 128, map, n0 + j, yk, full);
                if (++s == kStages) { s = 0; ++round; }
            }
        }
        // Nothing may be in flight into this block's shared memory when it ends: the copies (after
        // a failure the products may not have waited for them), then the stages' last release.
        // In a pair only the release says so for the second block; after a failure its wait runs
        // out, long after the last copy.
        wait_previous();
        for (uint32_t i = 0; i < kStages; ++i) {
            if (it <= i) continue;
            const uint32_t uses = (it - i + kStages - 1) / kStages;
            if (rank == 0) tc::mbar_wait(&bars[B::full + i], (uses - 1) & 1, failed(&s_fail) ? 100000000LL : 4000000000LL);
            if (!tc::mbar_wait(&bars[B::empty + i], (uses - 1) & 1, failed(&s_fail) ? 100000000LL : 4000000000LL))
                atomicExch(&s_fail, 1);
        }
    } else if (warp == 1) {
        if (rank == 0) {
            const uint32_t on = elect_lane();
            uint32_t s = 0, round = 0, tile = 0;
            const uint32_t base = tc::smem_addr(sm);
            TileId t;
            bool ok = true;
            if (!ahead) wait_previous();
            for (; ok && tile_at(p, tile, worker, workers, t); ++tile) {
                if (ahead && tile == 2) wait_previous();
                const Prod &q = p.prod[t.which];
                const int32_t k0 = t.split * q.k_per, k1 = min(q.k_blocks, k0 + q.k_per);
                const uint32_t buf = tile & 1, use = tile >> 1, d = tm + buf * kTN;
                const uint32_t id = tc::idesc_bf16(kTM * G, q.n, q.a_mn != 0, q.b_mn != 0);
                // descriptors of stage 0; 16 columns of K lie 32 bytes apart in an operand stored
                // by rows and 2 KB apart in one stored by K (descriptors count 16 bytes)
                const uint64_t da0 = q.a_mn ? tc::desc_sw128_mn(base, 8192) : tc::desc_sw128(base);
                const uint64_t db0 = q.b_mn ? tc::desc_sw128_mn(base + kABytes, 8192) : tc::desc_sw128(base + kABytes);
                const uint32_t ka = q.a_mn ? 128 : 2, kb = q.b_mn ? 128 : 2;
                if (use > 0 && !warp_wait(&bars[B::acc_empty + buf], (use - 1) & 1, &s_fail)) { ok = false; break; }
                tc::fence_after_sync();
                uint32_t acc = 0;
                for (int32_t k = k0; k < k1; ++k) {
                    if (!warp_wait(&bars[B::full + s], round & 1, &s_fail)) { ok = false; break; }
                    tc::fence_after_sync();
                    const uint64_t da = da0 + s * (kStageBytes / 16), db = db0 + s * (kStageBytes / 16);
#pragma unroll
                    for (uint32_t kk = 0; kk < kTK / 16; ++kk) {
                        pair_mma<G>(on, d, da + kk * ka, db + kk * kb, id, acc);
                        acc = 1;
                    }
                    pair_commit<G>(on, &bars[B::empty + s]);
                    if (++s == kStages) { s = 0; ++round; }
                }
                if (ok) pair_commit<G>(on, &bars[B::acc_full + buf]);
            }
            if (failed(&s_fail)) {                      // let the products in flight end
                pair_commit<G>(on, &bars[B::drain]);
                tc::mbar_wait(&bars[B::drain], 0, 1000000000LL);
            }
        }
    } else if (warp >= kEpiWarp0 && warp < kStoreWarp0) {
        const int lg = (warp - kEpiWarp0) & 3;          // TMEM lanes 32 lg .. 32 lg + 31
        const int half = (warp - kEpiWarp0) >> 2;       // of the two warps that share them
        const uint32_t lane_off = static_cast<uint32_t>(lg * 32) << 16;
        [[maybe_unused]] uint8_t *out = sm + kStages * kStageBytes + lg * 4096;   // this warp's rows of a slot
        const uint32_t released = G == 2 ? leader_addr(&bars[B::acc_empty]) : 0;
        uint32_t tile = 0;
        [[maybe_unused]] uint32_t groups = 0;                  // groups of 128 bytes of columns so far
        TileId t;
        bool ok = true;
        wait_previous();                                // dZ: rows' terms; the last piece's dZ has been read
        for (; ok && tile_at(p, tile, worker, workers, t); ++tile) {
            const Prod &q = p.prod[t.which];
            const uint32_t buf = tile & 1;
            if (!warp_wait(&bars[B::acc_full + buf], (tile >> 1) & 1, &s_fail)) break;
            tc::fence_after_sync();
            const uint32_t acc = tm + buf * kTN + lane_off;
            const int32_t n0 = t.nt * q.n, row = (t.mt * G + rank) * kTM + lg * 32 + lane;
            if constexpr (MODE == kFwd) {
                const int32_t nv = min(q.n, q.cols - n0);       // columns that are vocabulary entries
                // the accumulators that make the largest logit are the largest, or the smallest
                float mv = p.c2 < 0.f ? INFINITY : -INFINITY;
                for (int c = half * 32; c < nv; c += 64) {
                    float v[32];
                    tc::tmem_ld32(acc + c, v);
                    if (c + 32 > nv) {
#pragma unroll
                        for (int i = 0; i < 32; ++i) if (c + i >= nv) v[i] = mv;
                    }
                    float m1 = mv;
                    if (p.c2 < 0.f) {
#pragma unroll
                        for (int i = 0; i < 32; i += 4) { mv = min3(mv, v[i], v[i + 1]); m1 = min3(m1, v[i + 2], v[i + 3]); }
                        mv = fminf(mv, m1);
                    } else {
#pragma unroll
                        for (int i = 0; i < 32; i += 4) { mv = max3(mv, v[i], v[i + 1]); m1 = max3(m1, v[i + 2], v[i + 3]); }
                        mv = fmaxf(mv, m1);
                    }
                }
                float m = half * 32 < nv ? mv * p.c2 : -INFINITY, s = 0.f;
                int32_t top = 0;                                // column of the maximum
                for (int c = half * 32; c < nv; c += 64) {
                    float v[32], s0 = 0.f, s1 = 0.f;
                    tc::tmem_ld32(acc + c, v);
                    int32_t at = -1;
                    if (c + 32 <= nv) {
#pragma unroll
                        for (int i = 0; i < 32; i += 2) {
                            s0 += ex2(fmaf(v[i], p.c2, -m));
                            s1 += ex2(fmaf(v[i + 1], p.c2, -m));
                        }
#pragma unroll
                        for (int i = 0; i < 32; ++i) at = v[i] == mv ? i : at;
                    } else {
#pragma unroll
                        for (int i = 0; i < 32; ++i) if (c + i < nv) {
                            s0 += ex2(fmaf(v[i], p.c2, -m));
                            at = v[i] == mv ? i : at;
                        }
                    }
                    if (at >= 0) top = c + at;
                    s += s0 + s1;
                }
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) {
                    if (G == 2) arrive_at(released + buf * 8); else arrive(&bars[B::acc_empty + buf]);
                }
                // the two warps' pairs become one: the second hands its over, the first joins them
                float2 *pair = s_pair + lg * 32 + lane;
                uint64_t *give = &bars[B::pair_full + lg], *back = &bars[B::pair_free + lg];
                if (half == 1) {
                    if (tile > 0 && !warp_wait(back, (tile - 1) & 1, &s_fail)) break;
                    *pair = make_float2(mv, s);
                    s_top[lg * 32 + lane] = static_cast<uint8_t>(top);
                    __syncwarp();
                    if (lane == 0) arrive(give);
                } else {
                    if (!warp_wait(give, tile & 1, &s_fail)) break;
                    const float2 o = *pair;
                    const int32_t o_top = s_top[lg * 32 + lane];
                    __syncwarp();
                    if (lane == 0) arrive(back);
                    if (nv > 32) {
                        const float om = o.x * p.c2, n = fmaxf(m, om);
                        s = s * ex2(m - n) + o.y * ex2(om - n);
                        if (om > m) { mv = o.x; top = o_top; }
                    }
                    if (row < q.rows) {
                        const int64_t at = static_cast<int64_t>(row) * q.n_tiles + t.nt;
                        p.part[at] = make_float2(mv, s);
                        p.top[at] = static_cast<uint8_t>(top);
                    }
                }
            } else if constexpr (MODE != kFwd) {
                RowInfo ri{0.f, 0.f, 0, 0};
                if (MODE == kDz && row < q.rows) ri = p.rows[row];
                const int step = q.out_f32 ? 32 : 64, end = min(q.n, q.cols - n0);
                for (int c = 0; c < end; c += step, ++groups) {
                    if ((groups & 1) != static_cast<uint32_t>(half)) continue;
                    const uint32_t slot = groups % kSlots, use = groups / kSlots;
                    uint8_t *dst = out + slot * kSlotBytes;
                    if (use > 0 && !warp_wait(&bars[B::out_free + slot], (use - 1) & 1, &s_fail)) {
                        ok = false;
                        break;
                    }
                    if (q.out_f32) {
                        float v[32];
                        tc::tmem_ld32(acc + c, v);
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            *reinterpret_cast<float4 *>(dst + lane * 128 + ((j ^ (lane & 7)) << 4)) =
                                make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
                    } else if (MODE != kDz || !p.twin || lg == 0) {
                        float v[64];
                        tc::tmem_ld32x2(acc + c, reinterpret_cast<float(&)[32]>(v[0]), acc + c + 32,
                                        reinterpret_cast<float(&)[32]>(v[32]));
                        if (MODE == kDz) {
#pragma unroll
                            for (int i = 0; i < 64; ++i) v[i] = ri.neg_g * ex2(fmaf(v[i], p.c2, -ri.lse2));
                            if (n0 + c + 64 > q.cols || (p.twin && row >= q.rows)) {
                                // past the vocabulary dX must see zeros, past the rows dW (a twin's
                                // rows are all stored)
#pragma unroll
                                for (int i = 0; i < 64; ++i) if (n0 + c + i >= q.cols || row >= q.rows) v[i] = 0.f;
                            }
                        }
                        store_row(dst, lane, v);
                        if (MODE == kDz && p.twin) {
#pragma unroll
                            for (int i = 0; i < 64; ++i) v[i] -= __bfloat162float(__float2bfloat16_rn(v[i]));
                            store_row(dst + kTwin * 128, lane, v);
                        }
                        // The row's labels among these 64 columns.  Written by the kernel before,
                        // which this one overlaps: plain loads, the read-only path does not
                        // see what is written while a kernel runs.
                        if (MODE == kDz) {
                            const int32_t lo = p.v0 + n0 + c;
                            int32_t e = 0;
                            for (int32_t len = ri.count > 8 ? ri.count : 0; len > 0;) {     // first label >= lo
                                const int32_t half_len = len >> 1;
                                if (p.ent_y[ri.first + e + half_len] < lo) { e += half_len + 1; len -= half_len + 1; }
                                else len = half_len;
                            }
                            for (; e < ri.count; ++e) {
                                const int32_t y = p.ent_y[ri.first + e];
                                if (y >= lo + 64) break;
                                const uint32_t j = static_cast<uint32_t>(y - lo);
                                if (j < 64u) {
                                    uint8_t *at = dst + lane * 128 + (((j >> 3) ^ (lane & 7)) << 4) + (j & 7) * 2;
                                    const float val = p.ent_v[ri.first + e];
                                    const __nv_bfloat16 top = __float2bfloat16_rn(val);
                                    *reinterpret_cast<__nv_bfloat16 *>(at) = top;
                                    if (p.twin)
                                        *reinterpret_cast<__nv_bfloat16 *>(at + kTwin * 128) =
                                            __float2bfloat16_rn(val - __bfloat162float(top));
                                }
                            }
                        }
                    }
                    tc::fence_smem_to_async();
                    __syncwarp();
                    if (lane == 0) arrive(&bars[B::out_full + slot]);
                }
                tc::fence_before_sync();                // the accumulator has been read
                __syncwarp();
                if (lane == 0) {
                    if (G == 2) arrive_at(released + buf * 8); else arrive(&bars[B::acc_empty + buf]);
                }
            }
        }
    } else if (warp >= kStoreWarp0) {
        // Two threads send the slots out in turn, each with all but one of its stores read: a store
        // takes its thread a few hundred cycles, which the warps that fill the slots need not
        // wait for.
        if constexpr (MODE != kFwd) {
            if (lane == 0) {
                const uint32_t mine = warp - kStoreWarp0;
                constexpr uint32_t kLag = kSlots / 2 - 1;       // own stores that may still be read
                uint32_t groups = 0;
                TileId t;
                bool ok = true;
                wait_previous();
                for (uint32_t n = 0; ok && tile_at(p, n, worker, workers, t); ++n) {
                    const Prod &q = p.prod[t.which];
                    const int32_t n0 = t.nt * q.n, y = (t.mt * G + rank) * kTM;
                    const int step = q.out_f32 ? 32 : 64, end = min(q.n, q.cols - n0);
                    for (int c = 0; c < end; c += step, ++groups) {
                        if ((groups & 1) != mine) continue;
                        const uint32_t slot = groups % kSlots;
                        const uint8_t *src = sm + kStages * kStageBytes + slot * kSlotBytes;
                        if (!wait_or_fail(&bars[B::out_full + slot], (groups / kSlots) & 1, &s_fail)) { ok = false; break; }
                        if (y < q.rows) {
                            if (MODE == kDz) store_3d(&q.out, 0, y, (n0 + c) / 64, src, false);
                            else store_3d(&q.out, n0 + c, q.out_y0 + y, t.split, src, q.out_add != 0);
                        }
                        tc::bulk_commit();
                        if (kLag == 0) tc::bulk_wait_read(); else store_wait_read1();
                        if (kLag == 0) arrive(&bars[B::out_free + slot]);
                        else if (groups >= 2) arrive(&bars[B::out_free + (groups - 2) % kSlots]);
                    }
                }
                tc::bulk_wait_all();
            }
        }
    }
    tc::fence_before_sync();
    __syncthreads();
    if (tid == 0 && failed(&s_fail)) atomicCAS(p.error, 0, static_cast<int>(kDevErrTimeout));
    if (G == 2) cluster_sync();                         // neither block ends under the other's copies or arrivals
    tc::fence_after_sync();
    if (warp == 2) pair_dealloc<G>(tm);
}

// ---- forward: joining the tiles, and the positions' own logits --------------------------

__device__ __forceinline__ void add_products(const uint4 &a, const uint4 &b, float &s0, float &s1) {
    const __nv_bfloat162 *pa = reinterpret_cast<const __nv_bfloat162 *>(&a), *pb = reinterpret_cast<const __nv_bfloat162 *>(&b);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float2 u = __bfloat1622float2(pa[k]), v = __bfloat1622float2(pb[k]);
        s0 = fmaf(u.x, v.x, s0);
        s1 = fmaf(u.y, v.y, s1);
    }
}

// x_c . w_y over D (a multiple of 8), one warp; every lane returns it.  Four loads of either row
// at a time: a single one waits for memory as long.
__device__ __forceinline__ float row_dot(const __nv_bfloat16 *x, const __nv_bfloat16 *w, int32_t D) {
    const int lane = threadIdx.x & 31;
    constexpr int kAtOnce = 4;
    const uint4 *px = reinterpret_cast<const uint4 *>(x), *pw = reinterpret_cast<const uint4 *>(w);
    float s0 = 0.f, s1 = 0.f;
    int32_t i = lane;
    for (; i + 32 * (kAtOnce - 1) < D / 8; i += 32 * kAtOnce) {
        uint4 a[kAtOnce], b[kAtOnce];
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) { a[j] = __ldg(px + i + j * 32); b[j] = __ldg(pw + i + j * 32); }
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) add_products(a[j], b[j], s0, s1);
    }
    for (; i < D / 8; i += 32) add_products(__ldg(px + i), __ldg(pw + i), s0, s1);
    float s = s0 + s1;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return s;
}

struct SemParams {
    const __nv_bfloat16 *x, *w;
    const int32_t *row_ptr, *row_sem, *target;
    const float *lse, *dlogp;
    float *logp, *lse_out;
    const float2 *part;             // forward: [C][tiles]
    const uint8_t *top;
    RowInfo *rows;
    int32_t *ent_y, *raw_y;
    float *ent_v, *raw_v;
    int64_t C, S;
    int32_t V, D, tiles, width;     // tiles of `width` columns
    float scale, c2;                // c2: as the tiles'
};

// The positions' own logits, one warp each (the q-th of row_sem; its row by binary search in
// row_ptr), into logp.  They need only the inputs and are formed while the tiles are; the first
// block stays until the tiles are done, so that whoever waits for this kernel finds both.
__global__ void __launch_bounds__(256) head_labels_kernel(SemParams p) {
    const int64_t q = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    let_next_start();
    if (q < p.S) {
        int64_t lo = 0, hi = p.C;                   // last row with row_ptr <= q
        while (hi - lo > 1) {
            const int64_t mid = (lo + hi) >> 1;
            if (__ldg(p.row_ptr + mid) <= q) lo = mid; else hi = mid;
        }
        const int32_t s = __ldg(p.row_sem + q);
        if (s >= 0 && s < p.S) {
            const int32_t y = __ldg(p.target + s);
            float z = 0.f;
            if (y >= 0 && y < p.V) z = p.scale * row_dot(p.x + lo * p.D, p.w + static_cast<int64_t>(y) * p.D, p.D);
            if ((threadIdx.x & 31) == 0) p.logp[s] = z;
        }
    }
    if (blockIdx.x == 0) wait_previous();
}

// Joins a row's pairs (accumulator of the largest logit, sum of 2^(c2 v - c2 max)) to its lse, and takes it from
// the logits of the row's positions; one block a row.  The row's largest logit is formed again by
// a dot product: where one entry has most of the probability, as sampled tokens mostly do, its
// error is lse's, and what the tensor cores truncate from a sum whose terms are mostly of one
// sign is more than logit_factor gives back.  (1 x 157,184 x 2,048, lse 19.86: off by 1.0e-6 of
// it, 1.3e-7 with the dot product; a label's logp of -0.0031 by 2.0e-5, 1.6e-7.  4,096 rows: lse
// and logp off by 1.9e-7 in relative L2 without it, 5.4e-8 with.  It costs 1 us of 106 for that
// row, 2.5 us of 53 for 777 rows x 32,003 x 1,032, 0.5 % for the 4,096.)
constexpr int kRowThreads = 128;
__global__ void __launch_bounds__(kRowThreads) head_finish_kernel(SemParams p) {
    __shared__ float2 s_max[kRowThreads / 32], s_sum[kRowThreads / 32];
    const int64_t c = blockIdx.x;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int32_t b = max(0, __ldg(p.row_ptr + c));
    const int32_t e = static_cast<int32_t>(min(static_cast<int64_t>(__ldg(p.row_ptr + c + 1)), p.S));
    const float2 *pairs = p.part + c * p.tiles;
    // this thread's first position, its label and its logit are fetched ahead of what they wait for
    int32_t s = b + tid < e ? __ldg(p.row_sem + b + tid) : -1;
    int32_t y = s >= 0 && s < p.S ? __ldg(p.target + s) : -1;
    wait_previous();
    float label_z = y >= 0 && y < p.V ? p.logp[s] : 0.f;
    float m = -INFINITY;
    int32_t tile = 0;
#pragma unroll 4
    for (int32_t i = tid; i < p.tiles; i += kRowThreads) {
        const float t = pairs[i].x * p.c2;
        if (t > m) { m = t; tile = i; }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float m2 = __shfl_xor_sync(0xffffffffu, m, o);
        const int32_t t2 = __shfl_xor_sync(0xffffffffu, tile, o);
        if (m2 > m || (m2 == m && t2 < tile)) { m = m2; tile = t2; }
    }
    if (lane == 0) s_max[warp] = make_float2(m, __int_as_float(tile));
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kRowThreads / 32; ++i) {
        const float2 t = s_max[i];
        const int32_t t2 = __float_as_int(t.y);
        if (t.x > m || (t.x == m && t2 < tile)) { m = t.x; tile = t2; }
    }
    const int32_t top = min(tile * p.width + p.top[c * p.tiles + tile], p.V - 1);
    const float own = ex2(fmaf(pairs[tile].x, p.c2, -m));           // its term of the tile's sum: 1 but for m's rounding
    float sum = 0.f, d0 = 0.f, d1 = 0.f;
#pragma unroll 4
    for (int32_t i = tid; i < p.tiles; i += kRowThreads) {
        const float2 t = pairs[i];
        sum = fmaf(t.y, ex2(t.x * p.c2 - m), sum);
    }
    const uint4 *px = reinterpret_cast<const uint4 *>(p.x + c * p.D);
    const uint4 *pw = reinterpret_cast<const uint4 *>(p.w + static_cast<int64_t>(top) * p.D);
#pragma unroll 2
    for (int32_t i = tid; i < p.D / 8; i += kRowThreads) add_products(__ldg(px + i), __ldg(pw + i), d0, d1);
    d0 += d1;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        sum += __shfl_xor_sync(0xffffffffu, sum, o);
        d0 += __shfl_xor_sync(0xffffffffu, d0, o);
    }
    if (lane == 0) s_sum[warp] = make_float2(sum, d0);
    __syncthreads();
    sum = d0 = 0.f;
#pragma unroll
    for (int i = 0; i < kRowThreads / 32; ++i) { sum += s_sum[i].x; d0 += s_sum[i].y; }
    // lse = z + rest, z the largest logit
    float z = p.scale * d0, rest;
    const float off = m - z * kLog2e;
    if (fabsf(off) < 64.f) {
        const float others = sum - own;                 // a NaN among the logits is in the sum alone, and stays in it
        rest = log1pf((others < 0.f ? 0.f : others) * exp2f(off));
    } else {                                            // logits that are not finite, or beyond fp32's digits
        z = m * kLn2;
        rest = log2f(sum) * kLn2;
    }
    if (tid == 0) p.lse_out[c] = z + rest;
    for (int32_t i = b + tid; i < e;) {
        if (y >= 0 && y < p.V) p.logp[s] = ((y == top ? z : label_z) - z) - rest;
        if ((i += kRowThreads) >= e) break;
        s = __ldg(p.row_sem + i);
        y = s >= 0 && s < p.S ? __ldg(p.target + s) : -1;
        label_z = y >= 0 && y < p.V ? p.logp[s] : 0.f;
    }
}

// X in panels of 64 columns, [panels][rows][64], zero past D, where its rows straddle lines:
// each 128-byte row of a box then lies in one line instead of two; the rows are read once a tile
// of the vocabulary, and misaligned lines bound the product (777 x 32,003 x 1,032 forward: 66.8 us
// with X as it is, 54.3 us with the copy made first).  For a twin dZ (`fold` 32): rows 0 .. 31 and
// again, zero past C.
struct PadParams { const __nv_bfloat16 *x; __nv_bfloat16 *out; int64_t C, rows; int32_t D, fold; };
__device__ __forceinline__ void pad_rows(const PadParams &p, uint32_t block, uint32_t blocks) {
    const int64_t n = p.rows * ((p.D + 63) / 64) * 8;
    for (int64_t i = static_cast<int64_t>(block) * 256 + threadIdx.x; i < n; i += static_cast<int64_t>(blocks) * 256) {
        int64_t row = (i >> 3) % p.rows;
        const int64_t panel = (i >> 3) / p.rows, col = panel * 64 + (i & 7) * 8;
        if (p.fold > 0) row %= p.fold;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (col < p.D && row < p.C) v = __ldg(reinterpret_cast<const uint4 *>(p.x + row * p.D + col));
        reinterpret_cast<uint4 *>(p.out)[i] = v;
    }
}
__global__ void __launch_bounds__(256) head_pad_kernel(PadParams p) {
    let_next_start();
    pad_rows(p, blockIdx.x, gridDim.x);
}

// ---- backward: per row, G and the distinct labels with a gradient of their own ----------

// Label and gradient of the q-th of row_sem; -1 and 0 where the position has no label.
__device__ __forceinline__ int32_t label_of(const SemParams &p, int32_t q, float &g) {
    const int32_t s = __ldg(p.row_sem + q);
    g = 0.f;
    if (s < 0 || s >= p.S) return -1;
    const int32_t y = __ldg(p.target + s);
    if (y < 0 || y >= p.V) return -1;
    g = __ldg(p.dlogp + s);
    return y;
}
// (Labels are looked up again from the workspace: whatever it holds, the weight's rows are kept to.)
__device__ __forceinline__ float finish_entry(const SemParams &p, int64_t c, int32_t y, float sum, float G, float lse) {
    y = min(max(y, 0), p.V - 1);
    const float z = p.scale * row_dot(p.x + c * p.D, p.w + static_cast<int64_t>(y) * p.D, p.D);
    return p.scale * (sum - G * expf(z - lse));
}

// Distinct labels of a row that one warp gathers.  By measurement (the backward in us, 157,184 x
// 2,048, one row in eight of 64 with that many positions, by the warp / by the block): 32 labels
// 428 / 364, 64 524 / 371, 200 931 / 410; every row of 64: 32 labels 439 / 450, 64 532 / 532,
// 200 951 / 857, 100 labels in 3,000 positions 888 / 1,033.
constexpr int kFewLabels = 16;
constexpr int kRowWarps = 8;

struct SortSpace {
    int32_t base[256], count[kRowWarps][256], sums[kRowWarps];
};

// Sum over the block of what the threads before this one hold; `total` of all.
__device__ __forceinline__ int32_t block_before(int32_t v, SortSpace &sm, int32_t &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int32_t up = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int32_t t = __shfl_up_sync(0xffffffffu, up, o);
        if (lane >= o) up += t;
    }
    if (lane == 31) sm.sums[warp] = up;
    __syncthreads();
    int32_t before = 0;
    total = 0;
#pragma unroll
    for (int i = 0; i < kRowWarps; ++i) {
        if (i < warp) before += sm.sums[i];
        total += sm.sums[i];
    }
    __syncthreads();
    return before + up - v;
}

// n pairs by the eight bits of the key from `shift` on, equal ones in the order they had.
__device__ void radix_pass(const int32_t *y, const float *v, int32_t *to_y, float *to_v, int32_t n, int shift, SortSpace &sm) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    sm.base[tid] = 0;
#pragma unroll
    for (int w = 0; w < kRowWarps; ++w) sm.count[w][tid] = 0;
    __syncthreads();
    for (int32_t i = tid; i < n; i += 256) atomicAdd(&sm.base[y[i] >> shift & 255], 1);
    __syncthreads();
    int32_t total;
    const int32_t first = block_before(sm.base[tid], sm, total);
    sm.base[tid] = first;                               // where this digit's next pair goes
    for (int32_t from = 0; from < n; from += 256) {
        const int32_t i = from + tid;
        const bool on = i < n;
        const int32_t key = on ? y[i] : 0;
        const float val = on ? v[i] : 0.f;
        const int digit = on ? key >> shift & 255 : 256;
        const uint32_t same = __match_any_sync(0xffffffffu, digit);
        const int rank = __popc(same & ((1u << lane) - 1u));
        if (on && rank == 0) sm.count[warp][digit] = __popc(same);
        __syncthreads();
        int32_t at = sm.base[tid];
#pragma unroll
        for (int w = 0; w < kRowWarps; ++w) {
            const int32_t k = sm.count[w][tid];
            sm.count[w][tid] = at;
            at += k;
        }
        sm.base[tid] = at;
        __syncthreads();
        if (on) {
            const int32_t dst = min(sm.count[warp][digit] + rank, n - 1);   // rows that overlap would not add up
            to_y[dst] = key;
            to_v[dst] = val;
        }
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kRowWarps; ++w) sm.count[w][tid] = 0;
        __syncthreads();
    }
}

// A row with many distinct labels, by the whole block: its positions are sorted by label (a pass
// per eight bits of the vocabulary, between the two pairs of arrays), equal labels staying in
// position order; a warp adds up a label's run and finishes its entry.  Work grows with the
// positions, and with the labels only by a dot product each.
__device__ void many_labels(const SemParams &p, int64_t c, float G, SortSpace &sm) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int32_t b = max(0, __ldg(p.row_ptr + c));
    const int32_t n = static_cast<int32_t>(min(static_cast<int64_t>(__ldg(p.row_ptr + c + 1)), p.S)) - b;
    const int bits = 32 - __clz(p.V);                   // V stands for no label, and is sorted last
    int32_t *y0 = p.raw_y + b, *y1 = p.ent_y + b;
    float *v0 = p.raw_v + b, *v1 = p.ent_v + b;
    const bool odd = (bits + 7) / 8 & 1;                // the last pass has to end in the raw arrays
    int32_t *y = odd ? y1 : y0;
    float *v = odd ? v1 : v0;
    for (int32_t i = tid; i < n; i += 256) {
        float g;
        const int32_t label = label_of(p, b + i, g);
        y[i] = label < 0 ? p.V : label;
        v[i] = g;
    }
    __syncthreads();
    for (int shift = 0; shift < bits; shift += 8) {
        int32_t *to_y = y == y0 ? y1 : y0;
        float *to_v = v == v0 ? v1 : v0;
        radix_pass(y, v, to_y, to_v, n, shift, sm);
        y = to_y;
        v = to_v;
    }
    int32_t found = 0;
    for (int32_t from = 0; from < n; from += 256) {     // where each label's run begins
        const int32_t i = from + tid;
        const bool begins = i < n && y0[i] < p.V && (i == 0 || y0[i - 1] != y0[i]);
        int32_t total;
        const int32_t k = found + block_before(begins, sm, total);
        if (begins) y1[k] = i;
        found += total;
    }
    __syncthreads();
    const float lse = p.lse[c];
    for (int32_t k = warp; k < found; k += kRowWarps) {
        const int32_t from = min(max(y1[k], 0), n - 1), label = y0[from];
        float sum = 0.f;
        bool run = true;
        for (int32_t i = from + lane; run; i += 32) {
            const bool in = i < n && y0[i] == label;
            if (in) sum += v0[i];
            run = __all_sync(0xffffffffu, in);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        const float e = finish_entry(p, c, label, sum, G, lse);
        __syncwarp();
        if (lane == 0) {
            y1[k] = label;
            v1[k] = e;
        }
    }
    if (tid == 0) p.rows[c] = RowInfo{-p.scale * G, lse * kLog2e, found, b};
    __syncthreads();
}

// One warp a row.  Its positions are taken 32 at a time: lanes with one label are added in
// position order, and their sum to the label's entry in (raw_y, raw_v), found among the entries
// so far; a row's positions mostly share few labels.  Entries whose gradients do not cancel are
// then put in label order, so that a tile finds its own among many, and finished:
// ent_v = scale (sum g - G e^(z - lse)) in fp32, written over the row's softmax term when the
// tile is formed.  A row that turns out to have more than kFewLabels distinct labels is left to
// the whole block, which sorts it: the warp's steps grow with d^2, its dot products come one by one.
// Blocks from `pad_from` on copy X instead, where a copy is wanted.
__global__ void __launch_bounds__(32 * kRowWarps) head_rows_kernel(SemParams p, PadParams pad, uint32_t pad_from) {
    __shared__ SortSpace space;
    __shared__ float row_g[kRowWarps];
    __shared__ bool many[kRowWarps];
    if (blockIdx.x >= pad_from) {
        let_next_start();
        pad_rows(pad, blockIdx.x - pad_from, gridDim.x - pad_from);
        return;
    }
    const int64_t c0 = static_cast<int64_t>(blockIdx.x) * kRowWarps, c = c0 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    let_next_start();
    float G = 0.f;
    int32_t found = 0, b = 0;
    if (c < p.C) {
        b = max(0, __ldg(p.row_ptr + c));
        const int32_t e = static_cast<int32_t>(min(static_cast<int64_t>(__ldg(p.row_ptr + c + 1)), p.S));
        for (int32_t base = b; base < e; base += 32) {
            int32_t y = -1;
            float g = 0.f;
            if (base + lane < e) y = label_of(p, base + lane, g);
            G += g;
            if (found > kFewLabels) continue;           // only G is still wanted
            const uint32_t same = __match_any_sync(0xffffffffu, y);
            const bool leads = y >= 0 && lane == __ffs(same) - 1;
            float sum = 0.f;
#pragma unroll 8
            for (int i = 0; i < 32; ++i) {
                const float gi = __shfl_sync(0xffffffffu, g, i);
                if (same >> i & 1u) sum += gi;
            }
            int32_t at = -1;
            for (int32_t k = 0; k < found; ++k)
                if (p.raw_y[b + k] == y) at = k;
            const bool fresh = leads && at < 0;
            const uint32_t mask = __ballot_sync(0xffffffffu, fresh);
            if (fresh) {
                const int32_t k = b + found + __popc(mask & ((1u << lane) - 1u));
                p.raw_y[k] = y;
                p.raw_v[k] = sum;
            } else if (leads) {
                p.raw_v[b + at] += sum;
            }
            found += __popc(mask);
            __syncwarp();
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) G += __shfl_xor_sync(0xffffffffu, G, o);
    }
    if (c < p.C && found <= kFewLabels) {
        int32_t count = 0;
        for (int32_t base = 0; base < found; base += 32) {
            const int32_t k = base + lane;
            const int32_t y = k < found ? p.raw_y[b + k] : -1;
            const float v = k < found ? p.raw_v[b + k] : 0.f;
            int32_t before = 0;
            for (int32_t j = 0; j < found; ++j) before += p.raw_v[b + j] != 0.f && p.raw_y[b + j] < y;
            if (v != 0.f) {
                p.ent_y[b + before] = y;
                p.ent_v[b + before] = v;
            }
            count += __popc(__ballot_sync(0xffffffffu, v != 0.f));
        }
        __syncwarp();
        const float lse = p.lse[c];
        for (int32_t i = 0; i < count; ++i) {
            const float v = finish_entry(p, c, p.ent_y[b + i], p.ent_v[b + i], G, lse);
            __syncwarp();
            if (lane == 0) p.ent_v[b + i] = v;
        }
        if (lane == 0) p.rows[c] = RowInfo{-p.scale * G, lse * kLog2e, count, b};
    }
    if (lane == 0) {
        row_g[threadIdx.x >> 5] = G;
        many[threadIdx.x >> 5] = found > kFewLabels;
    }
    if (!__syncthreads_or(found > kFewLabels)) return;
    for (int i = 0; i < kRowWarps; ++i)
        if (many[i]) many_labels(p, c0 + i, row_g[i], space);
}

// dX in bf16 from the splits' fp32 sums, in ascending order; a twin dZ's second half last.
struct DxParams { const float *acc; __nv_bfloat16 *dx; int64_t n, layer, twin; int32_t splits; };
__global__ void __launch_bounds__(128) head_dx_kernel(DxParams p) {
    wait_previous();
    for (int64_t i = (static_cast<int64_t>(blockIdx.x) * 128 + threadIdx.x) * 4; i < p.n;
         i += static_cast<int64_t>(gridDim.x) * 128 * 4) {
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
        for (int32_t s = 0; s < p.splits; ++s) {
            const float4 a = *reinterpret_cast<const float4 *>(p.acc + s * p.layer + i);
            v.x += a.x; v.y += a.y; v.z += a.z; v.w += a.w;
        }
        if (p.twin > 0) {
            float4 u = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
            for (int32_t s = 0; s < p.splits; ++s) {
                const float4 a = *reinterpret_cast<const float4 *>(p.acc + s * p.layer + p.twin + i);
                u.x += a.x; u.y += a.y; u.z += a.z; u.w += a.w;
            }
            v.x += u.x; v.y += u.y; v.z += u.z; v.w += u.w;
        }
        *reinterpret_cast<uint2 *>(p.dx + i) = make_uint2(tc::pack_bf16(v.x, v.y), tc::pack_bf16(v.z, v.w));
    }
}

// ---- host ---------------------------------------------------------------------------------

size_t align256(size_t x) { return (x + 255) / 256 * 256; }

// What a tile costs, in columns: a step of K takes a pair two cycles a column, but no less than
// its copies and barriers do (430 - 450 cycles below 220 columns); 16 more for the tile's ends.
int32_t tile_cost(int32_t n) { return std::max(n, 220) + 16; }

// The forward's cut: blocks that share a tile (pairs: 256 rows) and the tile width, a multiple
// of 16 columns a block, by the busiest worker's tiles.  A block alone reads its columns from L2
// where a pair shares them, and takes 1.2 as long, 1.4 where the weight's rows straddle lines
// (777 x 32,003 x 1,032: 64.2 us alone, 54.3 us in pairs), but wastes less where the rows end early
// in a tile (300 x 157,184 x 2,048: 179 us alone, 202 us in pairs).
struct Cut { int group; int32_t width; };
Cut fwd_cut(int64_t C, int32_t V, int32_t D) {
    Cut best{1, kTN};
    double least = 0.0;
    const double alone = D % 64 ? 1.4 : 1.2;
    for (int G = 1; G <= (C > kTM ? 2 : 1); ++G)
        for (int32_t n = kTN; n >= 64; n -= 16 * G) {
            const int64_t tiles = int64_t(ceil_div(C, kTM * G)) * ceil_div(V, n), workers = sm_count() / G;
            const double cost = double((tiles + workers - 1) / workers) * tile_cost(n) * (G == 1 ? alone : 1.0);
            if (least == 0.0 || cost < least) { least = cost; best = Cut{G, n}; }
        }
    return best;
}

// The backward's group: pairs where their 256 rows are three quarters full.  By measurement (alone /
// pairs, us): 32,003 x 1,032, 129 rows 81 / 87, 224 90 / 92, 256 102 / 93, 300 119 / 106, 513
// 157 / 126; 157,184 x 2,048, 129 rows 428 / 423, 192 444 / 436, 224 480 / 449, 300 608 / 592.
int bwd_group(int64_t C) { return C <= 3 * kTM / 2 ? 1 : 2; }

// Tile width over `cols` columns in multiples of `unit`: the least work for the busiest worker,
// as above.
int32_t tile_width(int32_t m_tiles, int64_t cols, int32_t unit, int G) {
    int32_t best = kTN;
    int64_t cost = INT64_MAX;
    const int64_t workers = sm_count() / G;
    for (int32_t n = kTN; n >= 64; n -= unit) {
        const int64_t tiles = int64_t(m_tiles) * ceil_div(cols, n);
        const int64_t c = (tiles + workers - 1) / workers * tile_cost(n);
        if (c < cost) { cost = c; best = n; }
    }
    return best;
}

// [rows][cols] bf16, read in boxes of 64 columns x box_rows.
bool map_in(CUtensorMap *m, const void *base, int64_t rows, int64_t cols, int64_t pitch, int32_t box_rows) {
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(pitch) * 2};
    const cuuint32_t box[2] = {64, static_cast<cuuint32_t>(box_rows)};
    return encode_bf16(m, base, 2, dims, strides, box);
}

// Whether X is copied into aligned panels first: its rows straddle lines, and there are enough of
// them for several tiles to read each.  By measurement (as they are / copied, us, V = 32,003,
// D = 1,032): forward 129 rows 29.2 / 29.2, 256 31.0 / 29.1, 385 41.0 / 37.0; backward, where a
// smaller part of the work reads X, 256 rows 94 / 97, 300 107 / 107, 513 135 / 126.
bool pads_x(int64_t C, int32_t D, bool backward) { return D % 64 != 0 && C > (backward ? 2 * kTM : kTM); }
size_t pad_bytes(int64_t rows, int32_t D) { return align256(size_t(2) * static_cast<size_t>(rows) * ((D + 63) / 64 * 64)); }
int64_t pad_blocks(int64_t rows, int32_t D) {
    return std::min<int64_t>((rows * ((D + 63) / 64) * 8 + 255) / 256, int64_t(sm_count()) * 8);
}

// dZ in panels of 64 columns, [panels][C][64]: every box that is written, read as rows
// (dX) or as columns (dW) is one contiguous run, or two.  The aligned copy of X is kept so too.  Row-major, a box's 64 or 128
// rows lie a whole piece (128 KB) apart each.
bool map_panels(CUtensorMap *m, void *dz, int64_t C, int32_t nv, int32_t box_rows, int32_t box_panels) {
    const cuuint64_t dims[3] = {64, static_cast<cuuint64_t>(C), static_cast<cuuint64_t>((nv + 63) / 64)};
    const cuuint64_t strides[2] = {128, static_cast<cuuint64_t>(C) * 128};
    const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(box_rows), static_cast<cuuint32_t>(box_panels)};
    return encode_bf16(m, dz, 3, dims, strides, box);
}

// A row-major [rows][D] operand that is read as columns, in boxes of 64 rows x `cols` columns:
// the columns that fill panels of 64 as panels, so that one copy brings a tile's; the others
// (the panel they lie in would reach past the last row's end) in boxes of 64 through `edge`.
bool map_cols(CUtensorMap *m, CUtensorMap *edge, const void *base, int64_t rows, int64_t D, int32_t cols) {
    if (D % 64 && !map_in(edge, base, rows, D, D, 64)) return false;
    if (D < 64) { *m = *edge; return true; }            // no whole panel; a map is fetched all the same
    const cuuint64_t dims[3] = {64, static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(D / 64)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(D) * 2, 128};
    const cuuint32_t box[3] = {64, 64, static_cast<cuuint32_t>(cols / 64)};
    return encode_bf16(m, base, 3, dims, strides, box);
}

// [layers][rows][cols], written in boxes of 128 bytes x 128 rows.
bool map_out(CUtensorMap *m, void *base, int64_t layers, int64_t rows, int64_t cols, int64_t pitch, bool f32) {
    const cuuint64_t e = f32 ? 4 : 2;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(layers)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(pitch) * e, static_cast<cuuint64_t>(pitch) * e * rows};
    const cuuint32_t box[3] = {f32 ? 32u : 64u, kTM, 1};
    const cuuint32_t es[3] = {1, 1, 1};
    auto fn = encode_tiled();
    return fn && fn(m, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, base, dims, strides,
                    box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int MODE, int G>
cudaError_t launch_group(Params &p, bool behind, cudaStream_t st) {
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = allow_smem(head_tile_kernel<MODE, G>, Ring<MODE, G>::smem, done);
    if (e != cudaSuccess) return e;
    const uint32_t workers = share_tiles(p, sm_count() / G);
    return launch(head_tile_kernel<MODE, G>, int64_t(workers) * G, kThreads, Ring<MODE, G>::smem, G, behind, st, p);
}
template <int MODE>
cudaError_t launch_tiles(Params &p, int G, bool behind, cudaStream_t st) {
    return G == 2 ? launch_group<MODE, 2>(p, behind, st) : launch_group<MODE, 1>(p, behind, st);
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

int check(const harts_linear_logprob_fwd_args *a) {
    if (!a) { set_error("NULL args"); return HARTS_EINVAL; }
    if (a->dtype != HARTS_BF16) { set_error("hidden rows and weight must be bf16"); return HARTS_EUNSUPPORTED; }
    if (a->C < 0 || a->S < 0 || a->V < 1 || a->D < 1) { set_error("C, S >= 0 and V, D >= 1 required"); return HARTS_EINVAL; }
    if (a->D % 8) { set_error("D must be a multiple of 8 (rows start 16-byte aligned)"); return HARTS_EUNSUPPORTED; }
    // the kernels' int32 indices take steps of up to 256 past the last one
    if (a->S > 0x7fffff00 || a->C > 0x7fffff00 || a->V > 0x7fffff00) { set_error("C, V or S beyond int32 rows"); return HARTS_EOVERFLOW; }
    const int64_t c = a->C / kTM + 1, v = a->V / 64 + 1, d = a->D / 64 + 1;      // tiles are counted in 32 bits
    if (c * v > 0x3fffffff || (c + v) * d > 0xffffff) {
        set_error("more tiles than the library counts");
        return HARTS_EOVERFLOW;
    }
    if (!std::isfinite(a->scale)) { set_error("scale must be finite"); return HARTS_EINVAL; }
    if (a->C > 0 && (!a->x || !a->weight || !a->row_ptr || !a->lse)) { set_error("NULL x, weight, row_ptr or lse"); return HARTS_EINVAL; }
    if (a->S > 0 && (!a->row_sem || !a->target)) { set_error("NULL row_sem or target"); return HARTS_EINVAL; }
    if (!aligned16(a->x) || !aligned16(a->weight) || !aligned16(a->workspace)) {
        set_error("x, weight and workspace must be 16-byte aligned");
        return HARTS_EINVAL;
    }
    return HARTS_OK;
}

int cuda_fail(cudaError_t e, const char *what) {
    set_error(std::string(what) + ": " + cudaGetErrorString(e));
    return HARTS_ECUDA;
}

// scale * log2 e, with the tensor cores' truncation taken back to first order.  An accumulator
// is cut towards zero at every 16 columns of K, which shrinks a logit by D/16 times a quarter of
// 2^-24 on average (measured with one vocabulary entry, whose lse is its logit: 0.20 - 0.29 for
// products of either sign at D = 64 .. 4096, up to 0.9 where all have one sign).  Uncorrected
// that is the largest error of lse, 1.6e-6 of it at D = 2048.  Logits that nothing is cut from
// (one channel a row, values on a coarse grid) are off by the quarter instead: D/16 2^-26 of
// them, 3.8e-6 at D = 4096.
float logit_factor(float scale, int32_t D) {
    return static_cast<float>(double(scale) * 1.4426950408889634 * (1.0 + 0.25 * (D / 16.0) * 0x1p-24));
}

SemParams sem_params(const harts_linear_logprob_fwd_args *a) {
    SemParams s{};
    s.x = static_cast<const __nv_bfloat16 *>(a->x); s.w = static_cast<const __nv_bfloat16 *>(a->weight);
    s.row_ptr = a->row_ptr; s.row_sem = a->row_sem; s.target = a->target; s.lse = s.lse_out = a->lse; s.logp = a->logp;
    s.C = a->C; s.S = a->S; s.V = a->V; s.D = a->D; s.scale = a->scale;
    return s;
}

// How the backward is cut: vocabulary entries a piece, K splits of dX, and where things lie
// in the workspace.
struct BwdPlan {
    int32_t group, piece, n_pieces, n_dz, n_grad, splits, k_per;
    bool acc;                       // dX goes through fp32 sums
    bool twin;                      // dZ in two bf16 terms
    int32_t dz_rows;                // rows of dZ and of those sums
    size_t pad, rows, ent_y, ent_v, raw_y, raw_v, dz, dx, total;
};

constexpr size_t kPieceBytes = size_t(512) << 20;     // dZ of one piece, when the caller sets no piece

BwdPlan plan_bwd(int64_t C, int32_t V, int32_t D, int64_t S, int32_t piece) {
    BwdPlan b{};
    // Up to 32 rows a step of K has room for as many again, which take what bf16 cuts from dZ
    // (against X a second time).  With few rows one label's rounding is a whole row's error,
    // 2.8e-3 against the 1.7e-3 that rounding the result alone gives; over many rows it averages
    // out.  31 x 32,003 x 1,032 takes 62.8 us with it and 57.2 us without.  (64 rows, in two
    // steps: 71 us instead of 59 for 61 rows, for 2.4e-3; not taken.)
    b.twin = C <= kTwin;
    b.dz_rows = b.twin ? 2 * kTwin : static_cast<int32_t>(C);
    int64_t want = piece > 0 ? piece : static_cast<int64_t>(kPieceBytes / (2 * std::max<int64_t>(b.dz_rows, 1)));
    want = std::max<int64_t>(kTN, want / kTN * kTN);
    b.piece = static_cast<int32_t>(std::min<int64_t>(want, (int64_t(V) + 63) / 64 * 64));
    b.n_pieces = ceil_div(V, b.piece);
    const int G = b.group = bwd_group(C);
    const int32_t mt = ceil_div(C, kTM * G);
    b.n_dz = tile_width(mt, std::min<int32_t>(b.piece, V), 64, G);
    const int32_t unit = 64 * G;                        // columns stored [K][columns] come in 64s per block
    b.n_grad = (ceil_div(D, ceil_div(D, kTN)) + unit - 1) / unit * unit;
    const int32_t kb = ceil_div(std::min<int32_t>(b.piece, V), kTK), tiles = mt * ceil_div(D, b.n_grad);
    // about two rounds of dX tiles over the SMs, each at least 16 steps deep
    b.splits = std::max(1, std::min({static_cast<int32_t>(ceil_div(2 * sm_count() / G, tiles)), ceil_div(kb, 16), int32_t(32)}));
    b.k_per = ceil_div(kb, b.splits);
    b.splits = ceil_div(kb, b.k_per);
    b.acc = b.twin || b.splits > 1 || b.n_pieces > 1;
    b.pad = 0;
    b.rows = b.twin ? pad_bytes(b.dz_rows, D) : pads_x(C, D, true) ? pad_bytes(C, D) : 0;
    b.ent_y = b.rows + align256(sizeof(RowInfo) * static_cast<size_t>(C));
    b.ent_v = b.ent_y + align256(4 * static_cast<size_t>(S));
    b.raw_y = b.ent_v + align256(4 * static_cast<size_t>(S));
    b.raw_v = b.raw_y + align256(4 * static_cast<size_t>(S));
    b.dz = b.raw_v + align256(4 * static_cast<size_t>(S));
    b.dx = b.dz + align256(2 * static_cast<size_t>(b.dz_rows) * b.piece);
    b.total = b.dx + (b.acc ? align256(4 * static_cast<size_t>(b.dz_rows) * D * b.splits) : 0);
    return b;
}

}  // namespace
}  // namespace harts

using namespace harts;

extern "C" {

size_t harts_linear_logprob_fwd_workspace_bytes(int64_t C, int32_t V, int32_t D) {
    if (C < 0 || V < 1 || D < 1) return 0;
    const size_t pairs = static_cast<size_t>(C) * ceil_div(V, fwd_cut(C, V, D).width);
    return std::max<size_t>(256, (pads_x(C, D, false) ? pad_bytes(C, D) : 0) + (sizeof(float2) + 1) * pairs);
}

int harts_linear_logprob_fwd(const harts_linear_logprob_fwd_args *a, harts_stream_t stream) {
    const int rc = check(a);
    if (rc) return rc;
    if (a->S > 0 && !a->logp) { set_error("NULL logp"); return HARTS_EINVAL; }
    if (a->C == 0) {                                    // positions without rows have no label either
        const cudaError_t e = a->S > 0 ? cudaMemsetAsync(a->logp, 0, 4 * static_cast<size_t>(a->S), reinterpret_cast<cudaStream_t>(stream))
                                       : cudaSuccess;
        if (e != cudaSuccess) return cuda_fail(e, "linear log-prob forward");
        set_error("");
        return HARTS_OK;
    }
    if (!a->workspace || a->workspace_bytes < harts_linear_logprob_fwd_workspace_bytes(a->C, a->V, a->D)) {
        set_error("workspace too small");
        return HARTS_ESMALLBUF;
    }
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    Params p;
    std::memset(&p, 0, sizeof(p));
    Prod &q = p.prod[0];
    const Cut cut = fwd_cut(a->C, a->V, a->D);
    const int G = cut.group;
    q.m_tiles = ceil_div(a->C, kTM * G);
    q.n = cut.width;
    q.n_tiles = ceil_div(a->V, q.n);
    q.splits = 1;
    q.k_blocks = q.k_per = ceil_div(a->D, kTK);
    q.a_rows = static_cast<int32_t>(std::min<int64_t>(kTM, (a->C + 7) / 8 * 8));
    q.rows = static_cast<int32_t>(a->C);
    q.cols = a->V;
    p.n_prod = 1;
    p.error = a->error ? a->error : own_error_word();
    if (!p.error) { set_error("the library's error word is not to be had"); return HARTS_ECUDA; }
    p.c2 = logit_factor(a->scale, a->D);
    const bool pad = pads_x(a->C, a->D, false);
    p.part = reinterpret_cast<float2 *>(static_cast<uint8_t *>(a->workspace) + (pad ? pad_bytes(a->C, a->D) : 0));
    p.top = reinterpret_cast<uint8_t *>(p.part + a->C * q.n_tiles);
    q.a_panel = pad;
    if (!(pad ? map_panels(&q.a, a->workspace, a->C, a->D, q.a_rows, 1) : map_in(&q.a, a->x, a->C, a->D, a->D, q.a_rows)) ||
        !map_in(&q.b, a->weight, a->V, a->D, a->D, q.n / G)) {
        set_error("tensor map");
        return HARTS_ECUDA;
    }
    SemParams s = sem_params(a);
    s.part = p.part;
    s.tiles = q.n_tiles;
    s.width = q.n;
    s.c2 = p.c2;
    s.top = p.top;
    const PadParams copy{s.x, static_cast<__nv_bfloat16 *>(a->workspace), a->C, a->C, a->D, 0};
    cudaError_t e = pad ? launch(head_pad_kernel, pad_blocks(a->C, a->D), 256, 0, 1, false, st, copy) : cudaSuccess;
    if (e == cudaSuccess) e = launch_tiles<kFwd>(p, G, pad, st);
    if (e == cudaSuccess && a->S > 0) e = launch(head_labels_kernel, (a->S + 7) / 8, 256, 0, 1, true, st, s);
    if (e == cudaSuccess) e = launch(head_finish_kernel, a->C, kRowThreads, 0, 1, true, st, s);
    if (e != cudaSuccess) return cuda_fail(e, "linear log-prob forward launch");
    set_error("");
    return HARTS_OK;
}

size_t harts_linear_logprob_bwd_workspace_bytes(int64_t C, int32_t V, int32_t D, int64_t S, int32_t piece) {
    if (C < 0 || V < 1 || D < 1 || S < 0 || piece < 0) return 0;
    return std::max<size_t>(256, plan_bwd(C, V, D, S, piece).total);
}

int harts_linear_logprob_bwd(const harts_linear_logprob_bwd_args *a, harts_stream_t stream) {
    if (!a) { set_error("NULL args"); return HARTS_EINVAL; }
    const harts_linear_logprob_fwd_args &f = a->fwd;
    const int rc = check(&f);
    if (rc) return rc;
    if (a->piece < 0) { set_error("piece must be >= 0"); return HARTS_EINVAL; }
    if (f.S > 0 && !a->dlogp) { set_error("NULL dlogp"); return HARTS_EINVAL; }
    if (!a->dweight || (f.C > 0 && !a->dx)) { set_error("NULL dx or dweight"); return HARTS_EINVAL; }
    if (!aligned16(a->dx) || !aligned16(a->dweight)) { set_error("dx and dweight must be 16-byte aligned"); return HARTS_EINVAL; }
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (f.C == 0) {
        const cudaError_t e = cudaMemsetAsync(a->dweight, 0, 2 * static_cast<size_t>(f.V) * f.D, st);
        if (e != cudaSuccess) return cuda_fail(e, "linear log-prob backward");
        set_error("");
        return HARTS_OK;
    }
    const BwdPlan b = plan_bwd(f.C, f.V, f.D, f.S, a->piece);
    if (!f.workspace || f.workspace_bytes < b.total) { set_error("workspace too small"); return HARTS_ESMALLBUF; }
    if (reinterpret_cast<uintptr_t>(f.workspace) & 255) { set_error("workspace must be 256-B aligned"); return HARTS_EINVAL; }
    uint8_t *ws = static_cast<uint8_t *>(f.workspace);
    void *dz = ws + b.dz;
    float *acc = reinterpret_cast<float *>(ws + b.dx);

    SemParams s = sem_params(&f);
    s.dlogp = a->dlogp;
    s.rows = reinterpret_cast<RowInfo *>(ws + b.rows);
    s.ent_y = reinterpret_cast<int32_t *>(ws + b.ent_y);
    s.ent_v = reinterpret_cast<float *>(ws + b.ent_v);
    s.raw_y = reinterpret_cast<int32_t *>(ws + b.raw_y);
    s.raw_v = reinterpret_cast<float *>(ws + b.raw_v);
    const bool pad = pads_x(f.C, f.D, true), copies = pad || b.twin;
    const PadParams copy{s.x, reinterpret_cast<__nv_bfloat16 *>(ws + b.pad), f.C, b.dz_rows, f.D, b.twin ? kTwin : 0};
    const int64_t row_blocks = ceil_div(f.C, kRowWarps);
    const cudaError_t first = launch(head_rows_kernel, row_blocks + (copies ? pad_blocks(b.dz_rows, f.D) : 0), 32 * kRowWarps, 0, 1,
                                     false, st, s, copy, static_cast<uint32_t>(row_blocks));
    if (first != cudaSuccess) return cuda_fail(first, "linear log-prob backward launch");

    const int G = b.group;
    const int32_t mt = ceil_div(f.C, kTM * G), C = static_cast<int32_t>(f.C);
    const int32_t a_rows = static_cast<int32_t>(std::min<int64_t>(kTM, (f.C + 7) / 8 * 8));
    const int32_t dz_box = b.twin ? 2 * kTwin : a_rows;
    int32_t *error = f.error ? f.error : own_error_word();
    if (!error) { set_error("the library's error word is not to be had"); return HARTS_ECUDA; }
    Params pz, pg;
    std::memset(&pz, 0, sizeof(pz));
    std::memset(&pg, 0, sizeof(pg));
    Prod &z = pz.prod[0], &gx = pg.prod[0], &gw = pg.prod[1];
    void *xp = ws + b.pad;
    bool ok = (pad ? map_panels(&z.a, xp, f.C, f.D, a_rows, 1) : map_in(&z.a, f.x, f.C, f.D, f.D, a_rows)) && map_in(&z.b, f.weight, f.V, f.D, f.D, b.n_dz / G) &&
              map_cols(&gx.b, &gx.b_edge, f.weight, f.V, f.D, b.n_grad / G) &&
              (copies ? map_panels(&gw.b, xp, b.dz_rows, f.D, 64, b.n_grad / G / 64)
                   : map_cols(&gw.b, &gw.b_edge, f.x, f.C, f.D, b.n_grad / G)) &&
              map_out(&gw.out, a->dweight, 1, f.V, f.D, f.D, false) &&
              (b.acc ? map_out(&gx.out, acc, b.splits, b.dz_rows, f.D, f.D, true) : map_out(&gx.out, a->dx, 1, f.C, f.D, f.D, false));
    for (int32_t i = 0; ok && i < b.n_pieces; ++i) {
        const int32_t v0 = i * b.piece, nv = std::min(b.piece, f.V - v0);
        ok = map_panels(&z.out, dz, b.dz_rows, nv, kTM, 1) && map_panels(&gx.a, dz, b.dz_rows, nv, dz_box, 1) &&
             map_panels(&gw.a, dz, b.dz_rows, nv, 64, 2);
        if (!ok) break;
        // logits of the piece, as dz
        z.m_tiles = mt; z.n = b.n_dz; z.n_tiles = ceil_div(nv, b.n_dz); z.splits = 1;
        z.k_blocks = z.k_per = ceil_div(f.D, kTK);
        z.a_panel = pad; z.a_rows = a_rows; z.b_y0 = v0; z.out_y0 = 0; z.rows = C; z.cols = nv;
        pz.n_prod = 1; pz.error = error; pz.c2 = logit_factor(f.scale, f.D);
        pz.rows = s.rows; pz.ent_y = s.ent_y; pz.ent_v = s.ent_v; pz.v0 = v0; pz.twin = b.twin;
        cudaError_t e = launch_tiles<kDz>(pz, G, true, st);
        if (e != cudaSuccess) return cuda_fail(e, "linear log-prob backward launch");
        // dX (first: its tiles are the longest) and dW
        gx.b_mn = 1; gx.a_panel = gw.a_panel = 1; gx.b_whole = f.D % 64 ? f.D / 64 * 64 : INT32_MAX;
        gw.b_whole = copies ? INT32_MAX : gx.b_whole; gx.a_rows = dz_box; gx.m_tiles = mt; gx.n = b.n_grad; gx.n_tiles = ceil_div(f.D, b.n_grad);
        gx.k_blocks = ceil_div(nv, kTK); gx.k_per = b.k_per; gx.splits = ceil_div(gx.k_blocks, b.k_per);
        gx.b_y0 = v0; gx.out_y0 = 0; gx.rows = b.dz_rows; gx.cols = f.D; gx.out_f32 = b.acc; gx.out_add = i > 0;
        gw.a_mn = gw.b_mn = 1; gw.m_tiles = ceil_div(nv, kTM * G); gw.n = b.n_grad; gw.n_tiles = ceil_div(f.D, b.n_grad);
        gw.k_blocks = gw.k_per = ceil_div(b.dz_rows, kTK); gw.splits = 1;
        gw.out_y0 = v0; gw.rows = nv; gw.cols = f.D; gw.fast_n = 1;
        pg.n_prod = 2; pg.error = error;
        e = launch_tiles<kGrad>(pg, G, true, st);
        if (e != cudaSuccess) return cuda_fail(e, "linear log-prob backward launch");
    }
    if (!ok) { set_error("tensor map"); return HARTS_ECUDA; }
    if (b.acc) {
        const DxParams d{acc, static_cast<__nv_bfloat16 *>(a->dx), f.C * f.D, int64_t(b.dz_rows) * f.D,
                         b.twin ? int64_t(kTwin) * f.D : 0, b.splits};
        const int64_t blocks = std::min<int64_t>((d.n / 4 + 127) / 128, int64_t(sm_count()) * 16);
        const cudaError_t e = launch(head_dx_kernel, blocks, 128, 0, 1, true, st, d);
        if (e != cudaSuccess) return cuda_fail(e, "linear log-prob backward launch");
    }
    set_error("");
    return HARTS_OK;
}

}  // extern "C"
