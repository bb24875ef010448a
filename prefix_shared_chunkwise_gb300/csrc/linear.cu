// Matrix product with bias, activation and residual in its epilogue, and its gradients.
//
//   z = x w^T + b,   y = act(z) + residual          x [C][K], w [N][K], z, y [C][N]
//   dz = dy act'(z),  dx = dz w,  dw = dz^T x,  db = sum_rows dz
// act: identity, silu z sigmoid(z), or gelu z Phi(z) with the normal distribution's Phi.
//
// Forward: one product whose 128 x n tiles get bias, activation and residual between tensor memory
// and the store; z is kept beside y where the gradient will want it.  Backward: one pass forms dz in
// bf16 (the tensor cores' operands are bf16; each entry is formed in fp32 and rounded once) and the
// bias gradient from the unrounded values; then dx and dw in one launch, reading dz, w and x as
// they lie, by rows or by columns.  All sums are fp32 and in a fixed order.  dz's rounding leaves dx and dw 1.4
// times as far from the gradient, in norm, as their own alone would (2.35e-3 against 1.65e-3); a second bf16 term
// for what it takes would double the products.
//
// Tile kernel: persistent blocks, one per SM, in pairs where there are rows for it (a pair shares
// a tile of 256 rows: each block holds half of its columns); warps 0 and 3 fill a ring of
// shared-memory stages with either operand by TMA, warp 1 issues tcgen05.mma into one of two
// 256-column accumulators in TMEM, warps 4-11 empty the other one, and two threads send the
// finished columns out.  Where there are fewer tiles than SMs, the sum is cut into pieces, whose
// fp32 results a small kernel joins in order before the epilogue.  For one row or two, where
// reading w is all, warps form dot products instead.  All waits are bounded.
//
// The products bound many rows, and under the power limit their energy.  16,384 x 2,048 -> 8,192 in short runs: the product
// alone 282 us (1.95 PFLOP/s), gelu 292, bias and residual 303, gelu with z kept 309; back to back that last one takes
// 361 at 1.5 GHz, where a library's product alone takes 318.  Both gradients 596 - 620 us, with dz and db 766.  777 x 2,760 ->
// 1,032 with bias and residual: 49 K cycles from cold caches, of which the products of 24 tiles on 48 SMs are 20 K.  One
// row of 8,192 x 2,048: 3.7 us.  Few rows are far from reading the weight: 2,048 -> 8,192 with gelu and z, one call behind
// another, 3 rows 10.7 us, 48 15.4, 300 20.9, 777 29.7, the gradients 23.6, 23.4, 41 and 58 (floors 5.0, 5.2, 6.6, 13.7; 9.9,
// 10.2, 11.7, 27): a stage of the ring is laid out for whole tiles, whatever fills it, and pieces of a sum cost a launch.
#include <algorithm>
#include <cmath>
#include <cstring>
#include <type_traits>

#include "kda_common.cuh"
#include "launch_util.h"
#include "tc_primitives.cuh"
#include "tensor_map.h"
#include "tile_order.h"
#include "tile_pairs.cuh"
#include "two.cuh"

namespace harts {
namespace {

using namespace pairs;
using namespace two;

constexpr int kTM = 128, kTK = 64, kTN = 256;       // a block's tile rows, K step (one 128-byte swizzle row), tile columns
constexpr uint32_t kABytes = kTM * kTK * 2;
constexpr uint32_t kSlots = 4, kSlotBytes = kTM * 64;           // 128 rows x 64 bytes of output on their way out
constexpr int kThreads = 448, kEpiWarp0 = 4, kStoreWarp0 = 12;  // eight epilogue warps: two for each 32 TMEM lanes
constexpr int kDotRows = 2;                         // most rows that are done by dot products

// As many stages as fit beside small slots: copies are some 2,500 cycles on their way while results go out, five steps
// of a pair.  (8,192 x 2,048 x 8,192, cycles, plain / gelu and z: six stages and slots of 8 KB 259 K / 276 K, five and
// slots of 16 KB 271 K / 311 K, four 305 K / 339 K; 229 K are the products alone.)
template <int G> struct Ring {
    static constexpr uint32_t stages = G == 2 ? 6 : 4;
    static constexpr uint32_t stage_bytes = kABytes + kTN / G * kTK * 2;
    static constexpr uint32_t smem = stages * stage_bytes + kSlots * kSlotBytes + 1024;
    static_assert(smem <= 227 * 1024 - 512, "shared memory of an SM");
    // barriers
    static constexpr uint32_t full = 0, empty = stages, acc_full = 2 * stages, acc_empty = acc_full + 2, drain = acc_empty + 2,
                              out_full = drain + 1, out_free = out_full + kSlots, count = out_free + kSlots;
};

// One product D = A B^T cut into tiles and pieces of its sum.  An operand is stored [rows][sum]
// or, read by columns, [sum][rows].
struct Prod {
    CUtensorMap a, b, out, keep;    // keep: z
    CUtensorMap a_edge, b_edge;     // the last columns of an operand read by columns, where they do not fill a panel of 64
    int32_t a_mn, b_mn;             // read by columns
    int32_t a_whole, b_whole;       // columns in whole panels
    int32_t a_rows;                 // rows of A's box when read by rows
    int32_t m_tiles, n_tiles, splits, n;
    uint32_t items, per_split;
    int32_t k_blocks, k_per;        // steps of 64 in all, per piece
    int32_t rows, cols;             // of the output
    int32_t fast_n;                 // tiles that run together share A (walk n first) instead of B
    int32_t out_f32;                // a piece's sums
};

struct Epilogue {
    const float *bias;
    const __nv_bfloat16 *res;
};

struct Params {
    Prod prod[2];
    int32_t n_prod;
    uint32_t each0, over, extra;    // see tile_at
    int32_t *error;
    Epilogue ep;
    int32_t keep;                   // z goes out too
};

// ---- activations ------------------------------------------------------------------------

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ Two both(float c) { return make_float2(c, c); }

// Phi(z) and the density at z, up to a factor.  With x = |z| / sqrt 2, Phi(-|z|) = e^(-x^2) E(x) / 2
// where E(x) = e^(x^2) erfc(x) is smooth: t P(t), t = 1 / (1 + 3/8 x), P of degree 6 fitted to it over
// 0 .. 10 with least relative error (6.4e-7, against bf16's 2^-9).  One exponential serves both, and
// the far tail keeps its digits.
__device__ __forceinline__ Two normal(Two z, Two &density) {
    const Two t = each(z, [](float v) { return rcp(fmaf(fabsf(v), 0.375f * 0.70710678f, 1.f)); });
    density = each(mul(z, z), [](float v) { return ex2(v * -0.72134752f); });
    Two q = both(-0.13509675f);
    q = fma(q, t, both(0.38794115f));
    q = fma(q, t, both(-0.12960255f));
    q = fma(q, t, both(0.28306571f));
    q = fma(q, t, both(0.16666285f));
    q = fma(q, t, both(0.21568952f));
    q = fma(q, t, both(0.21133942f));
    const Two tail = mul(mul(density, both(0.5f)), mul(q, t));
    return each(z, tail, [](float v, float a) { return v < 0.f ? a : 1.f - a; });
}
__device__ __forceinline__ Two sigmoid(Two z) { return each(z, [](float v) { return rcp(1.f + ex2(v * -1.44269504f)); }); }
template <int ACT> __device__ __forceinline__ Two act_of(Two z) {
    if constexpr (ACT == HARTS_ACT_SILU) return mul(z, sigmoid(z));
    if constexpr (ACT == HARTS_ACT_GELU) {
        Two density;
        return mul(z, normal(z, density));
    }
    return z;
}
template <int ACT> __device__ __forceinline__ Two slope_of(Two z) {
    if constexpr (ACT == HARTS_ACT_SILU) {
        const Two q = sigmoid(z);
        return mul(q, fma(z, fma(q, both(-1.f), both(1.f)), both(1.f)));
    }
    if constexpr (ACT == HARTS_ACT_GELU) {
        Two density;
        const Two phi = normal(z, density);
        return fma(mul(z, both(0.39894228f)), density, phi);
    }
    return both(1.f);
}
__device__ __forceinline__ Two open(uint32_t u) { return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u)); }

// Eight columns of one row, with their bias and residual: z and y.  Columns come in eights.
struct Eight { Two v[4]; };
struct Bias8 { float4 a, b; };
__device__ __forceinline__ Bias8 bias_of(const float *bias, int32_t col) {
    return {__ldg(reinterpret_cast<const float4 *>(bias + col)), __ldg(reinterpret_cast<const float4 *>(bias + col) + 1)};
}
template <int ACT> __device__ __forceinline__ void finish8(const Bias8 &b, const uint4 &res, Eight &z, Eight &y) {
    z.v[0] = add(z.v[0], make_float2(b.a.x, b.a.y)); z.v[1] = add(z.v[1], make_float2(b.a.z, b.a.w));
    z.v[2] = add(z.v[2], make_float2(b.b.x, b.b.y)); z.v[3] = add(z.v[3], make_float2(b.b.z, b.b.w));
    const uint32_t *u = &res.x;
#pragma unroll
    for (int i = 0; i < 4; ++i) y.v[i] = add(act_of<ACT>(z.v[i]), open(u[i]));
}
__device__ __forceinline__ uint4 pack8(const Eight &e) {
    return make_uint4(tc::pack_bf16(e.v[0].x, e.v[0].y), tc::pack_bf16(e.v[1].x, e.v[1].y), tc::pack_bf16(e.v[2].x, e.v[2].y), tc::pack_bf16(e.v[3].x, e.v[3].y));
}

// ---- tiles ------------------------------------------------------------------------------

// ACT >= 0: bias, that activation and residual go into the output; otherwise it is the product, or a piece of it.
template <int ACT, int G>
__global__ void __launch_bounds__(kThreads, 1) linear_tile_kernel(const __grid_constant__ Params p) {
    using B = Ring<G>;
    constexpr bool FWD = ACT >= 0;
    constexpr uint32_t kStages = B::stages, kStageBytes = B::stage_bytes;
    extern __shared__ uint8_t smraw[];
    uint8_t *sm = smraw + ((1024 - (tc::smem_addr(smraw) & 1023)) & 1023);
    __shared__ uint64_t bars[B::count];
    __shared__ uint32_t s_tmem;
    __shared__ int s_fail;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = G == 2 ? static_cast<int>(cluster_rank()) : 0;
    const uint32_t worker = blockIdx.x / G, workers = gridDim.x / G;

    if (tid == 0) {
        for (uint32_t i = 0; i < kStages; ++i) { tc::mbar_init(&bars[B::full + i], 2); tc::mbar_init(&bars[B::empty + i], 1); }
        for (int i = 0; i < 2; ++i) { tc::mbar_init(&bars[B::acc_full + i], 1); tc::mbar_init(&bars[B::acc_empty + i], 8 * G); }
        for (uint32_t i = 0; i < kSlots; ++i) { tc::mbar_init(&bars[B::out_full + i], 4); tc::mbar_init(&bars[B::out_free + i], 1); }
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
    wait_previous();                                    // dz; bounded waits begin once the kernel before this one is done
    const uint32_t tm = s_tmem;

    if (warp == 0 || warp == 3) {
        // One warp each for A and B, whole like the issuing one: a lone thread, or one warp for both
        // operands, does not keep up with the 512 cycles of a step's products.
        const bool is_b = warp == 3;
        const uint32_t on = elect_lane(), arms = rank == 0 ? on : 0;
        uint32_t it = 0, s = 0, round = 0;              // stages filled; next stage, times the ring went round
        const uint32_t own0 = tc::smem_addr(&bars[B::full]), full0 = G == 2 ? leader_addr(&bars[B::full]) : own0;
        const uint32_t dst0 = tc::smem_addr(sm) + (is_b ? kABytes : 0);
        TileId t;
        bool ok = true;
        for (uint32_t n = 0; ok && tile_at(p, n, worker, workers, t); ++n) {
            const Prod &q = p.prod[t.which];
            const int32_t k0 = t.split * q.k_per, k1 = min(q.k_blocks, k0 + q.k_per);
            const int32_t nb = is_b ? q.n / G : kTM;    // rows of the operand that this block holds
            const int32_t r0 = is_b ? t.nt * q.n + rank * nb : (t.mt * G + rank) * kTM;
            const bool mn = is_b ? q.b_mn : q.a_mn;
            enum { kRows, kPanels, kBoxes };
            const int how = !mn ? kRows : r0 + nb <= (is_b ? q.b_whole : q.a_whole) ? kPanels : kBoxes;
            const CUtensorMap *map = is_b ? (how == kBoxes ? &q.b_edge : &q.b) : (how == kBoxes ? &q.a_edge : &q.a);
            const uint32_t bytes = (is_b || mn ? nb * 128u : q.a_rows * 128u) * G;
            for (int32_t k = k0; k < k1; ++k, ++it) {
                if (round > 0 && !warp_wait(&bars[B::empty + s], (round - 1) & 1, &s_fail)) { ok = false; break; }
                const uint32_t full = full0 + s * 8, dst = dst0 + s * kStageBytes;
                expect(arms, own0 + s * 8, bytes);
                if (how == kRows) pair_load<G>(on, dst, map, k * kTK, r0, full);
                else if (how == kPanels) pair_load3<G>(on, dst, map, 0, k * kTK, r0 / 64, full);
                else for (int j = 0; j < nb; j += 64) pair_load<G>(on, dst + j * 128, map, r0 + j, k * kTK, full);
                if (++s == kStages) { s = 0; ++round; }
            }
        }
        // Nothing may be in flight into this block's shared memory when it ends: the copies (after
        // a failure the products may not have waited for them), then the stages' last release.
        // In a pair only the release says so for the second block; after a failure its wait runs
        // out, long after the last copy.
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
            for (; ok && tile_at(p, tile, worker, workers, t); ++tile) {
                const Prod &q = p.prod[t.which];
                const int32_t k0 = t.split * q.k_per, k1 = min(q.k_blocks, k0 + q.k_per);
                const uint32_t buf = tile & 1, use = tile >> 1, d = tm + buf * kTN;
                const uint32_t id = tc::idesc_bf16(kTM * G, q.n, q.a_mn != 0, q.b_mn != 0);
                // descriptors of stage 0; 16 columns of the sum lie 32 bytes apart in an operand stored
                // by rows and 2 KB apart in one read by columns (descriptors count 16 bytes)
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
        // 64 bytes of columns at a time, taken in turn by the two warps of 32 TMEM lanes; each of
        // the two has two of the slots, z before y where both go out
        const int lg = (warp - kEpiWarp0) & 3, half = (warp - kEpiWarp0) >> 2;
        const uint32_t lane_off = static_cast<uint32_t>(lg * 32) << 16;
        uint8_t *out = sm + kStages * kStageBytes + lg * 2048 + lane * 64;  // this lane's row of a slot
        const int swizzle = (lane >> 1) & 3;
        const uint32_t released = G == 2 ? leader_addr(&bars[B::acc_empty]) : 0;
        uint32_t tile = 0, groups = 0, q_out = 0;
        TileId t;
        bool ok = true;
        auto slot_for = [&](uint32_t &slot) {                   // the next of this half's slots, once it is free
            slot = half + 2 * (q_out & 1);
            const uint32_t use = q_out >> 1;
            ++q_out;
            return use == 0 || warp_wait(&bars[B::out_free + slot], (use - 1) & 1, &s_fail);
        };
        auto send = [&](uint32_t slot) {
            tc::fence_smem_to_async();
            __syncwarp();
            if (lane == 0) arrive(&bars[B::out_full + slot]);
        };
        for (; ok && tile_at(p, tile, worker, workers, t); ++tile) {
            const Prod &q = p.prod[t.which];
            const uint32_t buf = tile & 1;
            const uint32_t acc = tm + buf * kTN + lane_off;
            const int32_t n0 = t.nt * q.n, row = (t.mt * G + rank) * kTM + lg * 32 + lane;
            if constexpr (FWD) {
                // what the tile's end will read is brought near while its products are formed: each
                // lane's row of the residual to L2, the bias to L1
                if (p.ep.res && row < q.rows)
                    for (int c = half * 64; c < q.n && n0 + c < q.cols; c += 128)
                        asm volatile("prefetch.global.L2 [%0];" :: "l"(p.ep.res + static_cast<int64_t>(row) * q.cols + n0 + c));
                if (p.ep.bias && lane * 32 < q.n && n0 + lane * 32 < q.cols)
                    asm volatile("prefetch.global.L1 [%0];" :: "l"(p.ep.bias + n0 + lane * 32));
            }
            if (!warp_wait(&bars[B::acc_full + buf], (tile >> 1) & 1, &s_fail)) break;
            tc::fence_after_sync();
            const int step = !FWD && q.out_f32 ? 16 : 32, end = min(q.n, q.cols - n0);
            for (int c = 0; c < end; c += step, ++groups) {
                if ((groups & 1) != static_cast<uint32_t>(half)) continue;
                // The values first, then a slot for them: what the unit before it left there is on its way out
                // meanwhile.  A row's four 16 bytes are swizzled by its number in pairs.
                auto leave = [&](const uint4 (&w)[4]) {
                    uint32_t slot;
                    if (!slot_for(slot)) return false;
#pragma unroll
                    for (int j = 0; j < 4; ++j) *reinterpret_cast<uint4 *>(out + slot * kSlotBytes + ((j ^ swizzle) << 4)) = w[j];
                    send(slot);
                    return true;
                };
                if (!FWD && q.out_f32) {
                    float v[16];
                    tc::tmem_ld16(acc + c, v);
                    ok = leave(reinterpret_cast<const uint4(&)[4]>(v));
                } else {
                    const int32_t col = n0 + c;
                    uint4 r[4] = {};
                    Bias8 b[4] = {};
                    if constexpr (FWD) {                        // on their way together, and ahead of the accumulator
                        if (p.ep.res && row < q.rows) {
                            const __nv_bfloat16 *res = p.ep.res + static_cast<int64_t>(row) * q.cols;
#pragma unroll
                            for (int j = 0; j < 4; ++j) r[j] = *reinterpret_cast<const uint4 *>(res + min(col + 8 * j, q.cols - 8));
                        }
                        if (p.ep.bias) {
#pragma unroll
                            for (int j = 0; j < 4; ++j) b[j] = bias_of(p.ep.bias, min(col + 8 * j, q.cols - 8));
                        }
                    }
                    float v[32];
                    tc::tmem_ld32(acc + c, v);
                    uint4 zs[4], ys[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        Eight z, y;
#pragma unroll
                        for (int i = 0; i < 4; ++i) z.v[i] = make_float2(v[8 * j + 2 * i], v[8 * j + 2 * i + 1]);
                        if constexpr (FWD) {
                            finish8<ACT>(b[j], r[j], z, y);
                            zs[j] = pack8(z);
                            ys[j] = pack8(y);
                        } else {
                            ys[j] = pack8(z);
                        }
                    }
                    ok = (!FWD || !p.keep || leave(zs)) && leave(ys);
                }
                if (!ok) break;
            }
            tc::fence_before_sync();                    // the accumulator has been read
            __syncwarp();
            if (lane == 0) {
                if (G == 2) arrive_at(released + buf * 8); else arrive(&bars[B::acc_empty + buf]);
            }
        }
    } else if (warp >= kStoreWarp0) {
        // Two threads send the slots of a half each: a store takes its thread a few hundred cycles, which the
        // warps that fill the slots need not wait for.  A slot is given back behind the next store; z's and y's
        // together (one behind the other keeps the next z waiting: 276 K cycles to 291 K for 8,192 x 2,048 x 8,192 with gelu).
        if (lane == 0) {
            const uint32_t mine = warp - kStoreWarp0;
            uint32_t groups = 0, q_out = 0;
            TileId t;
            bool ok = true;
            for (uint32_t n = 0; ok && tile_at(p, n, worker, workers, t); ++n) {
                const Prod &q = p.prod[t.which];
                const int32_t n0 = t.nt * q.n, y = (t.mt * G + rank) * kTM;
                const int step = !FWD && q.out_f32 ? 16 : 32, end = min(q.n, q.cols - n0);
                for (int c = 0; ok && c < end; c += step, ++groups) {
                    if ((groups & 1) != mine) continue;
                    for (int k = FWD && p.keep ? 0 : 1; k < 2; ++k) {
                        const uint32_t slot = mine + 2 * (q_out & 1), use = q_out >> 1;
                        const uint8_t *src = sm + kStages * kStageBytes + slot * kSlotBytes;
                        if (!wait_or_fail(&bars[B::out_full + slot], use & 1, &s_fail)) { ok = false; break; }
                        if (y < q.rows) store_3d(k == 0 ? &q.keep : &q.out, n0 + c, y, t.split, src, false);
                        tc::bulk_commit();
                        ++q_out;
                        if (FWD && p.keep) {            // z's and y's given back at once
                            if (k == 0) continue;
                            tc::bulk_wait_read();
                            arrive(&bars[B::out_free + mine]);
                            arrive(&bars[B::out_free + mine + 2]);
                        } else {
                            store_wait_read1();
                            if (q_out > 1) arrive(&bars[B::out_free + mine + 2 * (q_out & 1)]);
                        }
                    }
                }
            }
            tc::bulk_wait_all();
        }
    }
    tc::fence_before_sync();
    __syncthreads();
    if (tid == 0 && failed(&s_fail)) atomicCAS(p.error, 0, static_cast<int>(kDevErrTimeout));
    if (G == 2) cluster_sync();                         // neither block ends under the other's copies or arrivals
    tc::fence_after_sync();
    if (warp == 2) pair_dealloc<G>(tm);
}

// ---- pieces joined ----------------------------------------------------------------------

// Eight columns a thread: the pieces of up to two outputs in order, then the epilogue.
struct JoinOne { const float *part; __nv_bfloat16 *y, *z; int64_t values; int32_t cols, splits; };
struct Join { JoinOne of[2]; Epilogue ep; int64_t blocks0; };
template <int ACT>
__global__ void __launch_bounds__(128) linear_join_kernel(const Join p) {
    wait_previous();
    const int which = blockIdx.x >= p.blocks0;
    const JoinOne &o = p.of[which];
    const int64_t at = ((blockIdx.x - (which ? p.blocks0 : 0)) * 128 + threadIdx.x) * 8;
    if (at >= o.values) return;
    Eight z, y;
#pragma unroll
    for (int i = 0; i < 4; ++i) z.v[i] = both(0.f);
#pragma unroll 4
    for (int s = 0; s < o.splits; ++s) {
        const float4 *q = reinterpret_cast<const float4 *>(o.part + s * o.values + at);
        const float4 a = q[0], b = q[1];
        z.v[0] = add(z.v[0], make_float2(a.x, a.y)); z.v[1] = add(z.v[1], make_float2(a.z, a.w));
        z.v[2] = add(z.v[2], make_float2(b.x, b.y)); z.v[3] = add(z.v[3], make_float2(b.z, b.w));
    }
    uint4 r = make_uint4(0, 0, 0, 0);
    if (p.ep.res) r = *reinterpret_cast<const uint4 *>(p.ep.res + at);
    Bias8 b{};
    if (p.ep.bias) b = bias_of(p.ep.bias, static_cast<int32_t>(at % o.cols));
    finish8<ACT>(b, r, z, y);
    if (o.z) *reinterpret_cast<uint4 *>(o.z + at) = pack8(z);
    *reinterpret_cast<uint4 *>(o.y + at) = pack8(y);
}

// ---- few rows ---------------------------------------------------------------------------

// Dot products of R rows with a warp's two rows of w; x comes from L1.  (8,192 x 2,048 from L2: one row 4.2 us, two
// 6.2, three 10.6, where the tiles take 9.7.)
struct DotParams { const __nv_bfloat16 *x, *w; __nv_bfloat16 *y, *z; Epilogue ep; int32_t K, N; };
template <int R, int ACT>
__global__ void __launch_bounds__(256) linear_dot_kernel(const DotParams p) {
    const int lane = threadIdx.x & 31;
    const int32_t n0 = (blockIdx.x * 8 + (threadIdx.x >> 5)) * 2;
    if (n0 >= p.N) return;
    const uint4 *w0 = reinterpret_cast<const uint4 *>(p.w + static_cast<int64_t>(n0) * p.K), *w1 = w0 + p.K / 8;   // N is even
    Two acc[2][R];
#pragma unroll
    for (int r = 0; r < R; ++r) acc[0][r] = acc[1][r] = both(0.f);
    const int32_t chunks = p.K / 8;
    auto take = [&](const uint4 &a, const uint4 &b, int32_t i) {
        const uint32_t *ua = &a.x, *ub = &b.x;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const uint4 x = __ldg(reinterpret_cast<const uint4 *>(p.x + static_cast<int64_t>(r) * p.K) + i);
            const uint32_t *ux = &x.x;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                acc[0][r] = fma(open(ua[k]), open(ux[k]), acc[0][r]);
                acc[1][r] = fma(open(ub[k]), open(ux[k]), acc[1][r]);
            }
        }
    };
    constexpr int kAtOnce = 4;
    int32_t i = lane;
    for (; i + 32 * (kAtOnce - 1) < chunks; i += 32 * kAtOnce) {
        uint4 a[kAtOnce], b[kAtOnce];
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) { a[j] = __ldg(w0 + i + 32 * j); b[j] = __ldg(w1 + i + 32 * j); }
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) take(a[j], b[j], i + 32 * j);
    }
    for (; i < chunks; i += 32) take(__ldg(w0 + i), __ldg(w1 + i), i);
    float mine = 0.f;                                   // lane 2 r + c: row r, column c
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int r = 0; r < R; ++r) {
            float v = total(acc[c][r]);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
            if (lane == 2 * r + c) mine = v;
        }
    if (lane >= 2 * R) return;
    const int32_t col = n0 + (lane & 1);
    const int64_t at = static_cast<int64_t>(lane >> 1) * p.N + col;
    if (p.ep.bias) mine += __ldg(p.ep.bias + col);
    const float res = p.ep.res ? __bfloat162float(p.ep.res[at]) : 0.f;      // before z, which may be written over it
    if (p.z) p.z[at] = __float2bfloat16_rn(mine);
    p.y[at] = __float2bfloat16_rn(act_of<ACT>(both(mine)).x + res);
}

// ---- dz and the bias gradient -----------------------------------------------------------

// A block takes 256 columns, eight a thread, of `per` rows; its eight warps' column sums are added
// in order and leave one row of sums, which the second kernel adds in order.
struct DzParams { const __nv_bfloat16 *dy, *z; __nv_bfloat16 *dz; float *part; int64_t C; int32_t N, per; };
template <int ACT>
__global__ void __launch_bounds__(256) linear_dz_kernel(const DzParams p) {
    constexpr bool kCurved = ACT != HARTS_ACT_NONE;
    constexpr int kAtOnce = 4;                          // rows that a warp loads at a time
    __shared__ float sm[8][256];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int32_t strips = (p.N + 255) / 256, strip = blockIdx.x % strips, chunk = blockIdx.x / strips;
    const int32_t col = strip * 256 + lane * 8;
    let_next_start();
    Eight s;
#pragma unroll
    for (int k = 0; k < 4; ++k) s.v[k] = both(0.f);
    if (col < p.N) {
        const int64_t r0 = static_cast<int64_t>(chunk) * p.per + warp, r1 = min(p.C, static_cast<int64_t>(chunk + 1) * p.per);
        for (int64_t r = r0; r < r1; r += 8 * kAtOnce) {
            uint4 u[kAtOnce], v[kAtOnce];
#pragma unroll
            for (int j = 0; j < kAtOnce; ++j) {
                if (r + 8 * j >= r1) continue;
                const int64_t at = (r + 8 * j) * p.N + col;
                u[j] = __ldg(reinterpret_cast<const uint4 *>(p.dy + at));
                if (kCurved) v[j] = __ldg(reinterpret_cast<const uint4 *>(p.z + at));
            }
#pragma unroll
            for (int j = 0; j < kAtOnce; ++j) {
                if (r + 8 * j >= r1) continue;
                const uint32_t *pu = &u[j].x, *pv = &v[j].x;
                Eight d;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    d.v[k] = open(pu[k]);
                    if (kCurved) d.v[k] = mul(d.v[k], slope_of<ACT>(open(pv[k])));
                    s.v[k] = add(s.v[k], d.v[k]);
                }
                if (kCurved) *reinterpret_cast<uint4 *>(p.dz + (r + 8 * j) * p.N + col) = pack8(d);
            }
        }
    }
    if (!p.part) return;
#pragma unroll
    for (int k = 0; k < 4; ++k) { sm[warp][lane * 8 + 2 * k] = s.v[k].x; sm[warp][lane * 8 + 2 * k + 1] = s.v[k].y; }
    __syncthreads();
    const int32_t c = strip * 256 + threadIdx.x;
    if (c < p.N) {
        float v = sm[0][threadIdx.x];
#pragma unroll
        for (int w = 1; w < 8; ++w) v += sm[w][threadIdx.x];
        p.part[static_cast<int64_t>(chunk) * p.N + c] = v;
    }
}
struct DbParams { const float *part; float *db; int32_t N, chunks; };
__global__ void __launch_bounds__(1024) linear_db_kernel(const DbParams p) {
    __shared__ float sm[32][33];
    let_next_start();
    wait_previous();
    const int lane = threadIdx.x & 31, k = threadIdx.x >> 5;
    const int32_t col = blockIdx.x * 32 + lane;
    float s = 0.f;
    if (col < p.N) {
#pragma unroll 4
        for (int32_t g = k; g < p.chunks; g += 32) s += p.part[static_cast<int64_t>(g) * p.N + col];
    }
    sm[k][lane] = s;
    __syncthreads();
    if (k == 0 && col < p.N) {
#pragma unroll
        for (int i = 1; i < 32; ++i) s += sm[i][lane];
        p.db[col] = s;
    }
}

// ---- host ---------------------------------------------------------------------------------

size_t align256(size_t x) { return (x + 255) / 256 * 256; }

// How a product is cut.
struct Cut { int G; int32_t n, splits, k_per; };

// Blocks that share a tile, its width and the pieces of the sum, by the time of the busiest worker:
// a step of 64 takes two cycles a column, no less than its copies and barriers (430 - 450), and in
// single blocks 1.2 as long, as each reads its columns alone; a tile's ends cost about three steps.
// An operand read by columns comes in 64s per block.
// Pieces cost their fp32 sums, written and read again at some 3,500 bytes a cycle, a launch, and the caller a
// workspace.
Cut cut_of(int64_t M, int64_t N, int32_t kb, bool by_columns, int32_t outputs, int groups = 2) {
    Cut best{1, kTN, 1, kb};
    double least = 0.0;
    for (int G = 1; G <= (M > kTM ? groups : 1); ++G)
        for (int32_t n = kTN; n >= 64; n -= by_columns ? 64 * G : 64) {
            const int64_t tiles = int64_t(ceil_div(M, kTM * G)) * ceil_div(N, n), workers = sm_count() / G;
            const int32_t most = static_cast<int32_t>(std::max<int64_t>(1, std::min<int64_t>({(2 * workers + tiles - 1) / tiles, kb / 4, 32})));
            for (int32_t s = 1; s <= most; ++s) {
                const int32_t per = ceil_div(kb, s), used = ceil_div(kb, per);
                if (used != s) continue;
                const double step = 2.0 * std::max(n, 220) * (G == 1 ? 1.2 : 1.0);
                double cost = double((tiles * s + workers - 1) / workers) * (per + 3) * step;
                if (s > 1) cost += 9000.0 + double(M) * N * (8 * s + 2 * outputs) / 3500.0;
                if (least == 0.0 || cost < least) { least = cost; best = Cut{G, n, s, per}; }
            }
        }
    return best;
}

// [rows][cols] bf16, read in boxes of 64 columns x box_rows.
bool map_in(CUtensorMap *m, const void *base, int64_t rows, int64_t cols, int32_t box_rows) {
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(cols) * 2};
    const cuuint32_t box[2] = {64, static_cast<cuuint32_t>(box_rows)};
    return encode_bf16(m, base, 2, dims, strides, box);
}

// The same read as columns, in boxes of 64 rows x `cols` columns: those that fill panels of 64 as
// panels, so that one copy brings a tile's; the others (the panel they lie in would reach past the
// last row's end) in boxes of 64 through `edge`.
bool map_cols(CUtensorMap *m, CUtensorMap *edge, const void *base, int64_t rows, int64_t D, int32_t cols) {
    if (!map_in(edge, base, rows, D, 64)) return false;
    if (D < 64) { *m = *edge; return true; }            // no whole panel; a map is fetched all the same
    const cuuint64_t dims[3] = {64, static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(D / 64)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(D) * 2, 128};
    const cuuint32_t box[3] = {64, 64, static_cast<cuuint32_t>(cols / 64)};
    return encode_bf16(m, base, 3, dims, strides, box);
}

// [layers][rows][cols], written in boxes of 64 bytes x 128 rows.
bool map_out(CUtensorMap *m, void *base, int64_t layers, int64_t rows, int64_t cols, bool f32) {
    const cuuint64_t e = f32 ? 4 : 2;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(layers)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(cols) * e, static_cast<cuuint64_t>(cols) * e * rows};
    const cuuint32_t box[3] = {f32 ? 16u : 32u, kTM, 1};
    const cuuint32_t es[3] = {1, 1, 1};
    auto fn = encode_tiled();
    return fn && fn(m, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, base, dims, strides,
                    box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B,
                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// D [M][N] = A B^T with the sum over S; A is M x S, B N x S, either read by columns where `mn`.
bool make_prod(Prod &q, const Cut &c, int64_t M, int64_t N, int64_t S, const void *a, bool a_mn, const void *b, bool b_mn, void *out,
               float *part) {
    q.a_mn = a_mn; q.b_mn = b_mn;
    q.a_whole = static_cast<int32_t>(M / 64 * 64); q.b_whole = static_cast<int32_t>(N / 64 * 64);
    q.a_rows = static_cast<int32_t>(std::min<int64_t>(kTM, (M + 7) / 8 * 8));
    q.m_tiles = ceil_div(M, kTM * c.G); q.n_tiles = ceil_div(N, c.n); q.splits = c.splits; q.n = c.n;
    q.k_blocks = ceil_div(S, kTK); q.k_per = c.k_per;
    q.rows = static_cast<int32_t>(M); q.cols = static_cast<int32_t>(N);
    q.fast_n = q.n_tiles <= q.m_tiles;
    q.out_f32 = part != nullptr;
    return (a_mn ? map_cols(&q.a, &q.a_edge, a, S, M, kTM) : map_in(&q.a, a, M, S, q.a_rows)) &&
           (b_mn ? map_cols(&q.b, &q.b_edge, b, S, N, c.n / c.G) : map_in(&q.b, b, N, S, c.n / c.G)) &&
           map_out(&q.out, part ? static_cast<void *>(part) : out, part ? c.splits : 1, M, N, part != nullptr);
}

template <int ACT, int G>
cudaError_t launch_group(Params &p, bool behind, cudaStream_t st) {
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = allow_smem(linear_tile_kernel<ACT, G>, Ring<G>::smem, done);
    if (e != cudaSuccess) return e;
    const uint32_t workers = share_tiles(p, sm_count() / G);
    return launch(linear_tile_kernel<ACT, G>, int64_t(workers) * G, kThreads, Ring<G>::smem, G, behind, st, p);
}
template <int ACT> cudaError_t launch_tiles(Params &p, int G, bool behind, cudaStream_t st) {
    return G == 2 ? launch_group<ACT, 2>(p, behind, st) : launch_group<ACT, 1>(p, behind, st);
}

// Calls f with the activation as a constant.
template <typename F> cudaError_t with_act(int32_t act, F &&f) {
    if (act == HARTS_ACT_SILU) return f(std::integral_constant<int, HARTS_ACT_SILU>{});
    if (act == HARTS_ACT_GELU) return f(std::integral_constant<int, HARTS_ACT_GELU>{});
    return f(std::integral_constant<int, HARTS_ACT_NONE>{});
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

int cuda_fail(cudaError_t e, const char *what) {
    set_error(std::string(what) + ": " + cudaGetErrorString(e));
    return HARTS_ECUDA;
}

bool sizes_ok(int64_t C, int32_t K, int32_t N) {
    return C >= 0 && K >= 8 && N >= 8 && K % 8 == 0 && N % 8 == 0 && C <= 0x7fffff00 && K <= 0x7fffff00 && N <= 0x7fffff00 &&
           (C / kTM + 1) * (N / 64 + 1) <= 0xffffff && (C / kTM + 1) * (K / 64 + 1) <= 0xffffff && (int64_t(K) / 64 + 1) * (N / 64 + 1) <= 0xffffff;
}

int check(const harts_linear_args *a) {
    if (!a) { set_error("NULL args"); return HARTS_EINVAL; }
    if (a->dtype != HARTS_BF16) { set_error("x, weight, residual and outputs must be bf16"); return HARTS_EUNSUPPORTED; }
    if (a->C < 0 || a->K < 1 || a->N < 1) { set_error("C >= 0 and K, N >= 1 required"); return HARTS_EINVAL; }
    if (a->K % 8 || a->N % 8) { set_error("K and N must be multiples of 8 (rows start 16-byte aligned)"); return HARTS_EUNSUPPORTED; }
    if (!sizes_ok(a->C, a->K, a->N)) { set_error("more tiles than the library counts"); return HARTS_EOVERFLOW; }
    if (a->activation < HARTS_ACT_NONE || a->activation > HARTS_ACT_GELU) { set_error("activation must be 0, 1 or 2"); return HARTS_EINVAL; }
    if (a->C == 0) return HARTS_OK;
    if (!a->x || !a->weight) { set_error("NULL x or weight"); return HARTS_EINVAL; }
    if (!aligned16(a->x) || !aligned16(a->weight) || !aligned16(a->bias) || !aligned16(a->residual) || !aligned16(a->y) || !aligned16(a->z) ||
        !aligned16(a->workspace)) {
        set_error("x, weight, bias, residual, y, z and workspace must be 16-byte aligned");
        return HARTS_EINVAL;
    }
    return HARTS_OK;
}

Cut fwd_cut(int64_t C, int32_t K, int32_t N) { return cut_of(C, N, ceil_div(K, kTK), false, 1); }
bool by_dots(int64_t C) { return C <= kDotRows; }

// The backward's two products share a launch, and with it their blocks' grouping.  Workspace: dz,
// rows of column sums, and the pieces of either product.
struct BwdPlan { Cut dx, dw; int32_t per, chunks; size_t dz, sums, part_x, part_w, total; };
BwdPlan plan_bwd(int64_t C, int32_t K, int32_t N, int32_t act, bool bias) {
    BwdPlan b{};
    b.dx = cut_of(C, K, ceil_div(N, kTK), true, 0);
    b.dw = cut_of(N, K, ceil_div(C, kTK), true, 0);
    if (b.dx.G != b.dw.G) {                             // both in single blocks
        b.dx = cut_of(C, K, ceil_div(N, kTK), true, 0, 1);
        b.dw = cut_of(N, K, ceil_div(C, kTK), true, 0, 1);
    }
    const int32_t strips = ceil_div(N, 256);
    // about eight blocks an SM, each of 32 rows at least
    b.per = static_cast<int32_t>(std::max<int64_t>(32, (C * strips + 8 * sm_count() - 1) / (8 * sm_count()) + 7) / 8 * 8);
    b.chunks = ceil_div(C, b.per);
    b.sums = act != HARTS_ACT_NONE ? align256(2 * size_t(C) * N) : 0;
    b.part_x = b.sums + (bias ? align256(4 * size_t(b.chunks) * N) : 0);
    b.part_w = b.part_x + (b.dx.splits > 1 ? align256(4 * size_t(C) * K * b.dx.splits) : 0);
    b.total = b.part_w + (b.dw.splits > 1 ? align256(4 * size_t(N) * K * b.dw.splits) : 0);
    return b;
}

}  // namespace
}  // namespace harts

using namespace harts;

extern "C" {

size_t harts_linear_fwd_workspace_bytes(int64_t C, int32_t K, int32_t N) {
    if (!sizes_ok(C, K, N)) return 0;
    if (by_dots(C)) return 0;
    const Cut c = fwd_cut(C, K, N);
    return c.splits > 1 ? align256(4 * size_t(C) * N * c.splits) : 0;
}

int harts_linear_fwd(const harts_linear_args *a, harts_stream_t stream) {
    const int rc = check(a);
    if (rc) return rc;
    if (a->C == 0) { set_error(""); return HARTS_OK; }
    if (!a->y) { set_error("NULL y"); return HARTS_EINVAL; }
    if (a->y == a->z) { set_error("y and z are one buffer"); return HARTS_EINVAL; }
    const void *const in_use[] = {a->x, a->weight, a->bias};
    for (const void *q : in_use)
        if (a->y == q || (a->z && a->z == q)) { set_error("y and z may not be x, weight or bias"); return HARTS_EINVAL; }
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const Epilogue ep{a->bias, static_cast<const __nv_bfloat16 *>(a->residual)};
    const int32_t C = static_cast<int32_t>(a->C);
    __nv_bfloat16 *y = static_cast<__nv_bfloat16 *>(a->y), *z = static_cast<__nv_bfloat16 *>(a->z);
    if (by_dots(C)) {
        const DotParams d{static_cast<const __nv_bfloat16 *>(a->x), static_cast<const __nv_bfloat16 *>(a->weight), y, z, ep, a->K, a->N};
        const int64_t blocks = (a->N / 2 + 7) / 8;
        const cudaError_t e = with_act(a->activation, [&](auto act) {
            constexpr int kAct = decltype(act)::value;
            return C == 1 ? launch(linear_dot_kernel<1, kAct>, blocks, 256, 0, 1, false, st, d) : launch(linear_dot_kernel<2, kAct>, blocks, 256, 0, 1, false, st, d);
        });
        if (e != cudaSuccess) return cuda_fail(e, "linear forward launch");
        set_error("");
        return HARTS_OK;
    }
    const Cut c = fwd_cut(a->C, a->K, a->N);
    if (c.splits > 1 && (!a->workspace || a->workspace_bytes < align256(4 * size_t(a->C) * a->N * c.splits))) {
        set_error("workspace too small");
        return HARTS_ESMALLBUF;
    }
    float *part = c.splits > 1 ? static_cast<float *>(a->workspace) : nullptr;
    Params p;
    std::memset(&p, 0, sizeof(p));
    p.n_prod = 1;
    p.error = a->error ? a->error : own_error_word();
    if (!p.error) { set_error("the library's error word is not to be had"); return HARTS_ECUDA; }
    bool ok = make_prod(p.prod[0], c, a->C, a->N, a->K, a->x, false, a->weight, false, a->y, part);
    if (!part) {
        p.ep = ep;
        p.keep = z != nullptr;
        if (z) ok = ok && map_out(&p.prod[0].keep, z, 1, a->C, a->N, false);
    }
    if (!ok) { set_error("tensor map"); return HARTS_ECUDA; }
    cudaError_t e = part ? launch_tiles<-1>(p, c.G, false, st)
                         : with_act(a->activation, [&](auto act) { return launch_tiles<decltype(act)::value>(p, c.G, false, st); });
    if (e == cudaSuccess && part) {
        Join j{};
        j.of[0] = JoinOne{part, y, z, a->C * a->N, a->N, c.splits};
        j.ep = ep;
        j.blocks0 = (j.of[0].values / 8 + 127) / 128;
        e = with_act(a->activation, [&](auto act) { return launch(linear_join_kernel<decltype(act)::value>, j.blocks0, 128, 0, 1, true, st, j); });
    }
    if (e != cudaSuccess) return cuda_fail(e, "linear forward launch");
    set_error("");
    return HARTS_OK;
}

size_t harts_linear_bwd_workspace_bytes(int64_t C, int32_t K, int32_t N, int32_t activation, int32_t with_bias) {
    if (!sizes_ok(C, K, N) || activation < HARTS_ACT_NONE || activation > HARTS_ACT_GELU) return 0;
    return C == 0 ? 0 : plan_bwd(C, K, N, activation, with_bias != 0).total;
}

int harts_linear_bwd(const harts_linear_bwd_args *b, harts_stream_t stream) {
    if (!b) { set_error("NULL args"); return HARTS_EINVAL; }
    const harts_linear_args *a = &b->fwd;
    const int rc = check(a);
    if (rc) return rc;
    if (!b->dx && !b->dweight && !b->dbias) { set_error("no output: dx, dweight and dbias are all NULL"); return HARTS_EINVAL; }
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (a->C == 0) {
        cudaError_t e = cudaSuccess;
        if (b->dweight) e = cudaMemsetAsync(b->dweight, 0, 2 * size_t(a->N) * a->K, st);
        if (e == cudaSuccess && b->dbias) e = cudaMemsetAsync(b->dbias, 0, 4 * size_t(a->N), st);
        if (e != cudaSuccess) return cuda_fail(e, "linear backward");
        set_error("");
        return HARTS_OK;
    }
    const bool curved = a->activation != HARTS_ACT_NONE;
    if (!b->d_y || (curved && !a->z)) { set_error("NULL d_y or z"); return HARTS_EINVAL; }
    if (!aligned16(b->d_y) || !aligned16(b->dx) || !aligned16(b->dweight) || !aligned16(b->dbias)) {
        set_error("d_y, dx, dweight and dbias must be 16-byte aligned");
        return HARTS_EINVAL;
    }
    const void *const in_use[] = {a->x, a->weight, b->d_y, a->z};
    for (const void *q : in_use)
        if ((b->dx && b->dx == q) || (b->dweight && b->dweight == q)) { set_error("dx and dweight may be none of the inputs"); return HARTS_EINVAL; }
    if (b->dx && b->dx == b->dweight) { set_error("two outputs in one buffer"); return HARTS_EINVAL; }
    const BwdPlan w = plan_bwd(a->C, a->K, a->N, a->activation, b->dbias != nullptr);
    if (w.total && (!a->workspace || a->workspace_bytes < w.total)) { set_error("workspace too small"); return HARTS_ESMALLBUF; }
    if (reinterpret_cast<uintptr_t>(a->workspace) % 256) { set_error("workspace must be 256-byte aligned"); return HARTS_EINVAL; }
    uint8_t *ws = static_cast<uint8_t *>(a->workspace);
    Params p;
    std::memset(&p, 0, sizeof(p));
    p.error = a->error ? a->error : own_error_word();
    if (!p.error) { set_error("the library's error word is not to be had"); return HARTS_ECUDA; }
    const void *dz = curved ? static_cast<const void *>(ws) : b->d_y;
    float *part_x = w.dx.splits > 1 ? reinterpret_cast<float *>(ws + w.part_x) : nullptr;
    float *part_w = w.dw.splits > 1 ? reinterpret_cast<float *>(ws + w.part_w) : nullptr;
    bool ok = true;
    Join j{};
    int joins = 0;
    if (b->dweight) {
        ok = make_prod(p.prod[p.n_prod++], w.dw, a->N, a->K, a->C, dz, true, a->x, true, b->dweight, part_w);
        if (part_w) j.of[joins++] = JoinOne{part_w, static_cast<__nv_bfloat16 *>(b->dweight), nullptr, int64_t(a->N) * a->K, a->K, w.dw.splits};
    }
    if (b->dx) {
        ok = ok && make_prod(p.prod[p.n_prod++], w.dx, a->C, a->K, a->N, dz, false, a->weight, true, b->dx, part_x);
        if (part_x) j.of[joins++] = JoinOne{part_x, static_cast<__nv_bfloat16 *>(b->dx), nullptr, a->C * a->K, a->K, w.dx.splits};
    }
    if (!ok) { set_error("tensor map"); return HARTS_ECUDA; }
    cudaError_t e = cudaSuccess;
    bool behind = false;
    if (b->dbias || (curved && p.n_prod)) {
        const DzParams d{static_cast<const __nv_bfloat16 *>(b->d_y), curved ? static_cast<const __nv_bfloat16 *>(a->z) : nullptr,
                         reinterpret_cast<__nv_bfloat16 *>(ws), b->dbias ? reinterpret_cast<float *>(ws + w.sums) : nullptr,
                         a->C, a->N, w.per};
        e = with_act(a->activation, [&](auto act) {
            return launch(linear_dz_kernel<decltype(act)::value>, int64_t(ceil_div(a->N, 256)) * w.chunks, 256, 0, 1, false, st, d);
        });
        behind = true;
        if (e == cudaSuccess && b->dbias) {
            const DbParams s{reinterpret_cast<const float *>(ws + w.sums), b->dbias, a->N, w.chunks};
            e = launch(linear_db_kernel, ceil_div(a->N, 32), 1024, 0, 1, true, st, s);
        }
    }
    if (e == cudaSuccess && p.n_prod) e = launch_tiles<-1>(p, w.dx.G, behind, st);
    if (e == cudaSuccess && joins) {
        int64_t blocks[2] = {(j.of[0].values / 8 + 127) / 128, joins > 1 ? (j.of[1].values / 8 + 127) / 128 : 0};
        j.blocks0 = blocks[0];
        e = launch(linear_join_kernel<HARTS_ACT_NONE>, blocks[0] + blocks[1], 128, 0, 1, true, st, j);
    }
    if (e != cudaSuccess) return cuda_fail(e, "linear backward launch");
    set_error("");
    return HARTS_OK;
}

}  // extern "C"
