// Gated linear recurrence per channel over the rows of a forest, forward and backward.
//
//   a_r = e^(g_r),  h_r = a_r h_p(r) + b_r,   b_r = x_r (add) or (1 - a_r) x_r (mix)
//   lam_r = dh_r + sum over rows c with p(c) = r of a_c lam_c  (+ d_final at a sequence's end)
//   dx_r = lam_r (add) or (1 - a_r) lam_r (mix),   dg_r = lam_r a_r (h_p(r) - [mix] x_r)
// p(r): the row before r on its trajectory, the root's initial state at a trajectory's start.
// States, decays and their products are fp32; h in `dtype` is what the backward takes h_p from.
//
// Both directions compose affine maps c -> A c + B along a row's trajectory: forward with
// A = a_r, B = b_r, backward on c_r = a_r lam_r with A = a_r, B = a_r dh_r, from the leaves up.  Every
// value is read and written once; HBM bounds the work, and the chain of carries must not.  The
// planner cuts segments into tiles of 128 rows (a fork lies at a tile's end); a block takes a
// tile of 128 bytes of channels: eight warps of 16 rows each compose their rows' map, a ninth
// joins the eight and forms the carry, from the maps that the tiles before it in its group published
// (8 to 32 tiles of a segment, which need not wait for one another) and the state that the group before
// left, both fetched while the rows are still on their way: a chain waits once for 1,024 to 4,096 rows,
// about 1 us.  The order in which maps are joined is fixed by position: no atomics on values, the same
// bits on every run.  What is published carries its own validity: the workspace starts as all ones, a NaN
// that no published value has.  Tiles are taken in an order that has predecessors first, by a ticket
// counter, so that whatever a block waits for is in the hands of a running one; every wait is bounded all
// the same.
//
// bf16: 65,536 rows of 2,048 channels in 361 segments, add form: 141 us (84 % of the copy's rate), gradients 234 (84 %);
// mix form's gradients 314 (76 %).  fp32, 1,024 channels: 137 (86 %) and 226 (88 %).  One trajectory of 131,071 rows, 1,024
// channels, mix form with states: 182 us (65 %), bound by the chain of its groups, each of which waits for the finished
// state of the one before; gradients 421 (56 %).  512 segments of 128 rows: 140 (84 %); 4,096 of 16: 563 (21 %), where a
// tile's fixed time, 1.9 us a block, is all.  48 single rows: 1.4 us on the device.  Gradients behind a wide fork are far
// from either bound: the fork's last group adds its branches' states one after another, each fetched behind
// the one before, in every tile of it (512 branches of 120 rows off 4,096: 1,150 us, forward 145).
#include <algorithm>
#include <cstring>
#include <type_traits>

#include "kda_common.cuh"
#include "launch_util.h"
#include "tc_primitives.cuh"
#include "tensor_map.h"
#include "two.cuh"

namespace harts {
namespace {

using namespace two;

constexpr int kWarps = 8, kWarpRows = kScanRows / kWarps;      // consumers
constexpr int kThreads = 32 * (kWarps + 2);                    // and a warp each for carries and copies
constexpr int kAtOnce = 8;                                     // maps that are fetched at a time
constexpr int kBox = 32;                                       // rows of one copy
// Rows of a tile for a warp: sixteen, and none for the last warps of a short tile; but as many for each (EVEN) where
// a warp also fetches its rows' x itself.  (The mix form's gradients, 65,536 rows of 2,048 channels: 768 segments 430 us to
// 378, 361 335 to 314; elsewhere a short tile only gains more joins: forward, 1,024 segments of 64 rows 153 to 172.)
template <bool EVEN> __device__ __forceinline__ int rows_each(int rows) { return EVEN ? (rows + kWarps - 1) / kWarps : kWarpRows; }
constexpr uint32_t kTileBytes = kScanRows * 128;               // of one tensor
constexpr uint32_t kEmpty = 0xffffffffu;                       // not published yet

struct ScanParams {
    CUtensorMap map[3];             // forward g, x; backward g, dh, h
    const ScanTile *tiles;
    const int32_t *next;
    const float *h0, *d_final;
    const void *h_in, *x_in;        // backward: h, x
    void *out0, *out1;              // forward h; backward dx, dg
    float *final_state, *dh0;
    uint32_t *ticket;               // nullptr: tiles that wait for nothing are dealt out in turn
    float *inc;                     // [slots][width] state behind a group (backward: before it)
    float2 *agg;                    // [tiles][width] a tile's map
    int32_t *error;
    int32_t D, width, cols, group;  // channels, rounded up to tiles', tiles across; most tiles of a group
    uint32_t total;
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The channels of a lane, 4 bytes: two of bf16, whose fp32 arithmetic runs on pairs (half as many
// instructions, which are what the exact decay below would be bound by), or one of fp32.
template <typename T> struct Lane;
template <> struct Lane<__nv_bfloat16> {
    using V = Two;
    static constexpr int n = 2;
    __device__ __forceinline__ static V all(float c) { return make_float2(c, c); }
    __device__ __forceinline__ static V get(const void *p) {
        const uint32_t u = *static_cast<const uint32_t *>(p);
        return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
    }
    __device__ __forceinline__ static void put(void *p, V v) { *static_cast<__nv_bfloat162 *>(p) = __floats2bfloat162_rn(v.x, v.y); }
    __device__ __forceinline__ static V load(const float *p) { return *reinterpret_cast<const float2 *>(p); }
    __device__ __forceinline__ static void store(float *p, V v) { *reinterpret_cast<float2 *>(p) = v; }
};
template <> struct Lane<float> {
    using V = float;
    static constexpr int n = 1;
    __device__ __forceinline__ static V all(float c) { return c; }
    __device__ __forceinline__ static V get(const void *p) { return *static_cast<const float *>(p); }
    __device__ __forceinline__ static void put(void *p, V v) { *static_cast<float *>(p) = v; }
    __device__ __forceinline__ static V load(const float *p) { return *p; }
    __device__ __forceinline__ static void store(float *p, V v) { *p = v; }
};

// e^g for g <= 0, as one number that gives both a and 1 - a with few roundings.  2^y = 2^n 2^f with
// |f| <= 1/2, y = g log2 e with the factor in two terms (one alone is 2e-8 off, which g = -88 makes 20 u of
// a, u = 2^-24), and the series of e^(f ln 2) to its seventh power (the next term is 5e-9); below
// 2^-126.5, zero.  a is within 1.9 u of itself, 1 - a within 2.6 u.  Memories of a thousand rows multiply a thousand decays: an approximate
// exponential's 2^-22 would be 2e-4 of the state.  kExact keeps a.  kRest keeps 1 - a, which the
// rounding of an a near 1 would take most digits of: 2^n (1 + t) with t the series gives it as
// (1 - 2^n) - 2^n t, rounded once; a is then 1 - (1 - a), off by 2^-25 at most.  kBoth, for the mix
// form's gradients, which have a as a factor, keeps a below 2^(-1/2) and -(1 - a), its sign bit set,
// from there up.  kFast, the hardware's exponential, is for results that are all bf16, which
// rounds to 2^-9, in the add form, where no trajectory has more than kFastRows rows: so many decays
// are off by 2^-10 at most.  (A microbatch of 361 segments, 65,536 rows of 2,048 channels: 141 us, 168 with
// the series.  Slow decays over 131,072 rows: off by up to 2^-7.3 with it, with the series by the 2^-8 of
// the result's rounding.)  So the bits of h are those of one kernel or the other, by what else is asked for and by the
// longest trajectory of the forest.
constexpr int64_t kFastRows = 4096;
enum Kind { kFast, kExact, kRest, kBoth };
template <int KIND, typename T> __device__ __forceinline__ typename Lane<T>::V decay(typename Lane<T>::V g) {
    using L = Lane<T>;
    if constexpr (KIND == kFast) return each(mul(g, L::all(1.4426950408889634f)), [](float y) { return ex2(y); });
    g = each(g, [](float v) {
        float y;
        asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(v), "f"(-88.f));
        return y;
    });
    const auto z = fma(g, L::all(1.4426950408889634f), L::all(12582912.f));        // its low bits are n
    const auto n = fma(z, L::all(-1.f), L::all(12582912.f));                       // -n
    const auto f = fma(g, L::all(1.9259629911e-8f), fma(g, L::all(1.4426950408889634f), n));
    constexpr float sign = KIND == kExact ? 1.f : -1.f;
    auto q = L::all(sign * 1.5252733804e-5f);
    q = fma(q, f, L::all(sign * 1.5403530394e-4f));
    q = fma(q, f, L::all(sign * 1.3333558146e-3f));
    q = fma(q, f, L::all(sign * 9.6181291076e-3f));
    q = fma(q, f, L::all(sign * 5.5504108665e-2f));
    q = fma(q, f, L::all(sign * 2.4022650696e-1f));
    q = fma(q, f, L::all(sign * 6.9314718056e-1f));
    const auto t = mul(q, f);                                                      // times the sign
    const auto scale = each(z, [](float v) { return __uint_as_float((__float_as_uint(v) << 23) + 0x3f800000u); });
    if constexpr (KIND == kExact) return fma(t, scale, scale);
    const auto rest = fma(t, scale, fma(scale, L::all(-1.f), L::all(1.f)));
    if constexpr (KIND == kRest) return rest;
    const auto a = fma(mul(t, L::all(-1.f)), scale, scale);
    return each(a, rest, [](float u, float r) { return u < 0.70710678f ? u : __uint_as_float(__float_as_uint(r) | 0x80000000u); });
}
template <int KIND, typename V> __device__ __forceinline__ V keep_of(V v) {      // a
    if constexpr (KIND == kRest) return each(v, [](float u) { return 1.f - u; });
    if constexpr (KIND == kBoth) return each(v, [](float u) { return __float_as_int(u) < 0 ? 1.f + u : u; });
    return v;
}
template <int KIND, typename V> __device__ __forceinline__ V rest_of(V v) {      // 1 - a
    if constexpr (KIND == kRest) return v;
    return each(v, [](float u) { return __float_as_int(u) < 0 ? -u : 1.f - u; });
}

__device__ __forceinline__ uint32_t publishable(float v) { return v == v ? __float_as_uint(v) : 0x7fffffffu; }
__device__ __forceinline__ void publish(float2 *at, float a, float b) {
    const uint64_t u = static_cast<uint64_t>(publishable(b)) << 32 | publishable(a);
    asm volatile("st.relaxed.gpu.global.b64 [%0], %1;" :: "l"(at), "l"(u) : "memory");
}
__device__ __forceinline__ void publish(float *at, float v) {
    asm volatile("st.relaxed.gpu.global.b32 [%0], %1;" :: "l"(at), "r"(publishable(v)) : "memory");
}
__device__ __forceinline__ void publish(float *at, Two v) { publish(reinterpret_cast<float2 *>(at), v.x, v.y); }
__device__ __forceinline__ float2 look(const float2 *at) {
    uint64_t u;
    asm volatile("ld.relaxed.gpu.global.b64 %0, [%1];" : "=l"(u) : "l"(at) : "memory");
    return make_float2(__uint_as_float(static_cast<uint32_t>(u)), __uint_as_float(static_cast<uint32_t>(u >> 32)));
}
__device__ __forceinline__ float look(const float *at) {
    uint32_t u;
    asm volatile("ld.relaxed.gpu.global.b32 %0, [%1];" : "=r"(u) : "l"(at) : "memory");
    return __uint_as_float(u);
}
__device__ __forceinline__ bool is_there(float v) { return __float_as_uint(v) != kEmpty; }
__device__ __forceinline__ bool is_there(float2 v) { return is_there(v.x) && is_there(v.y); }

__device__ __forceinline__ bool gave_up(const int *f) { return *reinterpret_cast<const volatile int *>(f) != 0; }

__device__ __forceinline__ void arrive(uint64_t *bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" :: "r"(tc::smem_addr(bar)) : "memory");
}
// Whether the phase has completed, without the while that try_wait may stay for.
__device__ __forceinline__ bool is_done(uint64_t *bar, uint32_t phase) {
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(ok) : "r"(tc::smem_addr(bar)), "r"(phase) : "memory");
    return ok != 0;
}
// True, for the whole warp, once the phase completed; false when the wait ran out or another role gave up.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t phase, int *f) {
    bool ok = tc::mbar_try(bar, phase);
    if (!ok && !gave_up(f)) {
        ok = tc::mbar_wait(bar, phase);
        if (!ok) *reinterpret_cast<volatile int *>(f) = 1;
    }
    return __all_sync(0xffffffffu, ok) != 0;
}

// Tensors of a tile, stages of the ring and blocks of an SM: as many bytes on their way as shared
// memory holds.  AHEAD: a tile's map is composed, and published, before the results of the tile
// before it in the block, whose carry may be long in coming: on long trajectories all blocks would
// otherwise compose and then wait together.  That takes the registers of two tiles' decays, so a third
// block's, and does nothing for tiles that need not wait: the forward takes it where the longest trajectory has
// kAheadRows rows.  (bf16, mix form, groups of 16: one of 131,072 rows of 1,024 channels 192 us, 339 without; 4 of
// 16,384 rows of 2,048 channels 170 and 202, 8 of 8,192 rows 168 and 177, 16 of 4,200 rows 172 and 169,
// 16 chains of 40 segments of 200 rows 215 and 197; before the decay's argument had its second term.)
constexpr int64_t kAheadRows = 8192;
// Groups of 8 tiles are the forward's where more than eight tiles lie side by side; up to eight are too few to fill
// the chip with small groups, and up to two leave the chain of carries as all there is.  (131,072 rows, bf16, mix, in
// groups of 8 / 16 / 32: 1,024 channels 180 us / 192 / 221, 512 127 / 111 / 137, 256 110 / 76 / 79, 128 97 / 72 / 49, 64
// 90 / 54 / 35.  Backward, add form, 1,024 channels: 406 / 394 / 345, now 359 with the decay's second term.)
template <bool BWD, bool AHEAD> struct Ring {
    static constexpr int tensors = BWD ? 3 : 2, stages = AHEAD ? 3 : 2, blocks = BWD || AHEAD ? 2 : 3;
    static constexpr uint32_t stage_bytes = tensors * kTileBytes;
    static constexpr uint32_t smem = stages * stage_bytes + 128;
};

struct Meta { ScanPlace t; int32_t col; };                      // rows 0: the end

template <typename T, bool BWD, bool MIX, int KIND, bool AHEAD>
__global__ void __launch_bounds__(kThreads, Ring<BWD, AHEAD>::blocks) scan_kernel(const __grid_constant__ ScanParams p) {
    using R = Ring<BWD, AHEAD>;
    using L = Lane<T>;
    using V = typename L::V;
    constexpr int CH = L::n, kWide = 32 * CH;
    extern __shared__ uint8_t smraw[];
    uint8_t *sm = smraw + ((128 - (tc::smem_addr(smraw) & 127)) & 127);
    __shared__ uint64_t known[R::stages], full[R::stages], empty[R::stages];
    __shared__ uint64_t maps_full[R::stages], carry_full[R::stages];
    __shared__ Meta meta[R::stages];
    __shared__ V s_a[R::stages][kWarps][32], s_b[R::stages][kWarps][32], s_carry[R::stages][32];   // the warps' maps, the carry
    __shared__ int s_fail, s_mapped[R::stages];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < R::stages; ++s) {
            tc::mbar_init(&known[s], 1);
            tc::mbar_init(&full[s], 1);
            tc::mbar_init(&empty[s], kWarps + 1);
            tc::mbar_init(&maps_full[s], kWarps);
            tc::mbar_init(&carry_full[s], 1);
            s_mapped[s] = 0;
        }
        tc::fence_mbar_init();
        s_fail = 0;
    }
    __syncthreads();

    // Every role leaves its loop at the first wait that does not end, without a look at what it
    // waited for.
    if (warp == kWarps + 1) {
        // copies: the next ticket is drawn while the stage of the current one is waited for
        auto draw = [&]() -> uint32_t {
            uint32_t n = 0;
            if (lane == 0) n = atomicAdd(p.ticket, 1u) + 1;    // it starts at all ones
            return n;
        };
        uint32_t drawn = p.ticket ? draw() : 0, it = 0;
        bool ended = false;
        for (;; ++it) {
            const uint32_t idx = p.ticket ? __shfl_sync(0xffffffffu, drawn, 0) : blockIdx.x + it * gridDim.x;
            const int s = it % R::stages;
            Meta m{};
            if (idx < p.total) {
                m.t = scan_place(p.tiles[idx / p.cols], p.group);
                m.col = static_cast<int32_t>(idx % p.cols) * kWide;
                if (p.ticket) drawn = draw();
            }
            if (it >= R::stages && !warp_wait(&empty[s], (it / R::stages - 1) & 1, &s_fail)) break;
            const int boxes = (m.t.rows + kBox - 1) / kBox;
            if (lane == 0) {
                meta[s] = m;
                arrive(&known[s]);
                if (m.t.rows) tc::mbar_expect_tx(&full[s], boxes * R::tensors * kBox * 128);
                else arrive(&full[s]);
            }
            __syncwarp();
            if (!m.t.rows) { ended = true; break; }
            for (int b = lane; b < boxes * R::tensors; b += 32) {
                const int which = b / boxes, k = b % boxes;
                const int row = m.t.row0 + k * kBox - (BWD && which == 2 ? 1 : 0);       // h of the row before
                tc::tma_load_2d(sm + s * R::stage_bytes + which * kTileBytes + k * kBox * 128, &p.map[which], m.col, row, &full[s]);
            }
        }
        // No copy is in flight when the block ends: the stages' last ones are waited for (the one
        // before the end mark has been used already).
        for (uint32_t k = it > R::stages ? it - R::stages : 0; k < it; ++k)
            if (!ended || it - k < R::stages) tc::mbar_wait(&full[k % R::stages], (k / R::stages) & 1);
    } else if (warp == kWarps) {
        // Carries, a tile's ahead of its rows: as soon as it is known which tile it is, the maps
        // between the group's carry and the tile are joined, in the order of the rows; then comes
        // whichever is there first, the carry or the tile's own map, which others wait for.
        for (uint32_t it = 0;; ++it) {
            const int s = it % R::stages;
            if (!warp_wait(&known[s], (it / R::stages) & 1, &s_fail)) break;
            const Meta m = meta[s];
            if (m.t.rows == 0) break;
            const int64_t ch = m.col + lane * CH;
            const bool inside = ch < p.D;                      // channels come in eights
            float2 *agg = p.agg + static_cast<int64_t>(m.t.tile) * p.width + ch;
            V pa = L::all(1.f), pb = L::all(0.f), v = L::all(0.f), A = L::all(1.f), B = L::all(0.f);
            bool mapped = false, carried = false;
            const int between = BWD ? m.t.count - 1 - m.t.at : m.t.at;
            int k = between;                                   // maps still to be joined, the farthest first
            int left = BWD ? m.t.next_count : m.t.pred >= 0;   // states still to come, in order
            const long long t0 = clock64();
            while (!mapped || !carried) {
                if (!mapped && __all_sync(0xffffffffu, is_done(&maps_full[s], (it / R::stages) & 1))) {
#pragma unroll
                    for (int i = 0; i < kWarps; ++i) {
                        const int w = BWD ? kWarps - 1 - i : i;
                        B = fma(s_a[s][w][lane], B, s_b[s][w][lane]);
                        A = mul(s_a[s][w][lane], A);
                    }
                    if (!AHEAD && (BWD ? m.t.at > 0 : m.t.at < m.t.count - 1)) {
                        if constexpr (CH == 2) { publish(agg, A.x, B.x); publish(agg + 1, A.y, B.y); }
                        else publish(agg, A, B);
                    }
                    mapped = true;
                }
                V state = L::all(0.f);
                bool there = false;
                if (left > 0) {
                    const int64_t g = !BWD ? m.t.pred : m.t.next_begin < 0 ? -1 - m.t.next_begin : p.next[m.t.next_begin + m.t.next_count - left];
                    if constexpr (CH == 2) state = look(reinterpret_cast<const float2 *>(p.inc + g * p.width + ch));
                    else state = look(p.inc + g * p.width + ch);
                }
                if (k > 0) {                                   // up to kAtOnce maps, if they are all there
                    float2 w[kAtOnce][CH];
#pragma unroll
                    for (int i = 0; i < kAtOnce; ++i)
#pragma unroll
                        for (int c = 0; c < CH; ++c)
                            w[i][c] = k - i > 0 ? look(agg + static_cast<int64_t>(BWD ? k - i : i - k) * p.width + c) : make_float2(1.f, 0.f);
                    there = true;
#pragma unroll
                    for (int i = 0; i < kAtOnce; ++i)
#pragma unroll
                        for (int c = 0; c < CH; ++c) there = there && is_there(w[i][c]);
                    if (__all_sync(0xffffffffu, there)) {
#pragma unroll
                        for (int i = 0; i < kAtOnce; ++i) {    // (past the last one: a map that changes nothing)
                            if constexpr (CH == 2) {
                                const V a = make_float2(w[i][0].x, w[i][CH - 1].x);
                                pb = fma(a, pb, make_float2(w[i][0].y, w[i][CH - 1].y));
                                pa = mul(a, pa);
                            } else {
                                pb = fma(w[i][0].x, pb, w[i][0].y);
                                pa = mul(w[i][0].x, pa);
                            }
                        }
                        k -= kAtOnce;
                    }
                }
                if (left > 0) {
                    if (__all_sync(0xffffffffu, is_there(state))) { v = add(v, state); --left; }
                }
                if (!carried && left == 0 && k <= 0) {
                    if (!BWD && m.t.pred < 0 && p.h0 && inside) v = L::load(p.h0 + static_cast<int64_t>(-1 - m.t.pred) * p.D + ch);
                    if (BWD && m.t.seq_end >= 0 && p.d_final && inside)
                        v = add(v, L::load(p.d_final + static_cast<int64_t>(m.t.seq_end) * p.D + ch));
                    if (between > 0) v = fma(pa, v, pb);
                    s_carry[s][lane] = v;
                    __syncwarp();
                    if (lane == 0) arrive(&carry_full[s]);
                    carried = true;
                }
                if (clock64() - t0 > 4000000000LL) *reinterpret_cast<volatile int *>(&s_fail) = 1;
                if (__any_sync(0xffffffffu, gave_up(&s_fail))) break;
            }
            if (!mapped || !carried) break;
            v = fma(A, v, B);
            if (BWD ? m.t.at == 0 && m.t.pred >= 0 : m.t.at == m.t.count - 1 && m.t.next_count > 0)
                publish(p.inc + static_cast<int64_t>(m.t.slot) * p.width + ch, v);
            else if (BWD && m.t.at == 0 && p.dh0 && inside)
                L::store(p.dh0 + static_cast<int64_t>(-1 - m.t.pred) * p.D + ch, v);
            __syncwarp();
            if (lane == 0) arrive(&empty[s]);
        }
    } else {
        // The tile's rows, 0 behind the last one, -1 where a wait did not end.
        auto map_tile = [&](uint32_t it, V (&d)[kWarpRows], [[maybe_unused]] V &before, [[maybe_unused]] uint32_t *xr) -> int {
            const int s = it % R::stages;
            if (!warp_wait(&full[s], (it / R::stages) & 1, &s_fail)) return -1;
            const int rows = meta[s].t.rows;
            if (rows == 0) return 0;
            const int from = warp * rows_each<BWD && MIX>(rows), mine = min(max(rows - from, 0), rows_each<BWD && MIX>(rows));
            const uint8_t *src = sm + s * R::stage_bytes + from * 128 + lane * 4;
            const int64_t ch = meta[s].col + lane * CH;
            if (BWD && warp == 0 && ch < p.D) {                // state before the tile's first row
                const int32_t pr = meta[s].t.pred_row;
                before = L::all(0.f);
                if (pr >= 0) before = L::get(static_cast<const T *>(p.h_in) + static_cast<int64_t>(pr) * p.D + ch);
                else if (p.h0) before = L::load(p.h0 + static_cast<int64_t>(-1 - pr) * p.D + ch);
            }
            if constexpr (BWD && MIX) {
                const T *xp = static_cast<const T *>(p.x_in) + static_cast<int64_t>(meta[s].t.row0 + from) * p.D + ch;
#pragma unroll
                for (int i = 0; i < kWarpRows; ++i)
                    xr[i] = i < mine && ch < p.D ? __ldcs(reinterpret_cast<const uint32_t *>(xp + static_cast<int64_t>(i) * p.D)) : 0u;
            }
            V A = L::all(1.f), B = L::all(0.f);
            auto map_row = [&](int i) {
                const V u = L::get(src + kTileBytes + i * 128);
                d[i] = decay<KIND, T>(L::get(src + i * 128));
                const V a = keep_of<KIND>(d[i]);
                if (BWD) B = mul(a, add(u, B));
                else B = fma(a, B, MIX ? mul(rest_of<KIND>(d[i]), u) : u);
                A = mul(A, a);
            };
            if (mine == kWarpRows) {
#pragma unroll
                for (int k = 0; k < kWarpRows; ++k) map_row(BWD ? kWarpRows - 1 - k : k);
            } else {
#pragma unroll
                for (int k = 0; k < kWarpRows; ++k)
                    if ((BWD ? kWarpRows - 1 - k : k) < mine) map_row(BWD ? kWarpRows - 1 - k : k);
            }
            s_a[s][warp][lane] = A;
            s_b[s][warp][lane] = B;
            __syncwarp();
            int last = 0;
            if (lane == 0) {
                arrive(&maps_full[s]);
                if (AHEAD) {
                    __threadfence_block();
                    last = atomicAdd(&s_mapped[s], 1) == kWarps - 1;
                    __threadfence_block();
                    if (last) s_mapped[s] = 0;
                }
            }
            if (AHEAD && __shfl_sync(0xffffffffu, last, 0) && meta[s].t.at < meta[s].t.count - 1) {
                __syncwarp();                                  // the other warps' maps, which the first lane has seen
                A = L::all(1.f), B = L::all(0.f);
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    B = fma(s_a[s][w][lane], B, s_b[s][w][lane]);
                    A = mul(s_a[s][w][lane], A);
                }
                float2 *agg = p.agg + static_cast<int64_t>(meta[s].t.tile) * p.width + ch;
                if constexpr (CH == 2) { publish(agg, A.x, B.x); publish(agg + 1, A.y, B.y); }
                else publish(agg, A, B);
            }
            return rows;
        };
        auto results = [&](uint32_t it, const V (&d)[kWarpRows], [[maybe_unused]] V before, [[maybe_unused]] const uint32_t *xr) -> bool {
            const int s = it % R::stages;
            if (!warp_wait(&maps_full[s], (it / R::stages) & 1, &s_fail) || !warp_wait(&carry_full[s], (it / R::stages) & 1, &s_fail)) return false;
            const int rows = meta[s].t.rows, from = warp * rows_each<BWD && MIX>(rows), mine = min(max(rows - from, 0), rows_each<BWD && MIX>(rows));
            const uint8_t *src = sm + s * R::stage_bytes + from * 128 + lane * 4;
            const int64_t ch = meta[s].col + lane * CH;
            V v = s_carry[s][lane];
            for (int k = BWD ? kWarps - 1 : 0; k != warp; k += BWD ? -1 : 1) v = fma(s_a[s][k][lane], v, s_b[s][k][lane]);
            if (ch < p.D) {
                const int64_t at = static_cast<int64_t>(meta[s].t.row0 + from) * p.D + ch;
                T *out0 = static_cast<T *>(p.out0) + at;
                [[maybe_unused]] T *out1 = static_cast<T *>(p.out1) + at;
                auto row = [&](int i) {
                    const V u = L::get(src + kTileBytes + i * 128);
                    if constexpr (!BWD) {
                        v = fma(keep_of<KIND>(d[i]), v, MIX ? mul(rest_of<KIND>(d[i]), u) : u);
                        L::put(out0 + static_cast<int64_t>(i) * p.D, v);
                    } else {
                        V h = L::get(src + 2 * kTileBytes + i * 128);
                        if (i == 0 && warp == 0) h = before;
                        if (MIX) h = fma(L::get(&xr[MIX ? i : 0]), L::all(-1.f), h);
                        const V lam = add(u, v);
                        v = mul(keep_of<KIND>(d[i]), lam);
                        L::put(out0 + static_cast<int64_t>(i) * p.D, MIX ? mul(rest_of<KIND>(d[i]), lam) : lam);
                        L::put(out1 + static_cast<int64_t>(i) * p.D, mul(v, h));
                    }
                };
                if (mine == kWarpRows) {
#pragma unroll
                    for (int k = 0; k < kWarpRows; ++k) row(BWD ? kWarpRows - 1 - k : k);
                } else {
#pragma unroll
                    for (int k = 0; k < kWarpRows; ++k)
                        if ((BWD ? kWarpRows - 1 - k : k) < mine) row(BWD ? kWarpRows - 1 - k : k);
                }
                if (!BWD && p.final_state && meta[s].t.seq_end >= 0 && meta[s].t.at == meta[s].t.count - 1 && mine > 0 && from + mine == rows)
                    L::store(p.final_state + static_cast<int64_t>(meta[s].t.seq_end) * p.D + ch, v);
            }
            __syncwarp();
            if (lane == 0) arrive(&empty[s]);
            return true;
        };
        V d[kWarpRows], before = L::all(0.f);
        uint32_t xr[BWD && MIX ? kWarpRows : 1];
        if constexpr (AHEAD) {
            V next[kWarpRows];
            int rows = map_tile(0, d, before, xr);
            for (uint32_t it = 0; rows > 0; ++it) {
                rows = map_tile(it + 1, next, before, xr);
                if (rows < 0 || !results(it, d, before, xr)) break;
#pragma unroll
                for (int i = 0; i < kWarpRows; ++i) d[i] = next[i];
            }
        } else {
            for (uint32_t it = 0; map_tile(it, d, before, xr) > 0; ++it)
                if (!results(it, d, before, xr)) break;
        }
    }
    __syncthreads();
    if (threadIdx.x == 0 && s_fail) atomicCAS(p.error, 0, static_cast<int>(kDevErrTimeout));
}

// Every segment a root of one row (a decoding step): row, root and sequence have one number.
template <typename T, bool BWD, bool MIX>
__global__ void __launch_bounds__(128) scan_step_kernel(const __grid_constant__ ScanParams p, const T *g, const T *u, const T *x, int64_t n) {
    using L = Lane<T>;
    using V = typename L::V;
    constexpr int KIND = !MIX ? kExact : BWD ? kBoth : kRest;
    const int64_t i = (static_cast<int64_t>(blockIdx.x) * 128 + threadIdx.x) * L::n;
    if (i >= n) return;
    const V d = decay<KIND, T>(L::get(g + i)), a = keep_of<KIND>(d), in = L::get(u + i);
    V h = p.h0 ? L::load(p.h0 + i) : L::all(0.f);
    if constexpr (!BWD) {
        const V o = fma(a, h, MIX ? mul(rest_of<KIND>(d), in) : in);
        L::put(static_cast<T *>(p.out0) + i, o);
        if (p.final_state) L::store(p.final_state + i, o);
    } else {
        const V lam = p.d_final ? add(in, L::load(p.d_final + i)) : in, c = mul(a, lam);
        if (MIX) h = fma(L::get(x + i), L::all(-1.f), h);
        L::put(static_cast<T *>(p.out0) + i, MIX ? mul(rest_of<KIND>(d), lam) : lam);
        L::put(static_cast<T *>(p.out1) + i, mul(c, h));
        if (p.dh0) L::store(p.dh0 + i, c);
    }
}

// ---- host ---------------------------------------------------------------------------------

size_t align256(size_t x) { return (x + 255) / 256 * 256; }
int32_t wide_of(int32_t dtype) { return dtype == HARTS_BF16 ? 64 : 32; }
bool one_step(const harts_plan *P) { return P->info.n_seg == P->info.C && P->info.n_roots == P->info.n_seg; }

struct Space { size_t inc, agg, total; };       // behind 256 bytes with the ticket counter
Space space_of(const harts_plan *P, int32_t D, int32_t dtype) {
    const size_t width = size_t(ceil_div(D, wide_of(dtype))) * wide_of(dtype);
    Space s{};
    if (P->image.scan_alone) return s;
    s.inc = 256;
    s.agg = s.inc + align256(4 * width * P->image.n_scan_slots);
    s.total = s.agg + align256(8 * width * P->image.n_scan);
    return s;
}

template <typename T> bool map_rows(CUtensorMap *m, const void *base, int64_t C, int32_t D) {
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(C)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(D) * sizeof(T)};
    const cuuint32_t box[2] = {128 / sizeof(T), kBox}, es[2] = {1, 1};
    auto fn = encode_tiled();
    return fn && fn(m, sizeof(T) == 4 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
                    const_cast<void *>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, bool BWD, bool MIX, int KIND, bool AHEAD>
cudaError_t launch_scan(const ScanParams &p, cudaStream_t st) {
    using R = Ring<BWD, AHEAD>;
    static std::atomic<uint64_t> done{0};
    auto *k = scan_kernel<T, BWD, MIX, KIND, AHEAD>;
    const cudaError_t e = allow_smem(k, R::smem, done);
    if (e != cudaSuccess) return e;
    const int64_t blocks = std::min<int64_t>(p.total, int64_t(sm_count()) * R::blocks);
    return launch(k, blocks, kThreads, R::smem, 1, false, st, p);
}

// in: g, then x (forward) or dh, h, x
template <typename T, bool BWD, bool MIX>
cudaError_t run(const harts_plan *P, ScanParams &p, const void *const (&in)[4], bool precise, void *ws, size_t bytes, cudaStream_t st) {
    const int64_t C = P->info.C;
    if (one_step(P)) {
        const int64_t n = C * p.D;
        return launch(scan_step_kernel<T, BWD, MIX>, (n / Lane<T>::n + 127) / 128, 128, 0, 1, false, st, p, static_cast<const T *>(in[0]),
                      static_cast<const T *>(in[1]), static_cast<const T *>(in[3]), n);
    }
    for (int i = 0; i < Ring<BWD, false>::tensors; ++i)
        if (!map_rows<T>(&p.map[i], in[i], C, p.D)) return cudaErrorInvalidValue;
    if (p.ticket) {
        const cudaError_t e = cudaMemsetAsync(ws, 0xff, bytes, st);
        if (e != cudaSuccess) return e;
    }
    if constexpr (!MIX && std::is_same<T, __nv_bfloat16>::value)
        if (!precise && P->image.scan_longest <= kFastRows) return launch_scan<T, BWD, MIX, kFast, false>(p, st);
    constexpr int KIND = !MIX ? kExact : BWD ? kBoth : kRest;
    if constexpr (!BWD)
        if (P->image.scan_longest >= kAheadRows) return launch_scan<T, BWD, MIX, KIND, true>(p, st);
    return launch_scan<T, BWD, MIX, KIND, false>(p, st);
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

int check(const harts_plan *P, const harts_scan_fwd_args *a) {
    if (!P || !a) { set_error("NULL plan or args"); return HARTS_EINVAL; }
    if (a->dtype != HARTS_FP32 && a->dtype != HARTS_BF16) { set_error("dtype"); return HARTS_EUNSUPPORTED; }
    if (a->channels < 8 || a->channels % 8) { set_error("channels must be a positive multiple of 8"); return HARTS_EINVAL; }
    if (a->form != HARTS_SCAN_ADD && a->form != HARTS_SCAN_MIX) { set_error("form must be 0 (add) or 1 (mix)"); return HARTS_EINVAL; }
    if (!a->x || !a->g || !a->h) { set_error("NULL x, g or h"); return HARTS_EINVAL; }
    if (!aligned16(a->x) || !aligned16(a->g) || !aligned16(a->h) || !aligned16(a->workspace)) {
        set_error("x, g, h and workspace must be 16-byte aligned");
        return HARTS_EINVAL;
    }
    if (a->h == a->x || a->h == a->g) { set_error("h may be neither x nor g"); return HARTS_EINVAL; }
    if (!aligned16(a->h0) || !aligned16(a->final_state)) { set_error("h0 and final_state must be 16-byte aligned"); return HARTS_EINVAL; }
    if (a->final_state && a->final_state == a->h0 && !one_step(P)) {
        set_error("final_state may be h0 only in a plan of single rows");
        return HARTS_EINVAL;
    }
    if (P->info.C > (int64_t(1) << 38) / a->channels) { set_error("tensor too large"); return HARTS_EOVERFLOW; }
    if (int64_t(P->image.n_scan) * ceil_div(a->channels, wide_of(a->dtype)) > 0x7fffffff) {
        set_error("more tiles than the library counts");
        return HARTS_EOVERFLOW;
    }
    return HARTS_OK;
}

// What comes last: the plan's tables, and the workspace.
int check_space(const harts_plan *P, const harts_scan_fwd_args *a) {
    if (!P->dev) { set_error("plan not uploaded (harts_plan_upload)"); return HARTS_ENOPLAN; }
    const size_t need = space_of(P, a->channels, a->dtype).total;
    if (need && (!a->workspace || a->workspace_bytes < need)) {
        set_error("workspace too small");
        return HARTS_ESMALLBUF;
    }
    return HARTS_OK;
}

ScanParams params_of(const harts_plan *P, const harts_scan_fwd_args *a, bool backward) {
    ScanParams p;
    std::memset(&p, 0, sizeof(p));
    const Space s = space_of(P, a->channels, a->dtype);
    uint8_t *ws = static_cast<uint8_t *>(a->workspace);
    p.cols = ceil_div(a->channels, wide_of(a->dtype));
    p.group = kScanGroups[backward || p.cols <= 2 ? 2 : p.cols <= 8];
    p.tiles = backward ? P->view.scan_bwd : P->view.scan_fwd;
    p.next = P->view.scan_next;
    p.h0 = a->h0;
    if (!P->image.scan_alone) {
        p.ticket = reinterpret_cast<uint32_t *>(ws);
        p.inc = reinterpret_cast<float *>(ws + s.inc);
        p.agg = reinterpret_cast<float2 *>(ws + s.agg);
    }
    p.error = P->view.err;
    p.D = a->channels;
    p.width = p.cols * wide_of(a->dtype);
    p.total = static_cast<uint32_t>(P->image.n_scan) * p.cols;
    return p;
}

template <bool BWD>
cudaError_t dispatch(const harts_plan *P, const harts_scan_fwd_args *a, ScanParams &p, const void *const (&in)[4], bool precise, cudaStream_t st) {
    const size_t bytes = space_of(P, a->channels, a->dtype).total;
    if (a->dtype == HARTS_BF16)
        return a->form == HARTS_SCAN_MIX ? run<__nv_bfloat16, BWD, true>(P, p, in, precise, a->workspace, bytes, st)
                                         : run<__nv_bfloat16, BWD, false>(P, p, in, precise, a->workspace, bytes, st);
    return a->form == HARTS_SCAN_MIX ? run<float, BWD, true>(P, p, in, precise, a->workspace, bytes, st)
                                     : run<float, BWD, false>(P, p, in, precise, a->workspace, bytes, st);
}

int cuda_fail(cudaError_t e, const char *what) {
    set_error(std::string(what) + ": " + cudaGetErrorString(e));
    return HARTS_ECUDA;
}

}  // namespace
}  // namespace harts

using namespace harts;

extern "C" {

size_t harts_scan_workspace_bytes(const harts_plan *P, int32_t channels, int32_t dtype) {
    if (!P || channels < 8 || channels % 8 || (dtype != HARTS_FP32 && dtype != HARTS_BF16)) return 0;
    return space_of(P, channels, dtype).total;
}

int harts_scan_fwd(const harts_plan *P, const harts_scan_fwd_args *a, harts_stream_t stream) {
    int rc = check(P, a);
    if (!rc) rc = check_space(P, a);
    if (rc) return rc;
    ScanParams p = params_of(P, a, false);
    p.out0 = a->h;
    p.final_state = a->final_state;
    const void *in[4] = {a->g, a->x, nullptr, nullptr};
    const cudaError_t e = dispatch<false>(P, a, p, in, a->final_state != nullptr, reinterpret_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "scan forward");
    set_error("");
    return HARTS_OK;
}

int harts_scan_bwd(const harts_plan *P, const harts_scan_bwd_args *a, harts_stream_t stream) {
    if (!a) { set_error("NULL args"); return HARTS_EINVAL; }
    int rc = check(P, &a->fwd);
    if (rc) return rc;
    if (!a->d_h || !a->dx || !a->dg) { set_error("NULL d_h, dx or dg"); return HARTS_EINVAL; }
    if (!aligned16(a->d_h) || !aligned16(a->dx) || !aligned16(a->dg)) { set_error("d_h, dx and dg must be 16-byte aligned"); return HARTS_EINVAL; }
    const void *const in_use[] = {a->fwd.x, a->fwd.g, a->fwd.h, a->d_h};
    for (const void *q : in_use)
        if (a->dx == q || a->dg == q || a->dx == a->dg) { set_error("dx and dg may be none of the inputs"); return HARTS_EINVAL; }
    if (!aligned16(a->d_final) || !aligned16(a->dh0)) { set_error("d_final and dh0 must be 16-byte aligned"); return HARTS_EINVAL; }
    if (a->dh0 && a->dh0 == a->d_final && !one_step(P)) {
        set_error("dh0 may be d_final only in a plan of single rows");
        return HARTS_EINVAL;
    }
    if (a->dh0 && a->dh0 == a->fwd.h0) { set_error("dh0 may not be h0"); return HARTS_EINVAL; }
    rc = check_space(P, &a->fwd);
    if (rc) return rc;
    ScanParams p = params_of(P, &a->fwd, true);
    p.h_in = a->fwd.h;
    p.x_in = a->fwd.x;
    p.out0 = a->dx;
    p.out1 = a->dg;
    p.d_final = a->d_final;
    p.dh0 = a->dh0;
    const void *in[4] = {a->fwd.g, a->d_h, a->fwd.h, a->fwd.x};
    const cudaError_t e = dispatch<true>(P, &a->fwd, p, in, a->dh0 != nullptr, reinterpret_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "scan backward");
    set_error("");
    return HARTS_OK;
}

}  // extern "C"
