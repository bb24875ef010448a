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
// joins the eight and publishes the tile's map; the eight then fetch the maps of the tiles before
// it in its group, four each (up to 32 of a segment, which need not wait for one another), from
// which the ninth forms the carry with the state that the group before left.  So a chain waits once for 4,096 rows.  The order in which maps are joined is fixed
// by position: no atomics on values, the same bits on every run.  What is published carries its
// own validity: the workspace starts as all ones, a NaN that no published value has.  Tiles are
// taken in an order that has predecessors first, by a ticket counter, so that whatever a block
// waits for is in the hands of a running one; every wait is bounded all the same.
#include <algorithm>
#include <cstring>
#include <type_traits>

#include "kda_common.cuh"
#include "launch_util.h"
#include "tc_primitives.cuh"
#include "tensor_map.h"

namespace harts {
namespace {

constexpr int kWarps = 8, kWarpRows = kScanRows / kWarps;      // consumers
constexpr int kThreads = 32 * (kWarps + 2);                    // and a warp each for carries and copies
constexpr int kShare = kScanGroup / kWarps;                    // tiles of a group whose maps one consumer joins
constexpr int kBox = 16;                                       // rows of one copy
constexpr uint32_t kTileBytes = kScanRows * 128;               // of one tensor
constexpr uint32_t kEmpty = 0xffffffffu;                       // not published yet

struct ScanParams {
    CUtensorMap map[4];             // forward g, x; backward g, dh, h, x (mix)
    const ScanTile *tiles;
    const int32_t *next;
    const float *h0, *d_final;
    const void *h_in;               // backward: h
    void *out0, *out1;              // forward h; backward dx, dg
    float *final_state, *dh0;
    uint32_t *ticket;               // nullptr: tiles that wait for nothing are dealt out in turn
    float *inc;                     // [groups][width] state behind a group (backward: before it)
    float2 *agg;                    // [tiles][width] a tile's map
    int32_t *error;
    int32_t D, width, cols;         // channels, rounded up to tiles', tiles across
    uint32_t total;
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// e^g for g <= 0, as one number that gives both a and 1 - a with few roundings: a itself, or, from
// e^(-0.3466) = 2^(-1/2) up, -(1 - a) with its sign bit set.  2^y = 2^n 2^f with |f| <= 1/2 and the
// series of e^(f ln 2) to its seventh power (the next term is 5e-9).  Memories of a thousand rows
// multiply a thousand decays: an approximate exponential's 2^-22 would be 2e-4 of the state.
// Without PRECISE (bf16 results of the add form, which round to 2^-9) that is enough, and a is kept.
template <bool PRECISE> __device__ __forceinline__ float decay(float g) {
    if constexpr (!PRECISE) return ex2(g * 1.4426950408889634f);
    const float z = fmaf(g, 1.4426950408889634f, 12582912.f), n = z - 12582912.f;
    const float f = fmaf(g, 1.9259629911e-8f, fmaf(g, 1.4426950216293335f, -n));
    float q = 1.5252733804e-5f;
    q = fmaf(q, f, 1.5403530394e-4f);
    q = fmaf(q, f, 1.3333558146e-3f);
    q = fmaf(q, f, 9.6181291076e-3f);
    q = fmaf(q, f, 5.5504108665e-2f);
    q = fmaf(q, f, 2.4022650696e-1f);
    q = fmaf(q, f, 6.9314718056e-1f);
    const float t = q * f;
    const float scale = __int_as_float((__float_as_int(z) - 0x4b400000 + 127) << 23);
    float a = fmaf(t, scale, scale);
    if (n == 0.f) a = -fabsf(t);
    return g < -87.f ? 0.f : a;
}
template <bool PRECISE> __device__ __forceinline__ float keep_of(float v) {      // a
    if constexpr (!PRECISE) return v;
    return __float_as_int(v) < 0 && v == v ? 1.f + v : v;
}
__device__ __forceinline__ float rest_of(float v) { return __float_as_int(v) < 0 ? -v : 1.f - v; }     // 1 - a

template <typename T> struct Lane;                             // the channels of a lane: 4 bytes
template <> struct Lane<__nv_bfloat16> {
    static constexpr int n = 2;
    __device__ __forceinline__ static void get(const uint8_t *p, float (&v)[2]) {
        const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(p));
        v[0] = f.x; v[1] = f.y;
    }
    __device__ __forceinline__ static void put(void *p, const float (&v)[2]) {
        *reinterpret_cast<__nv_bfloat162 *>(p) = __floats2bfloat162_rn(v[0], v[1]);
    }
};
template <> struct Lane<float> {
    static constexpr int n = 1;
    __device__ __forceinline__ static void get(const uint8_t *p, float (&v)[1]) { v[0] = *reinterpret_cast<const float *>(p); }
    __device__ __forceinline__ static void put(void *p, const float (&v)[1]) { *static_cast<float *>(p) = v[0]; }
};

__device__ __forceinline__ uint32_t publishable(float v) { return v == v ? __float_as_uint(v) : 0x7fffffffu; }
__device__ __forceinline__ void publish(float2 *at, float a, float b) {
    const uint64_t u = static_cast<uint64_t>(publishable(b)) << 32 | publishable(a);
    asm volatile("st.relaxed.gpu.global.b64 [%0], %1;" :: "l"(at), "l"(u) : "memory");
}
__device__ __forceinline__ void publish(float *at, float v) {
    asm volatile("st.relaxed.gpu.global.b32 [%0], %1;" :: "l"(at), "r"(publishable(v)) : "memory");
}
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

// What is published at `at`, waiting for it; zeros once a wait of the block has run out.
template <typename V> __device__ __forceinline__ V await(const V *at, int *failed) {
    V v = look(at);
    if (is_there(v)) return v;
    const long long t0 = clock64();
    while (!gave_up(failed)) {
        v = look(at);
        if (is_there(v)) return v;
        if (clock64() - t0 > 4000000000LL) *reinterpret_cast<volatile int *>(failed) = 1;
    }
    return V{};
}

__device__ __forceinline__ void arrive(uint64_t *bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" :: "r"(tc::smem_addr(bar)) : "memory");
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
// memory holds.
template <bool BWD, bool MIX> struct Ring {
    static constexpr int tensors = BWD ? (MIX ? 4 : 3) : 2;
    static constexpr int stages = BWD && MIX ? 3 : 2;
    static constexpr int blocks = BWD ? (MIX ? 1 : 2) : 3;
    static constexpr uint32_t stage_bytes = tensors * kTileBytes;
    static constexpr uint32_t smem = stages * stage_bytes + 128;
};

struct Meta { ScanTile t; int32_t col; };                      // rows 0: the end

template <typename T, bool BWD, bool MIX, bool PRECISE>
__global__ void __launch_bounds__(kThreads, Ring<BWD, MIX>::blocks) scan_kernel(const __grid_constant__ ScanParams p) {
    using R = Ring<BWD, MIX>;
    constexpr int CH = Lane<T>::n, kWide = 32 * CH;
    extern __shared__ uint8_t smraw[];
    uint8_t *sm = smraw + ((128 - (tc::smem_addr(smraw) & 127)) & 127);
    __shared__ uint64_t full[R::stages], empty[R::stages];
    __shared__ Meta meta[R::stages];
    __shared__ float2 s_map[2][kWarps][kWide];                 // the warps' maps, by tile parity
    __shared__ float2 s_pre[kWarps][kWide];                    // maps of the tiles before this one, each of kShare of them
    __shared__ float s_carry[kWide];
    __shared__ uint64_t maps_full, pre_full, carry_full;
    __shared__ int s_fail;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < R::stages; ++s) { tc::mbar_init(&full[s], 1); tc::mbar_init(&empty[s], kWarps + 1); }
        tc::mbar_init(&maps_full, kWarps);
        tc::mbar_init(&pre_full, kWarps);
        tc::mbar_init(&carry_full, 1);
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
                m.t = p.tiles[idx / p.cols];
                m.col = static_cast<int32_t>(idx % p.cols) * kWide;
                if (p.ticket) drawn = draw();
            }
            if (it >= R::stages && !warp_wait(&empty[s], (it / R::stages - 1) & 1, &s_fail)) break;
            const int boxes = (m.t.rows + kBox - 1) / kBox;
            if (lane == 0) {
                meta[s] = m;
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
        // carries
        uint32_t uses = 0;
        for (uint32_t it = 0;; ++it) {
            const int s = it % R::stages;
            if (!warp_wait(&full[s], (it / R::stages) & 1, &s_fail)) break;
            const Meta m = meta[s];
            if (m.t.rows == 0 || !warp_wait(&maps_full, it & 1, &s_fail)) break;
            float A[CH], B[CH];
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                A[c] = 1.f; B[c] = 0.f;
#pragma unroll
                for (int k = 0; k < kWarps; ++k) {
                    const float2 w = s_map[it & 1][BWD ? kWarps - 1 - k : k][lane * CH + c];
                    B[c] = fmaf(w.x, B[c], w.y);
                    A[c] *= w.x;
                }
            }
            const int64_t ch = m.col + lane * CH;
            float2 *agg = p.agg + static_cast<int64_t>(m.t.tile) * p.width + ch;
            if (BWD ? m.t.at > 0 : m.t.at < m.t.count - 1) {
#pragma unroll
                for (int c = 0; c < CH; ++c) publish(agg + c, A[c], B[c]);
            }
            float v[CH];
#pragma unroll
            for (int c = 0; c < CH; ++c) v[c] = 0.f;
            if (!BWD) {
                if (m.t.pred >= 0) {
#pragma unroll
                    for (int c = 0; c < CH; ++c) v[c] = await(p.inc + static_cast<int64_t>(m.t.pred) * p.width + ch + c, &s_fail);
                } else if (p.h0) {
#pragma unroll
                    for (int c = 0; c < CH; ++c)
                        if (ch + c < p.D) v[c] = p.h0[static_cast<int64_t>(-1 - m.t.pred) * p.D + ch + c];
                }
            } else {
                for (int k = 0; k < m.t.next_count; ++k) {
                    const int64_t g = p.next[m.t.next_begin + k];
#pragma unroll
                    for (int c = 0; c < CH; ++c) v[c] += await(p.inc + g * p.width + ch + c, &s_fail);
                }
                if (p.d_final && m.t.seq_end >= 0) {
#pragma unroll
                    for (int c = 0; c < CH; ++c)
                        if (ch + c < p.D) v[c] += p.d_final[static_cast<int64_t>(m.t.seq_end) * p.D + ch + c];
                }
            }
            const int between = BWD ? m.t.count - 1 - m.t.at : m.t.at;
            if (between > 0) {
                if (!warp_wait(&pre_full, uses++ & 1, &s_fail)) break;
                for (int k = BWD ? (m.t.count - 1) / kShare : 0; BWD ? k >= (m.t.at + 1) / kShare : k <= (m.t.at - 1) / kShare; k += BWD ? -1 : 1) {
#pragma unroll
                    for (int c = 0; c < CH; ++c) {
                        const float2 w = s_pre[k][lane * CH + c];
                        v[c] = fmaf(w.x, v[c], w.y);
                    }
                }
            }
#pragma unroll
            for (int c = 0; c < CH; ++c) s_carry[lane * CH + c] = v[c];
            __syncwarp();
            if (lane == 0) arrive(&carry_full);
#pragma unroll
            for (int c = 0; c < CH; ++c) v[c] = fmaf(A[c], v[c], B[c]);
            if (!BWD) {
                if (m.t.at == m.t.count - 1 && m.t.next_count > 0) {
#pragma unroll
                    for (int c = 0; c < CH; ++c) publish(p.inc + static_cast<int64_t>(m.t.group) * p.width + ch + c, v[c]);
                }
            } else if (m.t.at == 0) {
                if (m.t.pred >= 0) {
#pragma unroll
                    for (int c = 0; c < CH; ++c) publish(p.inc + static_cast<int64_t>(m.t.group) * p.width + ch + c, v[c]);
                } else if (p.dh0) {
#pragma unroll
                    for (int c = 0; c < CH; ++c)
                        if (ch + c < p.D) p.dh0[static_cast<int64_t>(-1 - m.t.pred) * p.D + ch + c] = v[c];
                }
            }
            __syncwarp();
            if (lane == 0) arrive(&empty[s]);
        }
    } else {
        for (uint32_t it = 0;; ++it) {
            const int s = it % R::stages;
            if (!warp_wait(&full[s], (it / R::stages) & 1, &s_fail)) break;
            const int rows = meta[s].t.rows, row0 = meta[s].t.row0;
            if (rows == 0) break;
            const int mine = min(max(rows - warp * kWarpRows, 0), kWarpRows);
            const uint8_t *src = sm + s * R::stage_bytes + warp * kWarpRows * 128 + lane * 4;
            const int64_t ch = meta[s].col + lane * CH;
            [[maybe_unused]] float hp[CH] = {};                // state before the tile's first row
            if (BWD && warp == 0 && ch < p.D) {
                const int32_t pr = meta[s].t.pred_row;
                if (pr >= 0) {
                    Lane<T>::get(reinterpret_cast<const uint8_t *>(static_cast<const T *>(p.h_in) + static_cast<int64_t>(pr) * p.D + ch), hp);
                } else if (p.h0) {
#pragma unroll
                    for (int c = 0; c < CH; ++c) hp[c] = p.h0[static_cast<int64_t>(-1 - pr) * p.D + ch + c];
                }
            }
            float d[kWarpRows][CH], A[CH], B[CH];
#pragma unroll
            for (int c = 0; c < CH; ++c) { A[c] = 1.f; B[c] = 0.f; }
#pragma unroll
            for (int k = 0; k < kWarpRows; ++k) {
                const int i = BWD ? kWarpRows - 1 - k : k;
                if (i < mine) {
                    float g[CH], u[CH];
                    Lane<T>::get(src + i * 128, g);
                    Lane<T>::get(src + kTileBytes + i * 128, u);
#pragma unroll
                    for (int c = 0; c < CH; ++c) {
                        d[i][c] = decay<PRECISE>(g[c]);
                        const float a = keep_of<PRECISE>(d[i][c]);
                        if (BWD) B[c] = a * (u[c] + B[c]);
                        else B[c] = fmaf(a, B[c], MIX ? rest_of(d[i][c]) * u[c] : u[c]);
                        A[c] *= a;
                    }
                }
            }
#pragma unroll
            for (int c = 0; c < CH; ++c) s_map[it & 1][warp][lane * CH + c] = make_float2(A[c], B[c]);
            __syncwarp();
            if (lane == 0) arrive(&maps_full);
            const ScanTile &t = meta[s].t;
            if (BWD ? t.at < t.count - 1 : t.at > 0) {
                // this warp's share of the tiles between the group's carry and this tile
                const int lo = max(warp * kShare, BWD ? t.at + 1 : 0), hi = min(warp * kShare + kShare, BWD ? t.count : t.at);
                const float2 *at = p.agg + static_cast<int64_t>(t.tile - t.at) * p.width + meta[s].col + lane * CH;
                float2 w[kShare][CH];
#pragma unroll
                for (int k = 0; k < kShare; ++k) {
                    const int i = warp * kShare + k;
#pragma unroll
                    for (int c = 0; c < CH; ++c)
                        w[k][c] = i >= lo && i < hi ? look(at + static_cast<int64_t>(i) * p.width + c) : make_float2(1.f, 0.f);
                }
#pragma unroll
                for (int c = 0; c < CH; ++c) { A[c] = 1.f; B[c] = 0.f; }
#pragma unroll
                for (int k = 0; k < kShare; ++k) {
                    const int j = BWD ? kShare - 1 - k : k, i = warp * kShare + j;
#pragma unroll
                    for (int c = 0; c < CH; ++c) {
                        if (!is_there(w[j][c])) w[j][c] = await(at + static_cast<int64_t>(i) * p.width + c, &s_fail);
                        if (i >= lo && i < hi) {
                            B[c] = fmaf(w[j][c].x, B[c], w[j][c].y);
                            A[c] *= w[j][c].x;
                        }
                    }
                }
#pragma unroll
                for (int c = 0; c < CH; ++c) s_pre[warp][lane * CH + c] = make_float2(A[c], B[c]);
                __syncwarp();
                if (lane == 0) arrive(&pre_full);
            }
            if (!warp_wait(&carry_full, it & 1, &s_fail)) break;
            float v[CH];
#pragma unroll
            for (int c = 0; c < CH; ++c) v[c] = s_carry[lane * CH + c];
            for (int k = BWD ? kWarps - 1 : 0; k != warp; k += BWD ? -1 : 1) {
#pragma unroll
                for (int c = 0; c < CH; ++c) {
                    const float2 w = s_map[it & 1][k][lane * CH + c];
                    v[c] = fmaf(w.x, v[c], w.y);
                }
            }
            if (ch < p.D) {
                const int64_t at = static_cast<int64_t>(row0 + warp * kWarpRows) * p.D + ch;
                T *out0 = static_cast<T *>(p.out0) + at, *out1 = static_cast<T *>(p.out1) + at;
#pragma unroll
                for (int k = 0; k < kWarpRows; ++k) {
                    const int i = BWD ? kWarpRows - 1 - k : k;
                    if (i < mine) {
                        float u[CH];
                        Lane<T>::get(src + kTileBytes + i * 128, u);
                        if constexpr (!BWD) {
#pragma unroll
                            for (int c = 0; c < CH; ++c)
                                v[c] = fmaf(keep_of<PRECISE>(d[i][c]), v[c], MIX ? rest_of(d[i][c]) * u[c] : u[c]);
                            Lane<T>::put(out0 + static_cast<int64_t>(i) * p.D, v);
                        } else {
                            float h[CH], x[CH], dx[CH], dg[CH];
                            Lane<T>::get(src + 2 * kTileBytes + i * 128, h);
                            if (MIX) Lane<T>::get(src + 3 * kTileBytes + i * 128, x);
#pragma unroll
                            for (int c = 0; c < CH; ++c) {
                                if (i == 0 && warp == 0) h[c] = hp[c];
                                const float lam = u[c] + v[c];
                                v[c] = keep_of<PRECISE>(d[i][c]) * lam;
                                dx[c] = MIX ? rest_of(d[i][c]) * lam : lam;
                                dg[c] = v[c] * (MIX ? h[c] - x[c] : h[c]);
                            }
                            Lane<T>::put(out0 + static_cast<int64_t>(i) * p.D, dx);
                            Lane<T>::put(out1 + static_cast<int64_t>(i) * p.D, dg);
                        }
                    }
                }
                if (!BWD && p.final_state && meta[s].t.seq_end >= 0 && meta[s].t.at == meta[s].t.count - 1 && mine > 0 &&
                    rows - warp * kWarpRows <= kWarpRows) {
#pragma unroll
                    for (int c = 0; c < CH; ++c) p.final_state[static_cast<int64_t>(meta[s].t.seq_end) * p.D + ch + c] = v[c];
                }
            }
            __syncwarp();
            if (lane == 0) arrive(&empty[s]);
        }
    }
    __syncthreads();
    if (threadIdx.x == 0 && s_fail) atomicCAS(p.error, 0, static_cast<int>(kDevErrTimeout));
}

// Every segment a root of one row (a decoding step): row, root and sequence have one number.
template <typename T, bool BWD, bool MIX>
__global__ void __launch_bounds__(128) scan_step_kernel(const __grid_constant__ ScanParams p, const T *g, const T *u, const T *x, int64_t n) {
    constexpr int CH = Lane<T>::n;
    const int64_t i = (static_cast<int64_t>(blockIdx.x) * 128 + threadIdx.x) * CH;
    if (i >= n) return;
    float gv[CH], uv[CH], xv[CH], o0[CH], o1[CH];
    Lane<T>::get(reinterpret_cast<const uint8_t *>(g + i), gv);
    Lane<T>::get(reinterpret_cast<const uint8_t *>(u + i), uv);
    if (BWD && MIX) Lane<T>::get(reinterpret_cast<const uint8_t *>(x + i), xv);
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const float d = decay<true>(gv[c]), a = keep_of<true>(d), h = p.h0 ? p.h0[i + c] : 0.f;
        if (!BWD) {
            o0[c] = fmaf(a, h, MIX ? rest_of(d) * uv[c] : uv[c]);
            if (p.final_state) p.final_state[i + c] = o0[c];
        } else {
            const float lam = uv[c] + (p.d_final ? p.d_final[i + c] : 0.f);
            o0[c] = MIX ? rest_of(d) * lam : lam;
            o1[c] = a * lam * (MIX ? h - xv[c] : h);
            if (p.dh0) p.dh0[i + c] = a * lam;
        }
    }
    Lane<T>::put(static_cast<T *>(p.out0) + i, o0);
    if (BWD) Lane<T>::put(static_cast<T *>(p.out1) + i, o1);
}

// ---- host ---------------------------------------------------------------------------------

size_t align256(size_t x) { return (x + 255) / 256 * 256; }
int32_t wide_of(int32_t dtype) { return dtype == HARTS_BF16 ? 64 : 32; }
bool one_step(const harts_plan *P) { return P->info.n_seg == P->info.C && P->info.n_roots == P->info.n_seg; }

struct Space { size_t inc, agg, total; };       // behind 256 bytes with the ticket counter
Space space_of(const harts_plan *P, int32_t D, int32_t dtype) {
    const size_t width = size_t(ceil_div(D, wide_of(dtype))) * wide_of(dtype);
    Space s{};
    if (P->image.scan_alone) { s.total = 256; return s; }
    s.inc = 256;
    s.agg = s.inc + align256(4 * width * P->image.n_scan_groups);
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

template <typename T, bool BWD, bool MIX, bool PRECISE>
cudaError_t launch_scan(const ScanParams &p, cudaStream_t st) {
    using R = Ring<BWD, MIX>;
    static std::atomic<uint64_t> done{0};
    auto *k = scan_kernel<T, BWD, MIX, PRECISE>;
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
    for (int i = 0; i < Ring<BWD, MIX>::tensors; ++i)
        if (!map_rows<T>(&p.map[i], in[i], C, p.D)) return cudaErrorInvalidValue;
    if (p.ticket) {
        const cudaError_t e = cudaMemsetAsync(ws, 0xff, bytes, st);
        if (e != cudaSuccess) return e;
    }
    if constexpr (!MIX && std::is_same<T, __nv_bfloat16>::value)
        if (!precise) return launch_scan<T, BWD, MIX, false>(p, st);
    return launch_scan<T, BWD, MIX, true>(p, st);
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3) == 0; }

int check(const harts_plan *P, const harts_scan_fwd_args *a) {
    if (!P || !a) { set_error("NULL plan or args"); return HARTS_EINVAL; }
    if (!P->dev) { set_error("plan not uploaded (harts_plan_upload)"); return HARTS_ENOPLAN; }
    if (a->dtype != HARTS_FP32 && a->dtype != HARTS_BF16) { set_error("dtype"); return HARTS_EUNSUPPORTED; }
    if (a->channels < 8 || a->channels % 8) { set_error("channels must be a positive multiple of 8"); return HARTS_EINVAL; }
    if (a->form != HARTS_SCAN_ADD && a->form != HARTS_SCAN_MIX) { set_error("form must be 0 (add) or 1 (mix)"); return HARTS_EINVAL; }
    if (!a->x || !a->g || !a->h) { set_error("NULL x, g or h"); return HARTS_EINVAL; }
    if (!aligned16(a->x) || !aligned16(a->g) || !aligned16(a->h) || !aligned16(a->workspace)) {
        set_error("x, g, h and workspace must be 16-byte aligned");
        return HARTS_EINVAL;
    }
    if (a->h == a->x || a->h == a->g) { set_error("h may be neither x nor g"); return HARTS_EINVAL; }
    if (!aligned4(a->h0) || !aligned4(a->final_state)) { set_error("h0 and final_state must be aligned to their type"); return HARTS_EINVAL; }
    if (P->info.C > (int64_t(1) << 38) / a->channels) { set_error("tensor too large"); return HARTS_EOVERFLOW; }
    if (int64_t(P->image.n_scan) * ceil_div(a->channels, wide_of(a->dtype)) > 0x7fffffff) {
        set_error("more tiles than the library counts");
        return HARTS_EOVERFLOW;
    }
    if (!a->workspace || a->workspace_bytes < space_of(P, a->channels, a->dtype).total) {
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
    p.cols = ceil_div(a->channels, wide_of(a->dtype));
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
    const int rc = check(P, a);
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
    const int rc = check(P, &a->fwd);
    if (rc) return rc;
    if (!a->d_h || !a->dx || !a->dg) { set_error("NULL d_h, dx or dg"); return HARTS_EINVAL; }
    if (!aligned16(a->d_h) || !aligned16(a->dx) || !aligned16(a->dg)) { set_error("d_h, dx and dg must be 16-byte aligned"); return HARTS_EINVAL; }
    const void *const in_use[] = {a->fwd.x, a->fwd.g, a->fwd.h, a->d_h};
    for (const void *q : in_use)
        if (a->dx == q || a->dg == q || a->dx == a->dg) { set_error("dx and dg may be none of the inputs"); return HARTS_EINVAL; }
    if (!aligned4(a->d_final) || !aligned4(a->dh0)) { set_error("d_final and dh0 must be aligned to their type"); return HARTS_EINVAL; }
    ScanParams p = params_of(P, &a->fwd, true);
    p.h_in = a->fwd.h;
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
