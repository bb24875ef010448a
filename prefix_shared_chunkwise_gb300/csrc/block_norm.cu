// The norm behind a block with its gate and the residual's scaled addition, and the norm before the
// next block, in one pass, forward and backward.
//
//   r1 = 1 / sqrt(mean_j y_j^2 + eps),  u = y r1 w1   (u = y without a norm behind the block)
//   h = res + scale act(gate) u,   r2 = 1 / sqrt(mean_j h_j^2 + eps),  n = h r2 w2
// Backward, with D the gradient of h: D = dh + r2 (w2 dn - N mean_j(w2_j dn_j N_j)), N = h r2,
//   dres = D,  dgate = scale D u act'(gate),  e = scale D act(gate),
//   dy = r1 (w1 e - Y mean_j(w1_j e_j Y_j)),  Y = y r1,   dw1 = sum_rows e Y,  dw2 = sum_rows dn N
// Sums and statistics are fp32; h is normalised before its own rounding to the stream's type, so
// that n carries one rounding.  The backward reads the rounded h that the forward stored.
//
// Five streams forward and eight backward are read or written once each, with some 20 operations a
// value: HBM bounds both.  (As separate steps the norm, the gate, the addition and the next norm
// would move twelve.)  A row belongs to R threads, which keep it in registers over both of its
// sums.  Rows of 1 KB and more are copied ahead by cp.async.bulk into a ring in shared memory,
// whose bytes on their way do not depend on registers; shorter rows share a warp, and the next
// ones are loaded into registers ahead.  Blocks are persistent: weights and the weights' gradients
// of a thread's columns stay in its registers.  A block leaves one row of those gradients, a second
// kernel adds them in ascending order: no atomics, the same bits on every run.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstring>

#include "kda_common.cuh"
#include "launch_util.h"
#include "rows.cuh"
#include "tc_primitives.cuh"

namespace harts {
namespace {

using namespace rows;

constexpr int kMaxDim = 8192;       // 1024 threads x 8 values
constexpr int kMaxStages = 4;       // rows copied ahead

struct Fwd {
    const void *in[3];              // y; gate; residual
    const float *w1, *w2;
    void *h, *n;
    float *r1, *r2;
    int32_t *error;
    int64_t C;
    int32_t D, act;
    float scale, eps;
};

struct Bwd {
    const void *in[5];              // y; gate; dn; h; dh
    const float *w1, *w2, *r1, *r2;
    void *dy, *dgate, *dres;
    float *part;                    // [groups][2 D]: of w1, of w2
    int32_t *error;
    int64_t C;
    int32_t D, act;
    float scale;
};

// sigmoid(z) and sigmoid(-z), both from e^-|z|, which neither overflows nor is lost in a 1.
__device__ __forceinline__ float sigmoid(float z, float &other) {
    const float t = __expf(-fabsf(z)), big = __fdividef(1.f, 1.f + t), small = t * big;
    other = z < 0.f ? big : small;
    return z < 0.f ? small : big;
}
__device__ __forceinline__ float gate_of(float z, int act, float &slope) {
    slope = 1.f;
    if (act == HARTS_GATE_LINEAR) return z;
    float rest;
    const float q = sigmoid(z, rest);
    slope = act == HARTS_GATE_SILU ? q * fmaf(z, rest, 1.f) : q * rest;
    return act == HARTS_GATE_SILU ? z * q : q;
}

// Rows of a block on their way into shared memory: the N tensors that are there, row after row.
// Thread 0 fetches; a wait that runs out is reported once and never waited for again, and the block
// goes on with what its shared memory holds, so that its barriers stay matched.
template <typename T, int N> struct Ahead {
    uint8_t *mem;
    uint64_t *full;
    int *fail;
    uint32_t bytes, stage;
    int stages, s;
    uint32_t phase;
    __device__ __forceinline__ void fetch(const void *const (&in)[N], int64_t row, int32_t D, int slot) {
        uint8_t *dst = mem + slot * stage;
        tc::mbar_expect_tx(&full[slot], stage);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if (!in[i]) continue;
            bulk_load(dst, static_cast<const T *>(in[i]) + row * D, bytes, &full[slot]);
            dst += bytes;
        }
    }
    __device__ __forceinline__ void wait(int32_t *error) {
        if (tc::mbar_try(&full[s], phase) || *reinterpret_cast<volatile int *>(fail)) return;
        if (!tc::mbar_wait(&full[s], phase)) {
            *reinterpret_cast<volatile int *>(fail) = 1;
            atomicCAS(error, 0, static_cast<int>(kDevErrTimeout));
        }
    }
    __device__ __forceinline__ void next() { if (++s == stages) { s = 0; phase ^= 1; } }
    __device__ __forceinline__ void drain() {               // copies in flight, after a failure
        if (!*reinterpret_cast<volatile int *>(fail)) return;
        for (int i = 0; i < stages; ++i) tc::mbar_wait(&full[i], 0, 100000000LL), tc::mbar_wait(&full[i], 1, 100000000LL);
    }
};

template <typename T, int N>
__device__ __forceinline__ Ahead<T, N> begin_ahead(const void *const (&in)[N], int32_t D, int stages, uint8_t *mem, uint64_t *full,
                                                   int *fail, int64_t C) {
    Ahead<T, N> a;
    a.mem = mem; a.full = full; a.fail = fail; a.stages = stages; a.s = 0; a.phase = 0;
    a.bytes = static_cast<uint32_t>(D) * sizeof(T);
    a.stage = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) a.stage += in[i] ? a.bytes : 0;
    if (threadIdx.x == 0) {
        *fail = 0;
        for (int s = 0; s < stages; ++s) tc::mbar_init(&full[s], 1);
        tc::fence_mbar_init();
        for (int s = 0; s < stages; ++s)
            if (blockIdx.x + static_cast<int64_t>(s) * gridDim.x < C) a.fetch(in, blockIdx.x + static_cast<int64_t>(s) * gridDim.x, D, s);
    }
    __syncthreads();
    return a;
}

// RING: a block works on one row at a time, which has been copied into shared memory.
template <typename T, int VEC, int R, int NV, bool RING>
__global__ void __launch_bounds__(block_of(R)) block_norm_fwd_kernel(const Fwd p, int stages) {
    constexpr bool kKeep = R <= 512;
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ float sm[2][2][rows_of(R)][R < 32 ? 1 : R / 32];
    __shared__ uint64_t full[RING ? kMaxStages : 1];
    __shared__ int s_fail;
    const int t = threadIdx.x % R, sub = threadIdx.x / R;
    const int32_t D = p.D;
    const int64_t step = static_cast<int64_t>(gridDim.x) * rows_of(R);
    int64_t row = static_cast<int64_t>(blockIdx.x) * rows_of(R) + sub;
    const float inv_d = 1.f / static_cast<float>(D);
    Raw<T, VEC> a[3][NV];
    [[maybe_unused]] Ahead<T, 3> ahead;
    if constexpr (RING) ahead = begin_ahead<T, 3>(p.in, D, stages, ring, full, &s_fail, p.C);
    auto load = [&](int64_t r) {                                // without a ring: a row's values into registers
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int32_t col = (j * R + t) * VEC;
            if (col < D && r < p.C) {
#pragma unroll
                for (int i = 0; i < 3; ++i) if (p.in[i]) a[i][j] = ld<T, VEC>(p.in[i], r * D + col);
            }
        }
    };
    if constexpr (!RING) load(row);
    [[maybe_unused]] float w1[kKeep ? NV : 1][VEC], w2[kKeep ? NV : 1][VEC];
    if constexpr (kKeep) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int32_t col = (j * R + t) * VEC;
            if (col < D && p.w1) ld_w<VEC>(p.w1, col, w1[j]);
            if (col < D && p.w2) ld_w<VEC>(p.w2, col, w2[j]);
        }
    }
    auto weights = [&](const float *w, float (&kept)[kKeep ? NV : 1][VEC], int j, int32_t col, float (&v)[VEC]) {
        if constexpr (kKeep) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) v[i] = kept[j][i];
        } else {
            ld_w<VEC>(w, col, v);
        }
    };
    for (int slot = 0; row < p.C; row += step, slot ^= 1) {
        if constexpr (RING) {
            ahead.wait(p.error);
            const T *buf = reinterpret_cast<const T *>(ring + ahead.s * ahead.stage);
#pragma unroll
            for (int i = 0; i < 3; ++i) {
                if (!p.in[i]) continue;
#pragma unroll
                for (int j = 0; j < NV; ++j) {
                    const int32_t col = (j * R + t) * VEC;
                    if (col < D) a[i][j] = ld<T, VEC>(buf, col);
                }
                buf += D;
            }
        }
        float v[NV][VEC], g[NV][VEC], s = 0.f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            if ((j * R + t) * VEC >= D) continue;
            unpack(a[0][j], v[j]);
#pragma unroll
            for (int i = 0; i < VEC; ++i) s = fmaf(v[j][i], v[j][i], s);
            if (p.in[1]) {
                unpack(a[1][j], g[j]);
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    float slope;
                    g[j][i] = gate_of(g[j][i], p.act, slope);
                }
            } else {
#pragma unroll
                for (int i = 0; i < VEC; ++i) g[j][i] = 1.f;
            }
        }
        // behind a sum's barrier the stage is free; residuals are taken out of it before
        Raw<T, VEC> res[NV];
#pragma unroll
        for (int j = 0; j < NV; ++j) res[j] = a[2][j];
        auto free_stage = [&] {
            if constexpr (RING) {
                if (t == 0 && row + stages * step < p.C) ahead.fetch(p.in, row + stages * step, D, ahead.s);
            } else {
                load(row + step);
            }
        };
        float r1 = 1.f;
        if (p.w1) {
            r1 = __frsqrt_rn(fmaf(row_sum<R>(s, sm[slot][0][sub]), inv_d, p.eps));
            free_stage();
            if (t == 0 && p.r1) p.r1[row] = r1;
        }
        s = 0.f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int32_t col = (j * R + t) * VEC;
            if (col >= D) continue;
            if (p.w1) {
                float w[VEC];
                weights(p.w1, w1, j, col, w);
#pragma unroll
                for (int i = 0; i < VEC; ++i) v[j][i] = v[j][i] * r1 * w[i];
            }
#pragma unroll
            for (int i = 0; i < VEC; ++i) v[j][i] = v[j][i] * g[j][i] * p.scale;
            if (p.in[2]) {
                float x[VEC];
                unpack(res[j], x);
#pragma unroll
                for (int i = 0; i < VEC; ++i) v[j][i] += x[i];
            }
#pragma unroll
            for (int i = 0; i < VEC; ++i) s = fmaf(v[j][i], v[j][i], s);
            st<T, VEC>(p.h, row * D + col, v[j]);
        }
        if (p.w2) {
            const float r2 = __frsqrt_rn(fmaf(row_sum<R>(s, sm[slot][1][sub]), inv_d, p.eps));
            if (!p.w1) free_stage();
            if (t == 0 && p.r2) p.r2[row] = r2;
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int32_t col = (j * R + t) * VEC;
                if (col >= D) continue;
                float w[VEC];
                weights(p.w2, w2, j, col, w);
#pragma unroll
                for (int i = 0; i < VEC; ++i) v[j][i] = v[j][i] * r2 * w[i];
                st<T, VEC>(p.n, row * D + col, v[j]);
            }
        }
        if constexpr (RING) ahead.next();
    }
    if constexpr (RING) if (t == 0) ahead.drain();
}

template <typename T, int VEC, int R, int NV, bool RING>
__global__ void __launch_bounds__(block_of(R)) block_norm_bwd_kernel(const Bwd p, int stages) {
    constexpr bool kKeep = R <= 512;
    constexpr int kRows = rows_of(R);
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ float sm[2][2][kRows][R < 32 ? 1 : R / 32];
    __shared__ uint64_t full[RING ? kMaxStages : 1];
    __shared__ int s_fail;
    const int t = threadIdx.x % R, sub = threadIdx.x / R;
    const int32_t D = p.D;
    const int64_t step = static_cast<int64_t>(gridDim.x) * kRows;
    int64_t row = static_cast<int64_t>(blockIdx.x) * kRows + sub;
    const float inv_d = 1.f / static_cast<float>(D);
    let_next_start();
    Raw<T, VEC> a[5][NV];
    [[maybe_unused]] Ahead<T, 5> ahead;
    if constexpr (RING) ahead = begin_ahead<T, 5>(p.in, D, stages, ring, full, &s_fail, p.C);
    float next1 = 0.f, next2 = 0.f;
    auto load = [&](int64_t r) {
        if (r >= p.C) return;
        if (p.w1) next1 = __ldg(p.r1 + r);
        if (p.w2) next2 = __ldg(p.r2 + r);
        if constexpr (!RING) {
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int32_t col = (j * R + t) * VEC;
                if (col < D) {
#pragma unroll
                    for (int i = 0; i < 5; ++i) if (p.in[i]) a[i][j] = ld<T, VEC>(p.in[i], r * D + col);
                }
            }
        }
    };
    load(row);
    [[maybe_unused]] float w1[kKeep ? NV : 1][VEC], w2[kKeep ? NV : 1][VEC];
    float dw1[NV][VEC], dw2[NV][VEC];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int32_t col = (j * R + t) * VEC;
        if constexpr (kKeep) {
            if (col < D && p.w1) ld_w<VEC>(p.w1, col, w1[j]);
            if (col < D && p.w2) ld_w<VEC>(p.w2, col, w2[j]);
        }
#pragma unroll
        for (int i = 0; i < VEC; ++i) dw1[j][i] = dw2[j][i] = 0.f;
    }
    auto weights = [&](const float *w, float (&kept)[kKeep ? NV : 1][VEC], int j, int32_t col, float (&v)[VEC]) {
        if constexpr (kKeep) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) v[i] = kept[j][i];
        } else {
            ld_w<VEC>(w, col, v);
        }
    };
    for (int slot = 0; row < p.C; row += step, slot ^= 1) {
        const float r1 = next1, r2 = next2;
        if constexpr (RING) {
            ahead.wait(p.error);
            const T *buf = reinterpret_cast<const T *>(ring + ahead.s * ahead.stage);
#pragma unroll
            for (int i = 0; i < 5; ++i) {
                if (!p.in[i]) continue;
#pragma unroll
                for (int j = 0; j < NV; ++j) {
                    const int32_t col = (j * R + t) * VEC;
                    if (col < D) a[i][j] = ld<T, VEC>(buf, col);
                }
                buf += D;
            }
        }
        Raw<T, VEC> y[NV], g[NV];
        float d[NV][VEC], n[NV][VEC], f[NV][VEC], s = 0.f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            y[j] = a[0][j];
            g[j] = a[1][j];
            const int32_t col = (j * R + t) * VEC;
            if (col >= D) continue;
            if (p.in[4]) {
                unpack(a[4][j], d[j]);
            } else {
#pragma unroll
                for (int i = 0; i < VEC; ++i) d[j][i] = 0.f;
            }
            if (p.w2) {
                float w[VEC];
                weights(p.w2, w2, j, col, w);
                unpack(a[2][j], f[j]);
                unpack(a[3][j], n[j]);
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    n[j][i] *= r2;
                    dw2[j][i] = fmaf(f[j][i], n[j][i], dw2[j][i]);
                    f[j][i] *= w[i];
                    s = fmaf(f[j][i], n[j][i], s);
                }
            }
        }
        auto free_stage = [&] {
            if constexpr (RING) {
                if (t == 0 && row + stages * step < p.C) ahead.fetch(p.in, row + stages * step, D, ahead.s);
            }
            load(row + step);
        };
        if (p.w2) {
            const float m = row_sum<R>(s, sm[slot][0][sub]) * inv_d;
            free_stage();
#pragma unroll
            for (int j = 0; j < NV; ++j) {
#pragma unroll
                for (int i = 0; i < VEC; ++i) d[j][i] = fmaf(r2, f[j][i] - n[j][i] * m, d[j][i]);
            }
        }
        s = 0.f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int32_t col = (j * R + t) * VEC;
            if (col >= D) continue;
            if (p.dres) st<T, VEC>(p.dres, row * D + col, d[j]);
            float w[VEC];
            if (p.w1) weights(p.w1, w1, j, col, w);
            unpack(y[j], n[j]);
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                d[j][i] *= p.scale;
                if (p.w1) n[j][i] *= r1;
            }
            if (p.in[1]) {
                float z[VEC];
                unpack(g[j], z);
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    float slope;
                    const float value = gate_of(z[i], p.act, slope);
                    z[i] = d[j][i] * (p.w1 ? n[j][i] * w[i] : n[j][i]) * slope;
                    d[j][i] *= value;
                }
                if (p.dgate) st<T, VEC>(p.dgate, row * D + col, z);
            }
            if (p.w1) {
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    dw1[j][i] = fmaf(d[j][i], n[j][i], dw1[j][i]);
                    d[j][i] *= w[i];
                    s = fmaf(d[j][i], n[j][i], s);
                }
            }
        }
        float m = 0.f;
        if (p.w1) {
            m = row_sum<R>(s, sm[slot][1][sub]) * inv_d;
            if (!p.w2) free_stage();
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int32_t col = (j * R + t) * VEC;
            if (col >= D) continue;
            if (p.w1) {
#pragma unroll
                for (int i = 0; i < VEC; ++i) d[j][i] = r1 * (d[j][i] - n[j][i] * m);
            }
            st<T, VEC>(p.dy, row * D + col, d[j]);
        }
        if constexpr (RING) ahead.next();
    }
    if constexpr (RING) if (t == 0) ahead.drain();
    // the rows of a block leave one sum of either weight, added in ascending order
    __shared__ float all[kRows > 1 ? kRows : 1][kRows > 1 ? R * NV * VEC : 1];
    for (int which = 0; which < 2; ++which) {
        if (!(which ? p.w2 : p.w1)) continue;
        float *part = p.part + blockIdx.x * (2 * static_cast<int64_t>(D)) + which * D;
        if constexpr (kRows > 1) __syncthreads();
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int32_t col = (j * R + t) * VEC;
            if (col >= D) continue;
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const float v = which ? dw2[j][i] : dw1[j][i];
                if constexpr (kRows > 1) all[sub][col + i] = v;
                else part[col + i] = v;
            }
        }
        if constexpr (kRows > 1) {
            __syncthreads();
            for (int32_t c = threadIdx.x; c < D; c += block_of(R)) {
                float v = all[0][c];
#pragma unroll
                for (int k = 1; k < kRows; ++k) v += all[k][c];
                part[c] = v;
            }
        }
    }
}

// dw1 and dw2 from the groups' sums: 32 warps take every 32nd group each, in ascending order, and
// are added in order.
struct Dw { const float *part; float *dw1, *dw2; int32_t D, groups; };
__global__ void __launch_bounds__(1024) block_norm_dw_kernel(const Dw p) {
    __shared__ float sm[32][33];
    wait_previous();
    const int lane = threadIdx.x & 31, k = threadIdx.x >> 5;
    const int32_t blocks = (p.D + 31) / 32, which = blockIdx.x / blocks, col = (blockIdx.x - which * blocks) * 32 + lane;
    float *out = which ? p.dw2 : p.dw1;
    if (!out) return;
    float s = 0.f;
    if (col < p.D) {
#pragma unroll 8
        for (int32_t g = k; g < p.groups; g += 32) s += p.part[static_cast<int64_t>(g) * 2 * p.D + which * p.D + col];
    }
    sm[k][lane] = s;
    __syncthreads();
    if (k == 0 && col < p.D) {
#pragma unroll
        for (int i = 1; i < 32; ++i) s += sm[i][lane];
        out[col] = s;
    }
}

// Threads of a row and values that each of them keeps: eight, which leaves the registers of the
// backward (two sums and two weights a column) for two blocks of 256 threads an SM, and sixteen
// where a warp would not do otherwise.  Rows that are not whole vectors move single values.
struct Shape { int vec, r, values; bool ring; };
Shape shape_of(int32_t dtype, int32_t D) {
    const int full = dtype == HARTS_BF16 ? 8 : 4;
    Shape s{D % full == 0 ? full : 1, 8, 8, false};
    if (s.vec == 1) {
        s.r = D <= 256 ? 32 : D <= 2048 ? 256 : 1024;
    } else if (D <= 512) {
        while (s.r < 32 && s.r * 8 < D) s.r *= 2;
        if (s.r * 8 < D) s.values = 16;
    } else {
        s.ring = true;
        s.r = 128;
        while (s.r * 8 < D) s.r *= 2;
    }
    return s;
}

// Most blocks that are resident at a time, whatever the kernel's registers.
int64_t blocks_of(const Shape &s, int64_t C) {
    return std::min<int64_t>((C + rows_of(s.r) - 1) / rows_of(s.r), int64_t(sm_count()) * (2048 / block_of(s.r)));
}

// Resident blocks of a persistent kernel, and the rows that each of them has on its way.
template <typename T, int R, bool RING, typename K, typename P>
cudaError_t launch_rows(K *kernel, const P &p, int tensors, size_t budget, std::atomic<uint64_t> &allowed, std::atomic<int> &known,
                        int64_t *groups, cudaStream_t st) {
    int stages = 1, n = known.load(std::memory_order_relaxed);
    size_t smem = 0;
    if (RING) {
        const size_t stage = size_t(p.D) * sizeof(T) * tensors;
        stages = static_cast<int>(std::min<size_t>(kMaxStages, std::max<size_t>(1, budget / stage)));
        smem = stages * stage;
        const cudaError_t e = allow_smem(kernel, 200 * 1024, allowed);
        if (e != cudaSuccess) return e;
    }
    if (n == 0 || RING) {
        if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, block_of(R), smem) != cudaSuccess || n < 1) n = 1;
        if (!RING) known.store(n, std::memory_order_relaxed);
    }
    const int64_t rows = rows_of(R), grid = std::min<int64_t>((p.C + rows - 1) / rows, int64_t(sm_count()) * n);
    *groups = grid;
    return launch(kernel, grid, block_of(R), smem, 1, false, st, p, stages);
}

template <typename T, int VEC, int R, int VT, bool RING>
cudaError_t launch_one(const Fwd &p, int tensors, int64_t *groups, cudaStream_t st) {
    static std::atomic<uint64_t> allowed{0};
    static std::atomic<int> known{0};
    return launch_rows<T, R, RING>(block_norm_fwd_kernel<T, VEC, R, VT / VEC, RING>, p, tensors, std::min<size_t>(size_t(48) * 1024 * R / 256, 200 * 1024),
                                   allowed, known, groups, st);
}
template <typename T, int VEC, int R, int VT, bool RING>
cudaError_t launch_one(const Bwd &p, int tensors, int64_t *groups, cudaStream_t st) {
    static std::atomic<uint64_t> allowed{0};
    static std::atomic<int> known{0};
    return launch_rows<T, R, RING>(block_norm_bwd_kernel<T, VEC, R, VT / VEC, RING>, p, tensors, std::min<size_t>(size_t(100) * 1024 * R / 256, 200 * 1024),
                                   allowed, known, groups, st);
}

// The instances that shape_of names.
template <typename T, int VEC, typename P>
cudaError_t run(const Shape &s, const P &p, int tensors, int64_t *groups, cudaStream_t st) {
#define HARTS_CASE(V, R, VT, RING) \
    if (s.vec == V && s.r == R && s.values == VT && s.ring == RING) return launch_one<T, V, R, VT, RING>(p, tensors, groups, st);
    HARTS_CASE(VEC, 8, 8, false) HARTS_CASE(VEC, 16, 8, false) HARTS_CASE(VEC, 32, 8, false) HARTS_CASE(VEC, 32, 16, false)
    HARTS_CASE(VEC, 128, 8, true) HARTS_CASE(VEC, 256, 8, true) HARTS_CASE(VEC, 512, 8, true) HARTS_CASE(VEC, 1024, 8, true)
    HARTS_CASE(1, 32, 8, false) HARTS_CASE(1, 256, 8, false) HARTS_CASE(1, 1024, 8, false)
#undef HARTS_CASE
    return cudaErrorInvalidValue;
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

int cuda_fail(cudaError_t e, const char *what) {
    set_error(std::string(what) + ": " + cudaGetErrorString(e));
    return HARTS_ECUDA;
}

int check(const harts_block_norm_args *a) {
    if (!a) { set_error("NULL args"); return HARTS_EINVAL; }
    if (a->dtype != HARTS_FP32 && a->dtype != HARTS_BF16) { set_error("dtype"); return HARTS_EUNSUPPORTED; }
    if (a->C < 0 || a->D < 1) { set_error("C >= 0 and D >= 1 required"); return HARTS_EINVAL; }
    if (a->D > kMaxDim) { set_error("D above 8192"); return HARTS_EUNSUPPORTED; }
    if (!std::isfinite(a->scale)) { set_error("scale must be finite"); return HARTS_EINVAL; }
    if (a->gate_act < HARTS_GATE_LINEAR || a->gate_act > HARTS_GATE_SIGMOID) { set_error("gate_act must be 0, 1 or 2"); return HARTS_EINVAL; }
    return HARTS_OK;
}

int check_inputs(const harts_block_norm_args *a) {
    if (!a->post_weight && !a->pre_weight) { set_error("neither norm: post_weight and pre_weight are both NULL"); return HARTS_EINVAL; }
    if (!a->y || !a->h) { set_error("NULL y or h"); return HARTS_EINVAL; }
    if (!aligned16(a->y) || !aligned16(a->gate) || !aligned16(a->residual) || !aligned16(a->post_weight) || !aligned16(a->pre_weight) ||
        !aligned16(a->h) || !aligned16(a->n)) {
        set_error("y, gate, residual, weights, h and n must be 16-byte aligned");
        return HARTS_EINVAL;
    }
    return HARTS_OK;
}

}  // namespace
}  // namespace harts

using namespace harts;

extern "C" {

int harts_block_norm_fwd(const harts_block_norm_args *a, harts_stream_t stream) {
    int rc = check(a);
    if (rc) return rc;
    if (!(a->eps >= 0.f) || std::isinf(a->eps)) { set_error("eps must be finite and >= 0"); return HARTS_EINVAL; }
    if (a->C == 0) { set_error(""); return HARTS_OK; }
    rc = check_inputs(a);
    if (rc) return rc;
    if ((a->n == nullptr) != (a->pre_weight == nullptr)) { set_error("n and pre_weight go together"); return HARTS_EINVAL; }
    if (a->n == a->h) { set_error("h and n are one buffer"); return HARTS_EINVAL; }
    Fwd p{};
    p.in[0] = a->y; p.in[1] = a->gate; p.in[2] = a->residual;
    p.w1 = a->post_weight; p.w2 = a->pre_weight;
    p.h = a->h; p.n = a->n; p.r1 = a->rstd_post; p.r2 = a->rstd_pre;
    p.C = a->C; p.D = a->D; p.act = a->gate_act; p.scale = a->scale; p.eps = a->eps;
    p.error = a->error ? a->error : own_error_word();
    if (!p.error) { set_error("the library's error word is not to be had"); return HARTS_ECUDA; }
    int64_t groups = 0;
    const int tensors = 1 + (a->gate != nullptr) + (a->residual != nullptr);
    const Shape s = shape_of(a->dtype, a->D);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = a->dtype == HARTS_BF16 ? run<__nv_bfloat16, 8>(s, p, tensors, &groups, st) : run<float, 4>(s, p, tensors, &groups, st);
    if (e != cudaSuccess) return cuda_fail(e, "block norm forward launch");
    set_error("");
    return HARTS_OK;
}

size_t harts_block_norm_bwd_workspace_bytes(int64_t C, int32_t D, int32_t dtype) {
    if (C < 0 || D < 1 || D > kMaxDim || (dtype != HARTS_FP32 && dtype != HARTS_BF16)) return 0;
    return std::max<size_t>(256, 2 * sizeof(float) * static_cast<size_t>(blocks_of(shape_of(dtype, D), C)) * D);
}

int harts_block_norm_bwd(const harts_block_norm_bwd_args *b, harts_stream_t stream) {
    if (!b) { set_error("NULL args"); return HARTS_EINVAL; }
    const harts_block_norm_args *a = &b->fwd;
    int rc = check(a);
    if (rc) return rc;
    if ((a->post_weight && !b->dpost_weight) || (a->pre_weight && !b->dpre_weight)) { set_error("NULL dpost_weight or dpre_weight"); return HARTS_EINVAL; }
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (a->C == 0) {
        cudaError_t e = cudaSuccess;
        if (a->post_weight) e = cudaMemsetAsync(b->dpost_weight, 0, sizeof(float) * a->D, st);
        if (e == cudaSuccess && a->pre_weight) e = cudaMemsetAsync(b->dpre_weight, 0, sizeof(float) * a->D, st);
        if (e != cudaSuccess) return cuda_fail(e, "block norm backward");
        set_error("");
        return HARTS_OK;
    }
    rc = check_inputs(a);
    if (rc) return rc;
    if ((a->post_weight && !a->rstd_post) || (a->pre_weight && !a->rstd_pre)) { set_error("NULL rstd_post or rstd_pre"); return HARTS_EINVAL; }
    if ((b->d_n == nullptr) != (a->pre_weight == nullptr)) { set_error("d_n and pre_weight go together"); return HARTS_EINVAL; }
    if (!b->d_n && !b->d_h) { set_error("neither d_n nor d_h"); return HARTS_EINVAL; }
    if (!b->dy) { set_error("NULL dy"); return HARTS_EINVAL; }
    if (b->dgate && !a->gate) { set_error("dgate without a gate"); return HARTS_EINVAL; }
    if (b->dy == b->dgate || b->dy == b->dresidual || (b->dgate && b->dgate == b->dresidual)) { set_error("two outputs in one buffer"); return HARTS_EINVAL; }
    if (!aligned16(b->d_n) || !aligned16(b->d_h) || !aligned16(b->dy) || !aligned16(b->dgate) || !aligned16(b->dresidual) || !aligned16(b->workspace)) {
        set_error("d_n, d_h, dy, dgate, dresidual and workspace must be 16-byte aligned");
        return HARTS_EINVAL;
    }
    if (!b->workspace || b->workspace_bytes < harts_block_norm_bwd_workspace_bytes(a->C, a->D, a->dtype)) {
        set_error("workspace too small");
        return HARTS_ESMALLBUF;
    }
    Bwd p{};
    p.in[0] = a->y; p.in[1] = a->gate; p.in[2] = b->d_n; p.in[3] = a->pre_weight ? a->h : nullptr; p.in[4] = b->d_h;
    p.w1 = a->post_weight; p.w2 = a->pre_weight; p.r1 = a->rstd_post; p.r2 = a->rstd_pre;
    p.dy = b->dy; p.dgate = b->dgate; p.dres = b->dresidual;
    p.part = static_cast<float *>(b->workspace);
    p.C = a->C; p.D = a->D; p.act = a->gate_act; p.scale = a->scale;
    p.error = a->error ? a->error : own_error_word();
    if (!p.error) { set_error("the library's error word is not to be had"); return HARTS_ECUDA; }
    int tensors = 0;
    for (const void *q : p.in) tensors += q != nullptr;
    int64_t groups = 0;
    const Shape s = shape_of(a->dtype, a->D);
    cudaError_t e = a->dtype == HARTS_BF16 ? run<__nv_bfloat16, 8>(s, p, tensors, &groups, st) : run<float, 4>(s, p, tensors, &groups, st);
    if (e != cudaSuccess) return cuda_fail(e, "block norm backward launch");
    const Dw d{p.part, a->post_weight ? b->dpost_weight : nullptr, a->pre_weight ? b->dpre_weight : nullptr, a->D, static_cast<int32_t>(groups)};
    e = launch(block_norm_dw_kernel, 2 * ((a->D + 31) / 32), 1024, 0, 1, true, st, d);
    if (e != cudaSuccess) return cuda_fail(e, "block norm backward launch");
    set_error("");
    return HARTS_OK;
}

}  // extern "C"
