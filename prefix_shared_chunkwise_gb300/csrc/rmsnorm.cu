// Root-mean-square norm with the residual's addition, forward and backward, with an optional
// 8-bit block output.
//
//   h = x + r,  rstd = 1 / sqrt(mean_j h_j^2 + eps),  y_j = h_j rstd w_j
//   dx = dr = rstd (w dy - n mean_j(w_j dy_j n_j)) + dh,  n = h rstd,   dw_j = sum_c dy_cj n_cj
// Sums and statistics are fp32; h is normalised before its own rounding to the stream's type,
// so y carries one rounding.  The backward reads the rounded h that the forward stored.
//
// Both directions move every value once and do ~10 operations on it: HBM bounds them.  A row
// belongs to R threads that keep it in registers between the statistics and the output, so
// nothing is read twice.  Blocks are persistent: each thread keeps the weights (and, backward,
// the column sums of dw) of its columns in registers over all its rows where they fit --
// fp32 weights re-read per row would be as many bytes as two bf16 streams -- and the next
// row's loads are under way before the current row's reduction: in registers forward and for
// short rows, by bulk copies into shared memory for longer rows backward.  dw: each block
// writes its column sums, a second kernel adds them in ascending order: no atomics, the same
// bits on every run.
//
// Measured in TB/s with the residual, forward / backward: 65,536 x 2,048 bf16 6.1 / 6.8, with 8-bit
// output 6.2; 32,768 x 2,048 fp32 6.3 / 6.4; rows that are not whole vectors, 65,536 x 2,001 bf16
// 4.7 / 3.7, 32,768 x 2,001 fp32 6.3 / 5.6; rows above 8,192 values, which the backward reads twice,
// 4,096 x 12,288 bf16 5.9 / 2.8, 4,096 x 16,384 fp32 6.1 / 4.6.
#include <cuda_fp8.h>

#include <algorithm>
#include <cmath>
#include <cstring>

#include "kda_common.cuh"
#include "launch_util.h"
#include "tc_primitives.cuh"

namespace harts {
namespace {

constexpr int kMaxDim = 16384;      // 1024 threads x 16 values
constexpr int kMxBlock = 32;        // channels that share a scale
constexpr int kLongRow = 8192;      // values; longer rows take a kernel of their own backward
constexpr int kMaxStages = 4;       // rows copied ahead

struct NormFwd {
    const void *x, *res;
    const float *w;
    void *h, *y, *y8;
    uint8_t *scale8;
    float *rstd;
    int64_t C;
    int32_t D;
    float eps;
};

struct NormBwd {
    const void *dy, *h, *dh;
    const float *w, *rstd;
    void *dx;
    float *part;                    // [groups][D]
    int32_t *error;
    int64_t C;
    int32_t D;
};

template <typename T, int VEC> struct Raw;      // VEC values of T as they lie in memory
template <> struct Raw<__nv_bfloat16, 8> { uint4 u; };
template <> struct Raw<float, 4> { float4 u; };
template <> struct Raw<__nv_bfloat16, 1> { __nv_bfloat16 u; };
template <> struct Raw<float, 1> { float u; };

__device__ __forceinline__ void unpack(const Raw<__nv_bfloat16, 8> &r, float *v) {
    const __nv_bfloat162 *p = reinterpret_cast<const __nv_bfloat162 *>(&r.u);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __bfloat1622float2(p[i]);
        v[2 * i] = f.x; v[2 * i + 1] = f.y;
    }
}
__device__ __forceinline__ void unpack(const Raw<float, 4> &r, float *v) {
    v[0] = r.u.x; v[1] = r.u.y; v[2] = r.u.z; v[3] = r.u.w;
}
__device__ __forceinline__ void unpack(const Raw<__nv_bfloat16, 1> &r, float *v) { v[0] = __bfloat162float(r.u); }
__device__ __forceinline__ void unpack(const Raw<float, 1> &r, float *v) { v[0] = r.u; }

__device__ __forceinline__ void pack(Raw<__nv_bfloat16, 8> &r, const float *v) {
    __nv_bfloat162 *p = reinterpret_cast<__nv_bfloat162 *>(&r.u);
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
}
__device__ __forceinline__ void pack(Raw<float, 4> &r, const float *v) { r.u = make_float4(v[0], v[1], v[2], v[3]); }
__device__ __forceinline__ void pack(Raw<__nv_bfloat16, 1> &r, const float *v) { r.u = __float2bfloat16_rn(v[0]); }
__device__ __forceinline__ void pack(Raw<float, 1> &r, const float *v) { r.u = v[0]; }

template <typename T, int VEC>
__device__ __forceinline__ Raw<T, VEC> ld(const void *p, int64_t i) {
    return *reinterpret_cast<const Raw<T, VEC> *>(static_cast<const T *>(p) + i);
}
template <typename T, int VEC>
__device__ __forceinline__ void st(void *p, int64_t i, const float *v) {
    Raw<T, VEC> r;
    pack(r, v);
    *reinterpret_cast<Raw<T, VEC> *>(static_cast<T *>(p) + i) = r;
}

constexpr int block_of(int R) { return R < 128 ? 128 : R; }     // threads of a block
constexpr int rows_of(int R) { return block_of(R) / R; }        // rows it works on at a time
// Weights (and dw's sums) of a thread's columns stay in registers up to this many values;
// beyond, weights come from L1.
constexpr int kRegValues = 16;

// Sum over the R threads of a row.  sm holds two slots a row, used in turn, so that one barrier
// per row is enough; rows of a block (or of a warp, under 32 threads a row) do not wait for each
// other.
template <int R>
__device__ __forceinline__ uint32_t row_lanes() {
    if constexpr (R >= 32) return 0xffffffffu;
    else return ((1u << R) - 1u) << ((threadIdx.x & 31) & ~(R - 1));
}
template <int R>
__device__ __forceinline__ float row_sum(float v, float *sm) {
#pragma unroll
    for (int o = (R < 32 ? R : 32) / 2; o > 0; o >>= 1) v += __shfl_xor_sync(row_lanes<R>(), v, o);
    if constexpr (R <= 32) return v;
    const int in_row = (threadIdx.x % R) >> 5;
    if ((threadIdx.x & 31) == 0) sm[in_row] = v;
    if constexpr (R < 128) asm volatile("bar.sync %0, %1;" :: "r"(1 + static_cast<int>(threadIdx.x) / R), "n"(R) : "memory");
    else __syncthreads();
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < R / 32; ++i) s += sm[i];
    return s;
}

template <int VEC>
__device__ __forceinline__ void ld_w(const float *w, int32_t col, float (&v)[VEC]) {
    if constexpr (VEC >= 4) {
#pragma unroll
        for (int i = 0; i < VEC; i += 4) {
            const float4 f = __ldg(reinterpret_cast<const float4 *>(w + col + i));
            v[i] = f.x; v[i + 1] = f.y; v[i + 2] = f.z; v[i + 3] = f.w;
        }
    } else {
        v[0] = __ldg(w + col);
    }
}

// One block of 32 channels, spread over 32 / VEC neighbouring lanes, in 8 bits: the scale is
// the smallest power of two 2^e with amax <= 448 2^e (448 = 1.75 * 2^8 is e4m3's largest), so
// nothing saturates and the scaling itself is exact; only the 4-bit significand rounds.  A
// block that holds an infinity gets the NaN scale; a NaN stays a NaN.
template <int VEC>
__device__ __forceinline__ void store_mx(uint8_t *y8, uint8_t *scale8, int64_t row, int32_t D, int32_t col,
                                         const float *v) {
    float a = 0.f;
#pragma unroll
    for (int i = 0; i < VEC; ++i) a = fmaxf(a, fabsf(v[i]));
    constexpr int lanes = kMxBlock / VEC;
    const int lane = threadIdx.x & 31;
    const uint32_t mask = (lanes == 32 ? 0xffffffffu : ((1u << lanes) - 1u)) << (lane & ~(lanes - 1));
#pragma unroll
    for (int o = lanes / 2; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(mask, a, o));
    const uint32_t u = __float_as_uint(a);
    int e = static_cast<int>(u >> 23) - 127 - ((u & 0x7fffffu) <= 0x600000u ? 8 : 7);
    e = max(e, -127);
    const bool bad = u >= 0x7f800000u;
    const float inv = bad ? 1.f : __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
    uint8_t q[VEC];
#pragma unroll
    for (int i = 0; i < VEC; i += 2) {
        const __nv_fp8x2_storage_t t = __nv_cvt_float2_to_fp8x2(make_float2(v[i] * inv, v[i + 1] * inv),
                                                                __NV_SATFINITE, __NV_E4M3);
        q[i] = static_cast<uint8_t>(t & 0xff); q[i + 1] = static_cast<uint8_t>(t >> 8);
    }
    uint8_t *dst = y8 + row * D + col;
    if constexpr (VEC == 8) {
        uint2 w;
        memcpy(&w, q, 8);
        *reinterpret_cast<uint2 *>(dst) = w;
    } else {
        uint32_t w;
        memcpy(&w, q, 4);
        *reinterpret_cast<uint32_t *>(dst) = w;
    }
    if ((lane & (lanes - 1)) == 0) scale8[row * (D / kMxBlock) + col / kMxBlock] = bad ? 255 : static_cast<uint8_t>(e + 127);
}

template <typename T, int VEC, int R, int NV, bool MX>
__global__ void __launch_bounds__(block_of(R)) rmsnorm_fwd_kernel(NormFwd p) {
    constexpr bool kKeep = NV * VEC <= kRegValues;
    __shared__ float sm[2][rows_of(R)][R < 32 ? 1 : R / 32];
    const int t = threadIdx.x % R, sub = threadIdx.x / R;
    const int32_t D = p.D;
    const int64_t step = static_cast<int64_t>(gridDim.x) * rows_of(R);
    int64_t row = static_cast<int64_t>(blockIdx.x) * rows_of(R) + sub;
    const float inv_d = 1.f / static_cast<float>(D);
    [[maybe_unused]] float w[kKeep ? NV : 1][VEC];
    Raw<T, VEC> x[NV], r[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int32_t col = (j * R + t) * VEC;
        if (col < D && row < p.C) {
            x[j] = ld<T, VEC>(p.x, row * D + col);
            if (p.res) r[j] = ld<T, VEC>(p.res, row * D + col);
        }
    }
    if constexpr (kKeep) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int32_t col = (j * R + t) * VEC;
            if (col < D) ld_w<VEC>(p.w, col, w[j]);
        }
    }
    for (int slot = 0; row < p.C; row += step, slot ^= 1) {
        float h[NV][VEC], s = 0.f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int32_t col = (j * R + t) * VEC;
            if (col < D) {
                unpack(x[j], h[j]);
                if (p.res) {
                    float a[VEC];
                    unpack(r[j], a);
#pragma unroll
                    for (int i = 0; i < VEC; ++i) h[j][i] += a[i];
                }
#pragma unroll
                for (int i = 0; i < VEC; ++i) s = fmaf(h[j][i], h[j][i], s);
            }
        }
        const int64_t next = row + step;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int32_t col = (j * R + t) * VEC;
            if (col < D && next < p.C) {
                x[j] = ld<T, VEC>(p.x, next * D + col);
                if (p.res) r[j] = ld<T, VEC>(p.res, next * D + col);
            }
        }
        const float rstd = __frsqrt_rn(fmaf(row_sum<R>(s, sm[slot][sub]), inv_d, p.eps));
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int32_t col = (j * R + t) * VEC;
            if (col < D) {
                float v[VEC];
                if constexpr (kKeep) {
#pragma unroll
                    for (int i = 0; i < VEC; ++i) v[i] = w[j][i];
                } else {
                    ld_w<VEC>(p.w, col, v);
                }
                if (p.h) st<T, VEC>(p.h, row * D + col, h[j]);
#pragma unroll
                for (int i = 0; i < VEC; ++i) h[j][i] = h[j][i] * rstd * v[i];
                if (p.y) st<T, VEC>(p.y, row * D + col, h[j]);
                if constexpr (MX) store_mx<VEC>(static_cast<uint8_t *>(p.y8), p.scale8, row, D, col, h[j]);
            }
        }
        if (t == 0 && p.rstd) p.rstd[row] = rstd;
    }
}

template <typename T, int VEC, int R, int NV>
__global__ void __launch_bounds__(block_of(R)) rmsnorm_bwd_kernel(NormBwd p) {
    constexpr bool kKeep = NV * VEC <= kRegValues;
    __shared__ float sm[2][rows_of(R)][R < 32 ? 1 : R / 32];
    const int t = threadIdx.x % R, sub = threadIdx.x / R;
    const int32_t D = p.D;
    const int64_t step = static_cast<int64_t>(gridDim.x) * rows_of(R);
    int64_t row = static_cast<int64_t>(blockIdx.x) * rows_of(R) + sub;
    const float inv_d = 1.f / static_cast<float>(D);
    [[maybe_unused]] float w[kKeep ? NV : 1][VEC];
    float dw[NV][VEC];
    Raw<T, VEC> a[NV], b[NV], e[NV];
    float rstd = 0.f;
    let_next_start();
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int32_t col = (j * R + t) * VEC;
        if (col < D && row < p.C) {
            a[j] = ld<T, VEC>(p.dy, row * D + col);
            b[j] = ld<T, VEC>(p.h, row * D + col);
            if (p.dh) e[j] = ld<T, VEC>(p.dh, row * D + col);
        }
    }
    if (row < p.C) rstd = __ldg(p.rstd + row);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int32_t col = (j * R + t) * VEC;
        if constexpr (kKeep) if (col < D) ld_w<VEC>(p.w, col, w[j]);
#pragma unroll
        for (int i = 0; i < VEC; ++i) dw[j][i] = 0.f;
    }
    for (int slot = 0; row < p.C; row += step, slot ^= 1) {
        float g[NV][VEC], n[NV][VEC], d[NV][VEC], s = 0.f;
        const float rs = rstd;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int32_t col = (j * R + t) * VEC;
            if (col < D) {
                float v[VEC];
                if constexpr (kKeep) {
#pragma unroll
                    for (int i = 0; i < VEC; ++i) v[i] = w[j][i];
                } else {
                    ld_w<VEC>(p.w, col, v);
                }
                unpack(a[j], g[j]);
                unpack(b[j], n[j]);
                if (p.dh) unpack(e[j], d[j]);
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    n[j][i] *= rs;
                    dw[j][i] = fmaf(g[j][i], n[j][i], dw[j][i]);
                    g[j][i] *= v[i];
                    s = fmaf(g[j][i], n[j][i], s);
                }
            }
        }
        const int64_t next = row + step;
        if (next < p.C) rstd = __ldg(p.rstd + next);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int32_t col = (j * R + t) * VEC;
            if (col < D && next < p.C) {
                a[j] = ld<T, VEC>(p.dy, next * D + col);
                b[j] = ld<T, VEC>(p.h, next * D + col);
                if (p.dh) e[j] = ld<T, VEC>(p.dh, next * D + col);
            }
        }
        const float m = row_sum<R>(s, sm[slot][sub]) * inv_d;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int32_t col = (j * R + t) * VEC;
            if (col < D) {
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    g[j][i] = rs * (g[j][i] - n[j][i] * m);
                    if (p.dh) g[j][i] += d[j][i];
                }
                st<T, VEC>(p.dx, row * D + col, g[j]);
            }
        }
    }
    // the rows of a block leave one sum, added in ascending order
    constexpr int kRows = rows_of(R);
    __shared__ float all[kRows > 1 ? kRows : 1][kRows > 1 ? R * NV * VEC : 1];
    float *part = p.part + blockIdx.x * static_cast<int64_t>(D);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int32_t col = (j * R + t) * VEC;
        if (col < D) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                if constexpr (kRows > 1) all[sub][col + i] = dw[j][i];
                else part[col + i] = dw[j][i];
            }
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

// ---- backward with rows copied ahead into shared memory ----------------------------------
// The registers of a backward row (dw's sums, weights, two unpacked streams) leave too few
// threads for the loads that HBM wants on their way.  Rows of 1 KB and more are copied by
// cp.async.bulk into a ring of `stages` rows instead, whose bytes in flight do not depend on
// registers: 65,536 rows of 2,048 bf16 values with dh 5618 -> 6554 GB/s, without 3921 -> 6134.

__device__ __forceinline__ void bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                 :: "r"(tc::smem_addr(dst)), "l"(src), "r"(bytes), "r"(tc::smem_addr(bar)) : "memory");
}

template <typename T, int VEC, int R, int NV>
__global__ void __launch_bounds__(R) rmsnorm_bwd_ring_kernel(NormBwd p, int stages) {
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ float sm[2][R / 32];
    __shared__ uint64_t full[kMaxStages];
    __shared__ int s_fail;
    const int t = threadIdx.x;
    const int32_t D = p.D;
    const int64_t step = gridDim.x;
    const uint32_t bytes = static_cast<uint32_t>(D) * sizeof(T), stage = bytes * (p.dh ? 3 : 2);
    const float inv_d = 1.f / static_cast<float>(D);
    auto fetch = [&](int64_t row, int s) {              // thread 0
        uint8_t *dst = ring + s * stage;
        tc::mbar_expect_tx(&full[s], stage);
        bulk_load(dst, static_cast<const T *>(p.dy) + row * D, bytes, &full[s]);
        bulk_load(dst + bytes, static_cast<const T *>(p.h) + row * D, bytes, &full[s]);
        if (p.dh) bulk_load(dst + 2 * bytes, static_cast<const T *>(p.dh) + row * D, bytes, &full[s]);
    };
    // A wait that runs out is reported once and never waited for again; the block goes on with
    // what its shared memory holds, so that its barriers stay matched.
    auto wait = [&](int s, uint32_t phase) {
        if (tc::mbar_try(&full[s], phase) || *reinterpret_cast<volatile int *>(&s_fail)) return;
        if (!tc::mbar_wait(&full[s], phase)) {
            *reinterpret_cast<volatile int *>(&s_fail) = 1;
            atomicCAS(p.error, 0, static_cast<int>(kDevErrTimeout));
        }
    };
    if (t == 0) {
        s_fail = 0;
        for (int s = 0; s < stages; ++s) tc::mbar_init(&full[s], 1);
        tc::fence_mbar_init();
        for (int s = 0; s < stages && blockIdx.x + s * step < p.C; ++s) fetch(blockIdx.x + s * step, s);
    }
    let_next_start();
    float w[NV][VEC], dw[NV][VEC];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int32_t col = (j * R + t) * VEC;
        if (col < D) ld_w<VEC>(p.w, col, w[j]);
#pragma unroll
        for (int i = 0; i < VEC; ++i) dw[j][i] = 0.f;
    }
    __syncthreads();
    int s = 0, slot = 0;
    uint32_t phase = 0;
    float next_rs = blockIdx.x < p.C ? __ldg(p.rstd + blockIdx.x) : 0.f;
    for (int64_t row = blockIdx.x; row < p.C; row += step, slot ^= 1) {
        const float rs = next_rs;
        if (row + step < p.C) next_rs = __ldg(p.rstd + row + step);
        wait(s, phase);
        const T *buf = reinterpret_cast<const T *>(ring + s * stage);
        float g[NV][VEC], n[NV][VEC], sum = 0.f;
        Raw<T, VEC> e[NV];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int32_t col = (j * R + t) * VEC;
            if (col < D) {
                unpack(ld<T, VEC>(buf, col), g[j]);
                unpack(ld<T, VEC>(buf + D, col), n[j]);
                if (p.dh) e[j] = ld<T, VEC>(buf + 2 * D, col);
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    n[j][i] *= rs;
                    dw[j][i] = fmaf(g[j][i], n[j][i], dw[j][i]);
                    g[j][i] *= w[j][i];
                    sum = fmaf(g[j][i], n[j][i], sum);
                }
            }
        }
        const float m = row_sum<R>(sum, sm[slot]) * inv_d;      // behind its barrier the stage is free
        if (t == 0 && row + stages * step < p.C) fetch(row + stages * step, s);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int32_t col = (j * R + t) * VEC;
            if (col < D) {
                float d[VEC];
                if (p.dh) unpack(e[j], d);
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    g[j][i] = rs * (g[j][i] - n[j][i] * m);
                    if (p.dh) g[j][i] += d[i];
                }
                st<T, VEC>(p.dx, row * D + col, g[j]);
            }
        }
        if (++s == stages) { s = 0; phase ^= 1; }
    }
    if (t == 0 && *reinterpret_cast<volatile int *>(&s_fail))       // copies in flight, after a failure
        for (int i = 0; i < stages; ++i) tc::mbar_wait(&full[i], 0, 100000000LL), tc::mbar_wait(&full[i], 1, 100000000LL);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int32_t col = (j * R + t) * VEC;
        if (col < D) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) p.part[blockIdx.x * static_cast<int64_t>(D) + col + i] = dw[j][i];
        }
    }
}

// Rows above 8,192 values: a block of 1,024 threads reads them twice, the second time from L2,
// and keeps dw's sums in shared memory.
template <typename T, int VEC>
__global__ void __launch_bounds__(1024) rmsnorm_bwd_long_kernel(NormBwd p) {
    extern __shared__ float sdw[];
    __shared__ float sm[2][32];
    const int32_t D = p.D;
    const float inv_d = 1.f / static_cast<float>(D);
    let_next_start();
    for (int32_t c = threadIdx.x * VEC; c < D; c += 1024 * VEC)
        for (int i = 0; i < VEC; ++i) sdw[c + i] = 0.f;
    int slot = 0;
    for (int64_t row = blockIdx.x; row < p.C; row += gridDim.x, slot ^= 1) {
        const float rs = __ldg(p.rstd + row);
        float sum = 0.f;
        for (int32_t c = threadIdx.x * VEC; c < D; c += 1024 * VEC) {
            float g[VEC], n[VEC], w[VEC];
            unpack(ld<T, VEC>(p.dy, row * D + c), g);
            unpack(ld<T, VEC>(p.h, row * D + c), n);
            ld_w<VEC>(p.w, c, w);
#pragma unroll
            for (int i = 0; i < VEC; ++i) sum = fmaf(g[i] * w[i], n[i] * rs, sum);
        }
        const float m = row_sum<1024>(sum, sm[slot]) * inv_d;
        for (int32_t c = threadIdx.x * VEC; c < D; c += 1024 * VEC) {
            float g[VEC], n[VEC], w[VEC], d[VEC];
            unpack(ld<T, VEC>(p.dy, row * D + c), g);
            unpack(ld<T, VEC>(p.h, row * D + c), n);
            if (p.dh) unpack(ld<T, VEC>(p.dh, row * D + c), d);
            ld_w<VEC>(p.w, c, w);
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                n[i] *= rs;
                sdw[c + i] = fmaf(g[i], n[i], sdw[c + i]);
                g[i] = rs * (g[i] * w[i] - n[i] * m);
                if (p.dh) g[i] += d[i];
            }
            st<T, VEC>(p.dx, row * D + c, g);
        }
    }
    for (int32_t c = threadIdx.x * VEC; c < D; c += 1024 * VEC)
        for (int i = 0; i < VEC; ++i) p.part[blockIdx.x * static_cast<int64_t>(D) + c + i] = sdw[c + i];
}

// dw[j] = sum over the groups' column sums: 32 warps take every 32nd group each, in ascending
// order, and are added in order.
struct DwParams { const float *part; float *dw; int32_t D, groups; };
__global__ void __launch_bounds__(1024) rmsnorm_dw_kernel(DwParams p) {
    __shared__ float sm[32][33];
    wait_previous();
    const int lane = threadIdx.x & 31, k = threadIdx.x >> 5;
    const int32_t col = blockIdx.x * 32 + lane;
    float s = 0.f;
    if (col < p.D) {
#pragma unroll 8
        for (int32_t g = k; g < p.groups; g += 32) s += p.part[static_cast<int64_t>(g) * p.D + col];
    }
    sm[k][lane] = s;
    __syncthreads();
    if (k == 0 && col < p.D) {
#pragma unroll
        for (int i = 1; i < 32; ++i) s += sm[i][lane];
        p.dw[col] = s;
    }
}

// Threads of a row (R) and values that each of them keeps.  What counts is that R * values is
// little above D -- idle threads hold registers that could hold loads -- and how many bytes are
// on their way.  Measured in GB/s at 2^27 bf16 values, forward with / without a residual:
//   D = 1024: R 32 x 32 6218 / 5958, 64 x 16 6242 / 4855, 128 x 16 5825 / 4345
//   D = 4096: R 128 x 32 6242 / 6096, 256 x 16 6473 / 5574, 256 x 32 6019 / 4599
// so the forward keeps 32 values.  The backward needs registers for dw's sums too:
//   D = 1024: R 32 x 32 5444, 64 x 16 5405, 128 x 8 5937, 128 x 16 4096
//   D = 2048: R 64 x 32 5405, 128 x 16 5699, 256 x 8 5510, 256 x 16 4263
// so it keeps 16, and at least 128 threads beyond a warp.  Short rows share a warp.  Rows that are not whole vectors move
// single values; 8 a thread measured best in both directions (D = 2001: 256 x 8 4723 / 3799
// forward / backward, 128 x 16 4681 / 3312).
struct Shape { int vec, r, values; };
Shape shape_of(int32_t dtype, int32_t D, bool backward) {
    const int full = dtype == HARTS_BF16 ? 8 : 4;
    Shape s;
    s.vec = D % full == 0 ? full : 1;
    const int most = s.vec == 1 ? 8 : backward ? 16 : 32;
    s.r = s.vec == 1 ? 32 : 8;
    while (s.r < 1024 && s.r * most < D) s.r = backward && s.vec > 1 && s.r == 32 ? 128 : s.r * 2;
    s.values = 8;
    while (s.r * s.values < D) s.values *= 2;
    return s;
}

// Most blocks that are resident at a time, whatever the kernel's registers.
int64_t blocks_of(const Shape &s, int64_t C) {
    const int64_t rows = rows_of(s.r);
    return std::min<int64_t>((C + rows - 1) / rows, int64_t(sm_count()) * (2048 / block_of(s.r)));
}

// Blocks of a persistent kernel: as many as are resident at a time, but no more than have rows.
template <typename F>
int grid_of(F *kernel, int R, int64_t C, std::atomic<int> &known) {
    int n = known.load(std::memory_order_relaxed);
    if (n == 0) {
        if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, block_of(R), 0) != cudaSuccess || n < 1) n = 1;
        known.store(n, std::memory_order_relaxed);
    }
    const int64_t rows = rows_of(R);
    return static_cast<int>(std::min<int64_t>((C + rows - 1) / rows, int64_t(sm_count()) * n));
}

template <typename T, int VEC, int R, int VT>
cudaError_t launch_fwd(const NormFwd &p, int64_t *, cudaStream_t st) {
    constexpr int NV = VT / VEC;
    if constexpr (VEC > 1) {
        if (p.y8) {
            static std::atomic<int> known{0};
            auto *k = rmsnorm_fwd_kernel<T, VEC, R, NV, true>;
            return launch(k, grid_of(k, R, p.C, known), block_of(R), 0, 1, false, st, p);
        }
    }
    static std::atomic<int> known{0};
    auto *k = rmsnorm_fwd_kernel<T, VEC, R, NV, false>;
    return launch(k, grid_of(k, R, p.C, known), block_of(R), 0, 1, false, st, p);
}
template <typename T, int VEC, int R, int VT>
cudaError_t launch_bwd(const NormBwd &p, int64_t *groups, cudaStream_t st) {
    static std::atomic<int> known{0};
    if constexpr (VEC > 1 && R >= 128) {
        static std::atomic<uint64_t> allowed{0};
        auto *k = rmsnorm_bwd_ring_kernel<T, VEC, R, VT / VEC>;
        // 45 KB of rows on their way for each 128 threads
        const size_t stage = size_t(p.D) * sizeof(T) * (p.dh ? 3 : 2), budget = size_t(45) * 1024 * R / 128;
        const int stages = static_cast<int>(std::min<size_t>(kMaxStages, std::max<size_t>(2, budget / stage)));
        const cudaError_t e = allow_smem(k, 200 * 1024, allowed);       // two stages of 8,192 fp32 values are 192 KB
        if (e != cudaSuccess) return e;
        int n = 0;
        if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, k, R, stages * stage) != cudaSuccess || n < 1) n = 1;
        const int64_t grid = std::min<int64_t>(p.C, int64_t(sm_count()) * n);
        *groups = grid;
        return launch(k, grid, R, stages * stage, 1, false, st, p, stages);
    } else {
        auto *k = rmsnorm_bwd_kernel<T, VEC, R, VT / VEC>;
        const int grid = grid_of(k, R, p.C, known);
        *groups = grid;
        return launch(k, grid, block_of(R), 0, 1, false, st, p);
    }
}
template <typename T, int VEC>
cudaError_t launch_bwd_long(const NormBwd &p, int64_t *groups, cudaStream_t st) {
    static std::atomic<uint64_t> allowed{0};
    auto *k = rmsnorm_bwd_long_kernel<T, VEC>;
    const cudaError_t e = allow_smem(k, kMaxDim * sizeof(float), allowed);
    if (e != cudaSuccess) return e;
    *groups = std::min<int64_t>(p.C, sm_count() * 2);
    return launch(k, *groups, 1024, size_t(p.D) * sizeof(float), 1, false, st, p);
}

// The instances that shape_of names.
#define HARTS_NORM_CASE(LAUNCH, T, VEC, R, VT) \
    if (s.vec == VEC && s.r == R && s.values == VT) return LAUNCH<T, VEC, R, VT>(p, groups, st);
#define HARTS_NORM_SINGLE(LAUNCH, T)                                                                                \
    HARTS_NORM_CASE(LAUNCH, T, 1, 32, 8) HARTS_NORM_CASE(LAUNCH, T, 1, 64, 8) HARTS_NORM_CASE(LAUNCH, T, 1, 128, 8) \
    HARTS_NORM_CASE(LAUNCH, T, 1, 256, 8) HARTS_NORM_CASE(LAUNCH, T, 1, 512, 8)                                     \
    HARTS_NORM_CASE(LAUNCH, T, 1, 1024, 8)

template <typename T, int VEC>
cudaError_t run_fwd(const Shape &s, const NormFwd &p, cudaStream_t st) {
    int64_t *groups = nullptr;
    HARTS_NORM_CASE(launch_fwd, T, VEC, 8, 8) HARTS_NORM_CASE(launch_fwd, T, VEC, 8, 16)
    HARTS_NORM_CASE(launch_fwd, T, VEC, 8, 32) HARTS_NORM_CASE(launch_fwd, T, VEC, 16, 32)
    HARTS_NORM_CASE(launch_fwd, T, VEC, 32, 32) HARTS_NORM_CASE(launch_fwd, T, VEC, 64, 32)
    HARTS_NORM_CASE(launch_fwd, T, VEC, 128, 32) HARTS_NORM_CASE(launch_fwd, T, VEC, 256, 32)
    HARTS_NORM_CASE(launch_fwd, T, VEC, 512, 32)
    HARTS_NORM_SINGLE(launch_fwd, T)
    HARTS_NORM_CASE(launch_fwd, T, 1, 1024, 16)
    return cudaErrorInvalidValue;
}
template <typename T, int VEC>
cudaError_t run_bwd(const Shape &s, const NormBwd &p, int64_t *groups, cudaStream_t st) {
    if (p.D > kLongRow) return s.vec == VEC ? launch_bwd_long<T, VEC>(p, groups, st) : launch_bwd_long<T, 1>(p, groups, st);
    HARTS_NORM_CASE(launch_bwd, T, VEC, 8, 8) HARTS_NORM_CASE(launch_bwd, T, VEC, 8, 16)
    HARTS_NORM_CASE(launch_bwd, T, VEC, 16, 16) HARTS_NORM_CASE(launch_bwd, T, VEC, 32, 16)
    HARTS_NORM_CASE(launch_bwd, T, VEC, 128, 8) HARTS_NORM_CASE(launch_bwd, T, VEC, 128, 16)
    HARTS_NORM_CASE(launch_bwd, T, VEC, 256, 16) HARTS_NORM_CASE(launch_bwd, T, VEC, 512, 16)
    HARTS_NORM_SINGLE(launch_bwd, T)
    return cudaErrorInvalidValue;
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

int check_common(int64_t C, int32_t D, int32_t dtype) {
    if (dtype != HARTS_FP32 && dtype != HARTS_BF16) { set_error("dtype"); return HARTS_EUNSUPPORTED; }
    if (C < 0 || D < 1) { set_error("C >= 0 and D >= 1 required"); return HARTS_EINVAL; }
    if (D > kMaxDim) { set_error("D above 16384"); return HARTS_EUNSUPPORTED; }
    return HARTS_OK;
}

int cuda_fail(cudaError_t e, const char *what) {
    set_error(std::string(what) + ": " + cudaGetErrorString(e));
    return HARTS_ECUDA;
}

}  // namespace
}  // namespace harts

using namespace harts;

extern "C" {

int harts_rmsnorm_fwd(const harts_rmsnorm_fwd_args *a, harts_stream_t stream) {
    if (!a) { set_error("NULL args"); return HARTS_EINVAL; }
    const int rc = check_common(a->C, a->D, a->dtype);
    if (rc) return rc;
    if (!(a->eps >= 0.f) || std::isinf(a->eps)) { set_error("eps must be finite and >= 0"); return HARTS_EINVAL; }
    if (a->C == 0) { set_error(""); return HARTS_OK; }
    if (!a->x || !a->weight) { set_error("NULL x or weight"); return HARTS_EINVAL; }
    if (!a->y && !a->y8) { set_error("no output: y and y8 are both NULL"); return HARTS_EINVAL; }
    if (a->residual && !a->h) { set_error("h is required with a residual"); return HARTS_EINVAL; }
    if (a->h && a->h == a->y) { set_error("h and y are one buffer"); return HARTS_EINVAL; }
    if ((a->y8 == nullptr) != (a->y8_scale == nullptr)) { set_error("y8 and y8_scale go together"); return HARTS_EINVAL; }
    if (a->y8 && a->D % kMxBlock) { set_error("the 8-bit output needs D a multiple of 32"); return HARTS_EUNSUPPORTED; }
    if (!aligned16(a->x) || !aligned16(a->residual) || !aligned16(a->weight) || !aligned16(a->h) || !aligned16(a->y) ||
        !aligned16(a->y8)) {
        set_error("x, residual, weight, h, y and y8 must be 16-byte aligned");
        return HARTS_EINVAL;
    }
    NormFwd p;
    p.x = a->x; p.res = a->residual; p.w = a->weight; p.h = a->h; p.y = a->y; p.y8 = a->y8;
    p.scale8 = static_cast<uint8_t *>(a->y8_scale); p.rstd = a->rstd; p.C = a->C; p.D = a->D; p.eps = a->eps;
    const Shape s = shape_of(a->dtype, a->D, false);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = a->dtype == HARTS_BF16 ? run_fwd<__nv_bfloat16, 8>(s, p, st) : run_fwd<float, 4>(s, p, st);
    if (e != cudaSuccess) return cuda_fail(e, "rmsnorm forward launch");
    set_error("");
    return HARTS_OK;
}

size_t harts_rmsnorm_bwd_workspace_bytes(int64_t C, int32_t D, int32_t dtype) {
    if (C < 0 || D < 1 || D > kMaxDim || (dtype != HARTS_FP32 && dtype != HARTS_BF16)) return 0;
    return std::max<size_t>(256, sizeof(float) * static_cast<size_t>(blocks_of(shape_of(dtype, D, true), C)) * D);
}

int harts_rmsnorm_bwd(const harts_rmsnorm_bwd_args *a, harts_stream_t stream) {
    if (!a) { set_error("NULL args"); return HARTS_EINVAL; }
    const int rc = check_common(a->C, a->D, a->dtype);
    if (rc) return rc;
    if (!a->dweight) { set_error("NULL dweight"); return HARTS_EINVAL; }
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (a->C == 0) {
        const cudaError_t e = cudaMemsetAsync(a->dweight, 0, sizeof(float) * a->D, st);
        if (e != cudaSuccess) return cuda_fail(e, "rmsnorm backward");
        set_error("");
        return HARTS_OK;
    }
    if (!a->dy || !a->h || !a->weight || !a->rstd || !a->dx) { set_error("NULL dy, h, weight, rstd or dx"); return HARTS_EINVAL; }
    if (!aligned16(a->dy) || !aligned16(a->h) || !aligned16(a->dh) || !aligned16(a->weight) || !aligned16(a->dx) ||
        !aligned16(a->workspace)) {
        set_error("dy, h, dh, weight, dx and workspace must be 16-byte aligned");
        return HARTS_EINVAL;
    }
    if (!a->workspace || a->workspace_bytes < harts_rmsnorm_bwd_workspace_bytes(a->C, a->D, a->dtype)) {
        set_error("workspace too small");
        return HARTS_ESMALLBUF;
    }
    NormBwd p;
    p.dy = a->dy; p.h = a->h; p.dh = a->dh; p.w = a->weight; p.rstd = a->rstd; p.dx = a->dx;
    p.part = static_cast<float *>(a->workspace); p.C = a->C; p.D = a->D;
    p.error = a->error ? a->error : own_error_word();
    if (!p.error) { set_error("the library's error word is not to be had"); return HARTS_ECUDA; }
    int64_t groups = 0;
    const Shape s = shape_of(a->dtype, a->D, true);
    cudaError_t e = a->dtype == HARTS_BF16 ? run_bwd<__nv_bfloat16, 8>(s, p, &groups, st) : run_bwd<float, 4>(s, p, &groups, st);
    if (e != cudaSuccess) return cuda_fail(e, "rmsnorm backward launch");
    const DwParams d{p.part, a->dweight, a->D, static_cast<int32_t>(groups)};
    e = launch(rmsnorm_dw_kernel, (a->D + 31) / 32, 1024, 0, 1, true, st, d);
    if (e != cudaSuccess) return cuda_fail(e, "rmsnorm backward launch");
    set_error("");
    return HARTS_OK;
}

}  // extern "C"
