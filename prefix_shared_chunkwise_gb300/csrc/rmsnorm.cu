// Root-mean-square norm with the residual's addition, forward and backward, with an optional
// 8-bit block output.
//
//   h = x + r,  rstd = 1 / sqrt(mean_j h_j^2 + eps),  y_j = h_j rstd w_j
//   dx = dr = rstd (w dy - n mean_j(w_j dy_j n_j)) + dh,  n = h rstd,   dw_j = sum_c dy_cj n_cj
// Sums and statistics are fp32; h is normalised before its own rounding to the stream's type,
// so y carries one rounding.  The backward reads the rounded h that the forward stored.
//
// Both directions move every value once and do ~10 operations on it: they are bound by HBM.
// A row belongs to R threads that keep it in registers between the statistics and the
// output, so nothing is read twice.  Blocks are persistent: each thread keeps the weights
// (and, backward, the column sums of dw) of its columns in registers over all its rows --
// fp32 weights re-read per row would be as many bytes as two bf16 streams -- and the next
// row's loads are issued before the current row's reduction, so the barrier of a row costs
// no memory time.  dw: each group of R threads writes its column sums, a second kernel adds
// them in ascending order: no atomics, the same bits on every run.
#include <cuda_fp8.h>

#include <algorithm>
#include <cmath>
#include <cstring>

#include "kda_common.cuh"
#include "launch_util.h"

namespace harts {
namespace {

constexpr int kMaxDim = 16384;      // 1024 threads x 16 values
constexpr int kMxBlock = 32;        // channels that share a scale

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

// Sum over the R threads of a row; sm is one of two slots used in turn, so that one barrier
// per row is enough.
template <int R>
__device__ __forceinline__ float row_sum(float v, float *sm) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (R == 32) return v;
    if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < R / 32; ++i) s += sm[i];
    return s;
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
__global__ void __launch_bounds__(R == 32 ? 128 : R) rmsnorm_fwd_kernel(NormFwd p) {
    __shared__ float sm[2][R / 32];
    constexpr int G = R == 32 ? 4 : 1;                  // rows a block works on at a time
    const int t = R == 32 ? threadIdx.x & 31 : threadIdx.x;
    const int32_t D = p.D;
    const int64_t step = static_cast<int64_t>(gridDim.x) * G;
    int64_t row = static_cast<int64_t>(blockIdx.x) * G + (R == 32 ? threadIdx.x >> 5 : 0);
    const float inv_d = 1.f / static_cast<float>(D);
    float w[NV][VEC];
    Raw<T, VEC> x[NV], r[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int32_t col = (j * R + t) * VEC;
        if (col < D && row < p.C) {
            x[j] = ld<T, VEC>(p.x, row * D + col);
            if (p.res) r[j] = ld<T, VEC>(p.res, row * D + col);
        }
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int32_t col = (j * R + t) * VEC;
#pragma unroll
        for (int i = 0; i < VEC; ++i) w[j][i] = col < D ? __ldg(p.w + col + i) : 0.f;
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
        const float rstd = __frsqrt_rn(fmaf(row_sum<R>(s, sm[slot]), inv_d, p.eps));
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int32_t col = (j * R + t) * VEC;
            if (col < D) {
                if (p.h) st<T, VEC>(p.h, row * D + col, h[j]);
#pragma unroll
                for (int i = 0; i < VEC; ++i) h[j][i] = h[j][i] * rstd * w[j][i];
                if (p.y) st<T, VEC>(p.y, row * D + col, h[j]);
                if constexpr (MX) store_mx<VEC>(static_cast<uint8_t *>(p.y8), p.scale8, row, D, col, h[j]);
            }
        }
        if (t == 0 && p.rstd) p.rstd[row] = rstd;
    }
}

template <typename T, int VEC, int R, int NV>
__global__ void __launch_bounds__(R == 32 ? 128 : R) rmsnorm_bwd_kernel(NormBwd p) {
    __shared__ float sm[2][R / 32];
    constexpr int G = R == 32 ? 4 : 1;
    const int t = R == 32 ? threadIdx.x & 31 : threadIdx.x;
    const int32_t D = p.D;
    const int64_t step = static_cast<int64_t>(gridDim.x) * G;
    const int64_t group = static_cast<int64_t>(blockIdx.x) * G + (R == 32 ? threadIdx.x >> 5 : 0);
    int64_t row = group;
    const float inv_d = 1.f / static_cast<float>(D);
    float w[NV][VEC], dw[NV][VEC];
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
#pragma unroll
        for (int i = 0; i < VEC; ++i) { w[j][i] = col < D ? __ldg(p.w + col + i) : 0.f; dw[j][i] = 0.f; }
    }
    for (int slot = 0; row < p.C; row += step, slot ^= 1) {
        float g[NV][VEC], n[NV][VEC], d[NV][VEC], s = 0.f;
        const float rs = rstd;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int32_t col = (j * R + t) * VEC;
            if (col < D) {
                unpack(a[j], g[j]);
                unpack(b[j], n[j]);
                if (p.dh) unpack(e[j], d[j]);
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    n[j][i] *= rs;
                    dw[j][i] = fmaf(g[j][i], n[j][i], dw[j][i]);
                    g[j][i] *= w[j][i];
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
        const float m = row_sum<R>(s, sm[slot]) * inv_d;
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
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int32_t col = (j * R + t) * VEC;
        if (col < D)
            for (int i = 0; i < VEC; ++i) p.part[group * D + col + i] = dw[j][i];
    }
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

// Threads of a row: few enough that each keeps up to 16 values (8 of unaligned rows, whose
// loads are single values), but never under a warp.
struct Shape { int vec, r; };
Shape shape_of(int32_t dtype, int32_t D) {
    const int full = dtype == HARTS_BF16 ? 8 : 4;
    Shape s;
    s.vec = D % full == 0 ? full : 1;
    const int per = s.vec == 1 ? 8 : 16;
    s.r = D <= 32 * per ? 32 : D <= 128 * per ? 128 : D <= 256 * per ? 256 : D <= 512 * per ? 512 : 1024;
    return s;
}

// Groups of R threads that work at a time, at most: 1,024 threads an SM.
int64_t group_limit(const Shape &s) {
    return static_cast<int64_t>(sm_count()) * (s.r == 32 ? 4 * 8 : std::max(1, 1024 / s.r));
}
int64_t groups_of(const Shape &s, int64_t C) {
    const int64_t g = std::min<int64_t>(C, group_limit(s));
    return s.r == 32 ? (g + 3) / 4 * 4 : g;
}

template <typename T, int VEC, int R, int NV>
void launch_fwd(const NormFwd &p, int grid, cudaStream_t st) {
    if constexpr (VEC > 1) {
        if (p.y8) {
            rmsnorm_fwd_kernel<T, VEC, R, NV, true><<<grid, R == 32 ? 128 : R, 0, st>>>(p);
            return;
        }
    }
    rmsnorm_fwd_kernel<T, VEC, R, NV, false><<<grid, R == 32 ? 128 : R, 0, st>>>(p);
}
template <typename T, int VEC, int R, int NV>
void launch_bwd(const NormBwd &p, int grid, cudaStream_t st) {
    rmsnorm_bwd_kernel<T, VEC, R, NV><<<grid, R == 32 ? 128 : R, 0, st>>>(p);
}

#define HARTS_NORM_DISPATCH(LAUNCH, T, VEC, NV, p, s, grid, st)                                     \
    do {                                                                                            \
        if ((s).r == 32) LAUNCH<T, VEC, 32, NV>(p, grid, st);                                       \
        else if ((s).r == 128) LAUNCH<T, VEC, 128, NV>(p, grid, st);                                \
        else if ((s).r == 256) LAUNCH<T, VEC, 256, NV>(p, grid, st);                                \
        else if ((s).r == 512) LAUNCH<T, VEC, 512, NV>(p, grid, st);                                \
        else if (VEC > 1 || (p).D <= 8192) LAUNCH<T, VEC, 1024, NV>(p, grid, st);                   \
        else LAUNCH<T, VEC, 1024, VEC == 1 ? 16 : NV>(p, grid, st);                                 \
    } while (0)

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

int check_common(int64_t C, int32_t D, int32_t dtype) {
    if (dtype != HARTS_FP32 && dtype != HARTS_BF16) { set_error("dtype"); return HARTS_EUNSUPPORTED; }
    if (C < 0 || D < 1) { set_error("C >= 0 and D >= 1 required"); return HARTS_EINVAL; }
    if (D > kMaxDim) { set_error("D above 16384"); return HARTS_EUNSUPPORTED; }
    return HARTS_OK;
}

int launched(const char *what) {
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) { set_error(std::string(what) + ": " + cudaGetErrorString(e)); return HARTS_ECUDA; }
    set_error("");
    return HARTS_OK;
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
    if ((a->y8 == nullptr) != (a->y8_scale == nullptr)) { set_error("y8 and y8_scale go together"); return HARTS_EINVAL; }
    if (a->y8 && a->D % kMxBlock) { set_error("the 8-bit output needs D a multiple of 32"); return HARTS_EUNSUPPORTED; }
    if (!aligned16(a->x) || !aligned16(a->residual) || !aligned16(a->h) || !aligned16(a->y) || !aligned16(a->y8)) {
        set_error("x, residual, h, y and y8 must be 16-byte aligned");
        return HARTS_EINVAL;
    }
    NormFwd p;
    p.x = a->x; p.res = a->residual; p.w = a->weight; p.h = a->h; p.y = a->y; p.y8 = a->y8;
    p.scale8 = static_cast<uint8_t *>(a->y8_scale); p.rstd = a->rstd; p.C = a->C; p.D = a->D; p.eps = a->eps;
    const Shape s = shape_of(a->dtype, a->D);
    const int64_t groups = groups_of(s, a->C);
    const int grid = static_cast<int>(s.r == 32 ? groups / 4 : groups);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (a->dtype == HARTS_BF16) {
        if (s.vec == 8) HARTS_NORM_DISPATCH(launch_fwd, __nv_bfloat16, 8, 2, p, s, grid, st);
        else HARTS_NORM_DISPATCH(launch_fwd, __nv_bfloat16, 1, 8, p, s, grid, st);
    } else {
        if (s.vec == 4) HARTS_NORM_DISPATCH(launch_fwd, float, 4, 4, p, s, grid, st);
        else HARTS_NORM_DISPATCH(launch_fwd, float, 1, 8, p, s, grid, st);
    }
    return launched("rmsnorm forward launch");
}

size_t harts_rmsnorm_bwd_workspace_bytes(int64_t C, int32_t D, int32_t dtype) {
    if (C < 0 || D < 1 || D > kMaxDim || (dtype != HARTS_FP32 && dtype != HARTS_BF16)) return 0;
    return std::max<size_t>(256, sizeof(float) * static_cast<size_t>(groups_of(shape_of(dtype, D), C)) * D);
}

int harts_rmsnorm_bwd(const harts_rmsnorm_bwd_args *a, harts_stream_t stream) {
    if (!a) { set_error("NULL args"); return HARTS_EINVAL; }
    const int rc = check_common(a->C, a->D, a->dtype);
    if (rc) return rc;
    if (!a->dweight) { set_error("NULL dweight"); return HARTS_EINVAL; }
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (a->C == 0) {
        const cudaError_t e = cudaMemsetAsync(a->dweight, 0, sizeof(float) * a->D, st);
        if (e != cudaSuccess) { set_error(std::string("rmsnorm backward: ") + cudaGetErrorString(e)); return HARTS_ECUDA; }
        set_error("");
        return HARTS_OK;
    }
    if (!a->dy || !a->h || !a->weight || !a->rstd || !a->dx) { set_error("NULL dy, h, weight, rstd or dx"); return HARTS_EINVAL; }
    if (!aligned16(a->dy) || !aligned16(a->h) || !aligned16(a->dh) || !aligned16(a->dx) || !aligned16(a->workspace)) {
        set_error("dy, h, dh, dx and workspace must be 16-byte aligned");
        return HARTS_EINVAL;
    }
    if (!a->workspace || a->workspace_bytes < harts_rmsnorm_bwd_workspace_bytes(a->C, a->D, a->dtype)) {
        set_error("workspace too small");
        return HARTS_ESMALLBUF;
    }
    NormBwd p;
    p.dy = a->dy; p.h = a->h; p.dh = a->dh; p.w = a->weight; p.rstd = a->rstd; p.dx = a->dx;
    p.part = static_cast<float *>(a->workspace); p.C = a->C; p.D = a->D;
    const Shape s = shape_of(a->dtype, a->D);
    const int64_t groups = groups_of(s, a->C);
    const int grid = static_cast<int>(s.r == 32 ? groups / 4 : groups);
    if (a->dtype == HARTS_BF16) {
        if (s.vec == 8) HARTS_NORM_DISPATCH(launch_bwd, __nv_bfloat16, 8, 2, p, s, grid, st);
        else HARTS_NORM_DISPATCH(launch_bwd, __nv_bfloat16, 1, 8, p, s, grid, st);
    } else {
        if (s.vec == 4) HARTS_NORM_DISPATCH(launch_bwd, float, 4, 4, p, s, grid, st);
        else HARTS_NORM_DISPATCH(launch_bwd, float, 1, 8, p, s, grid, st);
    }
    const int ok = launched("rmsnorm backward launch");
    if (ok) return ok;
    const DwParams d{p.part, a->dweight, a->D, static_cast<int32_t>(groups)};
    const cudaError_t e = launch(rmsnorm_dw_kernel, (a->D + 31) / 32, 1024, 0, 1, true, st, d);
    if (e != cudaSuccess) { set_error(std::string("rmsnorm backward launch: ") + cudaGetErrorString(e)); return HARTS_ECUDA; }
    return HARTS_OK;
}

}  // extern "C"
