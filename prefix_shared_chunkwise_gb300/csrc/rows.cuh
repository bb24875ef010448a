// Row-wise kernels: values of a row as they lie in memory, sums over the threads that share a row,
// and rows copied ahead into shared memory.
#pragma once
#include <cuda_bf16.h>

#include <cstdint>

#include "tc_primitives.cuh"

namespace harts {
namespace rows {

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

__device__ __forceinline__ void bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                 :: "r"(tc::smem_addr(dst)), "l"(src), "r"(bytes), "r"(tc::smem_addr(bar)) : "memory");
}

// The same for what nobody reads again: it leaves L2 first, and does not drive out what is on its way to memory.
__device__ __forceinline__ void bulk_load_once(void *dst, const void *src, uint32_t bytes, uint64_t *bar) {
    uint64_t policy;
    asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;"
                 :: "r"(tc::smem_addr(dst)), "l"(src), "r"(bytes), "r"(tc::smem_addr(bar)), "l"(policy) : "memory");
}

}  // namespace rows
}  // namespace harts
