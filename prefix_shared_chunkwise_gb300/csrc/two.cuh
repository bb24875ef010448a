// fp32 arithmetic on pairs of values (one instruction for two), and the same names for single ones.
#pragma once
#include <cstdint>
#include <cstring>

namespace harts {
namespace two {

using Two = float2;
__device__ __forceinline__ uint64_t bits_of(Two a) { uint64_t u; memcpy(&u, &a, 8); return u; }
__device__ __forceinline__ Two two_of(uint64_t u) { Two a; memcpy(&a, &u, 8); return a; }
__device__ __forceinline__ Two fma(Two a, Two b, Two c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(bits_of(a)), "l"(bits_of(b)), "l"(bits_of(c)));
    return two_of(d);
}
__device__ __forceinline__ Two mul(Two a, Two b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(bits_of(a)), "l"(bits_of(b)));
    return two_of(d);
}
__device__ __forceinline__ Two add(Two a, Two b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(bits_of(a)), "l"(bits_of(b)));
    return two_of(d);
}
__device__ __forceinline__ float fma(float a, float b, float c) { return fmaf(a, b, c); }
__device__ __forceinline__ float mul(float a, float b) { return a * b; }
__device__ __forceinline__ float add(float a, float b) { return a + b; }
template <typename F> __device__ __forceinline__ Two each(Two a, F f) { return make_float2(f(a.x), f(a.y)); }
template <typename F> __device__ __forceinline__ float each(float a, F f) { return f(a); }
template <typename F> __device__ __forceinline__ Two each(Two a, Two b, F f) { return make_float2(f(a.x, b.x), f(a.y, b.y)); }
template <typename F> __device__ __forceinline__ float each(float a, float b, F f) { return f(a, b); }
template <typename F> __device__ __forceinline__ Two each(Two a, Two b, Two c, F f) { return make_float2(f(a.x, b.x, c.x), f(a.y, b.y, c.y)); }
template <typename F> __device__ __forceinline__ float each(float a, float b, float c, F f) { return f(a, b, c); }
__device__ __forceinline__ float total(Two a) { return a.x + a.y; }
__device__ __forceinline__ float total(float a) { return a; }

}  // namespace two
}  // namespace harts
