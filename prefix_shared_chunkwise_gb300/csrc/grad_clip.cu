// The global norm of many gradient tensors, and clipping by it.
//
//   n = sqrt(sum_i sum_j g_ij^2),   out_i = g_i * (n > max_norm ? max_norm / n : 1)
// Two kernels over the same spans of all tensors: squares (each block leaves one fp64 partial
// sum), then the scaling, whose blocks each add up the partials in the same fixed order -- a few
// kilobytes from L2 -- so that clipping needs neither atomics nor a launch for the norm.  (The
// norm alone has a second, one-warp kernel.)  The scaling walks the spans backwards: what the first kernel read
// last is still in L2, and outputs are stored as the first to leave it.  Both kernels only
// stream: HBM bounds them, two reads and one write of every value for sets larger than L2, one
// read and one write below that.
//
// Squares are summed in fp32 over the 16 to 32 values that a thread loads at a time and in fp64
// from there on.  A block whose sum is not finite reads its spans again in fp64: squares overflow
// fp32 from 1.8e19 on, which bf16 and fp32 values reach.  So does
// one whose sum is below 2^-90 and not one of zeros: a square below 2^-126 loses up to 2^-150,
// which over the 2^34 values that a block has at most is 2^-26 of such a sum, and more of a
// smaller one.  (Whether values are zeros is looked at where their squares are: doing so for all
// of them took 4 % of the sum's time.)  If the norm itself is not finite the gradients pass
// through unscaled; the caller sees it in the norm.
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>
#include <string>
#include <type_traits>

#include "launch_util.h"
#include "plan_internal.h"

namespace harts {
namespace {

constexpr int kThreads = 256;
constexpr int kSet = 512;                   // tensors a launch carries in its parameters
constexpr int64_t kChunk = 2048;            // values; shares are whole chunks of a tensor
constexpr int kPerSm = 6;                   // resident blocks

struct Item {
    const void *g;
    void *out;
    int64_t n;
    int32_t chunk0;                         // first chunk of the tensor within the launch
    int32_t kinds;                          // bit 0: g is bf16, bit 1: out is bf16
};

struct Set {
    Item item[kSet];
    int32_t count, chunks, chunk, partials;
    int32_t span, spans;                    // consecutive chunks that a block takes at a time, and how many such
    int32_t first;                          // index of the launch's first partial
    float max_norm;
    float *norm;
    double *part;
};

__device__ __forceinline__ int find(const Set &s, int32_t c) {
    int lo = 0, hi = s.count - 1;           // last item whose chunk0 <= c
    while (lo < hi) {
        const int m = (lo + hi + 1) >> 1;
        if (s.item[m].chunk0 <= c) lo = m; else hi = m - 1;
    }
    return lo;
}

__device__ __forceinline__ float get(const float *p) { return *p; }
__device__ __forceinline__ float get(const __nv_bfloat16 *p) { return __bfloat162float(*p); }
__device__ __forceinline__ void put(float *p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }

template <typename T> struct Pack { static constexpr int n = 16 / sizeof(T); };

__device__ __forceinline__ void expand(uint4 u, float (&v)[8], const __nv_bfloat16 *) {
    const __nv_bfloat162 *p = reinterpret_cast<const __nv_bfloat162 *>(&u);
#pragma unroll
    for (int i = 0; i < 4; ++i) { const float2 f = __bfloat1622float2(p[i]); v[2 * i] = f.x; v[2 * i + 1] = f.y; }
}
__device__ __forceinline__ void expand(uint4 u, float (&v)[4], const float *) {
    v[0] = __uint_as_float(u.x); v[1] = __uint_as_float(u.y); v[2] = __uint_as_float(u.z); v[3] = __uint_as_float(u.w);
}
// Values before the first 16-byte boundary at or after p.
template <typename T>
__device__ __forceinline__ int64_t head_of(const T *p, int64_t n) {
    const int64_t h = ((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) / static_cast<int64_t>(sizeof(T));
    return h < n ? h : n;
}

// The bits of a pack that are set where a value is not zero.
__device__ __forceinline__ uint32_t magnitude(uint4 u, const __nv_bfloat16 *) { return (u.x | u.y | u.z | u.w) & 0x7fff7fffu; }
__device__ __forceinline__ uint32_t magnitude(uint4 u, const float *) { return (u.x | u.y | u.z | u.w) & 0x7fffffffu; }

// This thread's part of the sum; WIDE: all of it in fp64.  `seen` is set where values are not zero
// whose fp32 squares are.
template <bool WIDE, typename T>
__device__ double squares(const T *g, int64_t n, uint32_t &seen) {
    constexpr int N = Pack<T>::n;
    const int t = threadIdx.x;
    const int64_t head = head_of(g, n);
    double sum = 0.0;
    const uint4 *q = reinterpret_cast<const uint4 *>(g + head);
    const int64_t nv = (n - head) / N, tail = head + nv * N + t;
    if (t < head || tail < n) {
        const float a = t < head ? get(g + t) : 0.f, b = tail < n ? get(g + tail) : 0.f;
        if (WIDE) sum = static_cast<double>(a) * a + static_cast<double>(b) * b;
        else sum = fmaf(a, a, b * b);
        seen |= (a != 0.f) | (b != 0.f);
    }
    for (int64_t i = t; i < nv; i += 4 * kThreads) {
        uint4 u[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            u[k] = i + k * kThreads < nv ? __ldg(q + i + k * kThreads) : make_uint4(0, 0, 0, 0);
        if constexpr (WIDE) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                float v[N];
                expand(u[k], v, g);
#pragma unroll
                for (int j = 0; j < N; ++j) sum = fma(static_cast<double>(v[j]), static_cast<double>(v[j]), sum);
            }
        } else {
            float s0 = 0.f, s1 = 0.f, s2 = 0.f, s3 = 0.f;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                float v[N];
                expand(u[k], v, g);
#pragma unroll
                for (int j = 0; j < N; j += 4) {
                    s0 = fmaf(v[j], v[j], s0); s1 = fmaf(v[j + 1], v[j + 1], s1);
                    s2 = fmaf(v[j + 2], v[j + 2], s2); s3 = fmaf(v[j + 3], v[j + 3], s3);
                }
            }
            const float s = (s0 + s1) + (s2 + s3);
            if (s == 0.f) seen |= magnitude(u[0], g) | magnitude(u[1], g) | magnitude(u[2], g) | magnitude(u[3], g);
            sum += s;
        }
    }
    return sum;
}

// Sum over the block in a fixed order; thread 0 returns it.  GB300 has few fp64 units (the norm of
// 600 M bf16 values takes 0.18 ms, and 2.4 ms more where all squares have to be summed in fp64),
// so fp64 is kept to one addition per 64 bytes a thread loads, one such sum a block, and one warp
// for the norm.
__device__ double block_sum(double v, double *sm) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = v;
    __syncthreads();
    double s = 0.0;
    if (threadIdx.x == 0)
        for (int i = 0; i < kThreads / 32; ++i) s += sm[i];
    return s;
}

// The part of chunks [c, end) that lies in item k: its first value and how many.
__device__ __forceinline__ int64_t run_of(const Set &s, int k, int32_t c, int32_t end, int64_t *at) {
    const Item &it = s.item[k];
    *at = static_cast<int64_t>(c - it.chunk0) * s.chunk;
    const int64_t n = static_cast<int64_t>(end - c) * s.chunk;
    return it.n - *at < n ? it.n - *at : n;
}

__global__ void __launch_bounds__(kThreads, kPerSm) grad_squares_kernel(const __grid_constant__ Set s) {
    __shared__ double sm[kThreads / 32];
    __shared__ int s_wide;
    let_next_start();
    double sum = 0.0;
    uint32_t seen = 0;
    for (int wide = 0; wide < 2; ++wide) {
        sum = 0.0;
        for (int32_t j = blockIdx.x; j < s.spans; j += gridDim.x) {
            int32_t c = j * s.span;
            const int32_t end = min(c + s.span, s.chunks);
            for (int k = find(s, c); c < end; ++k) {
                const int32_t stop = k + 1 < s.count && s.item[k + 1].chunk0 < end ? s.item[k + 1].chunk0 : end;
                int64_t at;
                const int64_t n = run_of(s, k, c, stop, &at);
                const __nv_bfloat16 *b = static_cast<const __nv_bfloat16 *>(s.item[k].g) + at;
                const float *f = static_cast<const float *>(s.item[k].g) + at;
                if (wide) sum += s.item[k].kinds & 1 ? squares<true>(b, n, seen) : squares<true>(f, n, seen);
                else sum += s.item[k].kinds & 1 ? squares<false>(b, n, seen) : squares<false>(f, n, seen);
                c = stop;
            }
        }
        sum = block_sum(sum, sm);
        const int some = __syncthreads_or(seen != 0);
        if (threadIdx.x == 0) s_wide = !isfinite(sum) || (sum < 0x1p-90 && (sum > 0.0 || some));
        __syncthreads();
        if (!s_wide) break;
    }
    if (threadIdx.x == 0) s.part[s.first + blockIdx.x] = sum;
}

// The norm from the partial sums, by one warp in a fixed order; all lanes return it.
__device__ double norm_of(const double *part, int32_t partials) {
    double v = 0.0;
#pragma unroll 4
    for (int32_t i = threadIdx.x; i < partials; i += 32) v += part[i];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return sqrt(v);
}

__global__ void __launch_bounds__(32) grad_norm_kernel(const double *part, int32_t partials, float *norm) {
    const double n = norm_of(part, partials);
    if (threadIdx.x == 0) *norm = static_cast<float>(n);
}

// Stores that leave L2 first: the gradients that are still to be read should stay.
template <int N>
__device__ __forceinline__ void store_pack(float *p, const float (&v)[N]) {
#pragma unroll
    for (int i = 0; i < N; i += 4) __stcs(reinterpret_cast<float4 *>(p + i), make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]));
}
template <int N>
__device__ __forceinline__ void store_pack(__nv_bfloat16 *p, const float (&v)[N]) {
    uint32_t u[N / 2];
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        u[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    if constexpr (N == 8) __stcs(reinterpret_cast<uint4 *>(p), make_uint4(u[0], u[1], u[2], u[3]));
    else __stcs(reinterpret_cast<uint2 *>(p), make_uint2(u[0], u[1]));
}

// Packs of as many values as 16 bytes hold of the wider type: loads and stores of a warp are
// then contiguous in both.
template <typename T, typename U> struct Packs {
    static constexpr int n = 16 / (sizeof(T) > sizeof(U) ? sizeof(T) : sizeof(U));
    using Load = std::conditional_t<n * sizeof(T) == 16, uint4, uint2>;
};
__device__ __forceinline__ void expand(uint2 u, float (&v)[4], const __nv_bfloat16 *) {
    const __nv_bfloat162 *p = reinterpret_cast<const __nv_bfloat162 *>(&u);
#pragma unroll
    for (int i = 0; i < 2; ++i) { const float2 f = __bfloat1622float2(p[i]); v[2 * i] = f.x; v[2 * i + 1] = f.y; }
}
template <typename T, typename U>
__device__ __forceinline__ void scale_pack(typename Packs<T, U>::Load u, U *out, float f) {
    constexpr int N = Packs<T, U>::n;
    float v[N];
    expand(u, v, static_cast<const T *>(nullptr));
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] *= f;
    store_pack(out, v);
}

// Packs from the last to the first, four a thread on their way at a time; what lies before and
// behind them, and outputs that do not start on their gradient's boundary, value by value.
template <typename T, typename U>
__device__ __forceinline__ void scale(const T *g, U *out, int64_t n, float f) {
    constexpr int N = Packs<T, U>::n;
    using Load = typename Packs<T, U>::Load;
    const int64_t head = head_of(g, n);
    int64_t nv = (n - head) / N;
    if (reinterpret_cast<uintptr_t>(out + head) & 15) nv = 0;
    const Load *q = reinterpret_cast<const Load *>(g + head);
    U *o = out + head;
    constexpr int32_t kStep = 4 * kThreads;
    const int64_t full = nv / kStep * kStep;
    for (int64_t i = full + threadIdx.x; i < nv; i += kThreads) scale_pack<T>(__ldcs(q + i), o + i * N, f);
    for (int64_t i = full - kStep + threadIdx.x; i >= 0; i -= kStep) {
        const Load *s = q + i;
        U *d = o + i * N;
        const Load u0 = __ldcs(s), u1 = __ldcs(s + kThreads), u2 = __ldcs(s + 2 * kThreads), u3 = __ldcs(s + 3 * kThreads);
        scale_pack<T>(u0, d, f);
        scale_pack<T>(u1, d + kThreads * N, f);
        scale_pack<T>(u2, d + 2 * kThreads * N, f);
        scale_pack<T>(u3, d + 3 * kThreads * N, f);
    }
    if (threadIdx.x < head) put(out + threadIdx.x, get(g + threadIdx.x) * f);
    for (int64_t i = head + nv * N + threadIdx.x; i < n; i += kThreads) put(out + i, get(g + i) * f);
}

// With a coefficient that fp32 holds with few bits or as zero: value by value, by fp64.
template <typename T, typename U>
__device__ void scale64(const T *g, U *out, int64_t n, double f) {
    for (int64_t i = threadIdx.x; i < n; i += kThreads) put(out + i, static_cast<float>(get(g + i) * f));
}

__global__ void __launch_bounds__(kThreads, kPerSm) grad_scale_kernel(const __grid_constant__ Set s) {
    __shared__ float s_f;
    __shared__ double s_f64;
    wait_previous();
    if (threadIdx.x < 32) {
        const double norm = norm_of(s.part, s.partials);
        if (threadIdx.x == 0) {
            const float told = static_cast<float>(norm);     // what the caller sees decides
            s_f64 = norm > s.max_norm && isfinite(told) ? s.max_norm / norm : 1.0;
            s_f = static_cast<float>(s_f64);
            if (blockIdx.x == 0 && s.first == 0) *s.norm = told;
        }
    }
    __syncthreads();
    const float f = s_f;
    const bool tiny = f < 0x1p-126f && s_f64 > 0.0;
    for (int32_t j = s.spans - 1 - static_cast<int32_t>(blockIdx.x); j >= 0; j -= gridDim.x) {
        const int32_t begin = j * s.span;
        int32_t end = min(begin + s.span, s.chunks);
        for (int k = find(s, end - 1); end > begin; --k) {
            const Item &it = s.item[k];
            const int32_t c = it.chunk0 > begin ? it.chunk0 : begin;
            int64_t at;
            const int64_t n = run_of(s, k, c, end, &at);
            end = c;
            if (f == 1.f && it.out == it.g) continue;       // in place and nothing to scale
            const __nv_bfloat16 *gb = static_cast<const __nv_bfloat16 *>(it.g) + at;
            const float *gf = static_cast<const float *>(it.g) + at;
            __nv_bfloat16 *ob = static_cast<__nv_bfloat16 *>(it.out) + at;
            float *of = static_cast<float *>(it.out) + at;
            if (tiny) {
                switch (it.kinds) {
                    case 0: scale64(gf, of, n, s_f64); break;
                    case 1: scale64(gb, of, n, s_f64); break;
                    case 2: scale64(gf, ob, n, s_f64); break;
                    default: scale64(gb, ob, n, s_f64); break;
                }
                continue;
            }
            switch (it.kinds) {
                case 0: scale(gf, of, n, f); break;
                case 1: scale(gb, of, n, f); break;
                case 2: scale(gf, ob, n, f); break;
                default: scale(gb, ob, n, f); break;
            }
        }
    }
}

int grid_limit() { return sm_count() * kPerSm; }

// Chunks that a block takes at a time.  Blocks go round the spans in turn, so that all of them
// read and write near each other (600 M bf16 values: spans of 16 chunks 565 us, 4 chunks 588,
// one contiguous share a block 573), and of 8 .. 24 chunks the span is taken that leaves the
// busiest block the fewest (22.7 M fp32 values: 46 us, against 67 with spans of fixed size).
int32_t span_of(int32_t chunks) {
    const int32_t grid = grid_limit(), each = (chunks + grid - 1) / grid;
    if (each <= 8) return std::max(1, each);
    int32_t best = 8;
    int64_t least = INT64_MAX;
    for (int32_t k = 8; k <= 24; ++k) {
        const int64_t busiest = int64_t(k) * ((chunks + int64_t(k) * grid - 1) / (int64_t(k) * grid));
        if (busiest < least) { least = busiest; best = k; }
    }
    return best;
}

// The arguments of either call; 0 or an error code.  `total` receives the number of values.
int check(const harts_grad_tensor *t, int32_t count, bool clip, int64_t *total) {
    if (count < 0 || (count > 0 && !t)) { set_error("count >= 0 and a tensor list required"); return HARTS_EINVAL; }
    *total = 0;
    for (int32_t i = 0; i < count; ++i) {
        if (t[i].n < 0) { set_error("negative length"); return HARTS_EINVAL; }
        if (t[i].dtype != HARTS_FP32 && t[i].dtype != HARTS_BF16) { set_error("dtype"); return HARTS_EUNSUPPORTED; }
        if (t[i].n == 0) continue;
        if (!t[i].g || (clip && !t[i].out)) { set_error("NULL gradient or output"); return HARTS_EINVAL; }
        const uintptr_t ga = t[i].dtype == HARTS_BF16 ? 1 : 3;
        if (reinterpret_cast<uintptr_t>(t[i].g) & ga) { set_error("gradient not aligned to its type"); return HARTS_EINVAL; }
        if (clip) {
            if (t[i].out_dtype != HARTS_FP32 && t[i].out_dtype != HARTS_BF16) { set_error("output dtype"); return HARTS_EUNSUPPORTED; }
            const uintptr_t oa = t[i].out_dtype == HARTS_BF16 ? 1 : 3;
            if (reinterpret_cast<uintptr_t>(t[i].out) & oa) { set_error("output not aligned to its type"); return HARTS_EINVAL; }
            if (t[i].out == t[i].g && t[i].out_dtype != t[i].dtype) { set_error("in place needs one dtype"); return HARTS_EINVAL; }
        }
        if (t[i].n > (int64_t(1) << 44) - *total) { set_error("more than 2^44 values"); return HARTS_EOVERFLOW; }
        *total += t[i].n;
    }
    return HARTS_OK;
}

// Values of a chunk: chunks are counted in 32 bits.
int32_t chunk_of(int64_t total) {
    int64_t c = kChunk;
    while (total / c > (int64_t(1) << 29)) c *= 2;
    return static_cast<int32_t>(c);
}

int run(const harts_grad_tensor *t, int32_t count, bool clip, float max_norm, float *norm, void *ws, size_t ws_bytes,
        cudaStream_t st) {
    int64_t total = 0;
    const int rc = check(t, count, clip, &total);
    if (rc) return rc;
    if (!norm) { set_error("NULL norm"); return HARTS_EINVAL; }
    if (clip && !(max_norm >= 0.f)) { set_error("max_norm must be >= 0"); return HARTS_EINVAL; }
    if (!ws || ws_bytes < harts_grad_workspace_bytes(count)) { set_error("workspace too small"); return HARTS_ESMALLBUF; }
    if (reinterpret_cast<uintptr_t>(ws) & 15) { set_error("workspace must be 16-byte aligned"); return HARTS_EINVAL; }
    const int32_t chunk = chunk_of(total);
    static thread_local Set s;              // 20 KB: passed by value to each launch
    s.chunk = chunk; s.max_norm = max_norm; s.norm = norm; s.part = static_cast<double *>(ws);
    int32_t partials = 0;
    for (int pass = 0; pass < (clip ? 2 : 1); ++pass) {
        int32_t first = 0, i = 0;
        do {
            s.count = s.chunks = 0;
            for (; i < count && s.count < kSet; ++i) {
                if (t[i].n == 0) continue;
                const int64_t c = (t[i].n + chunk - 1) / chunk;
                Item &it = s.item[s.count++];
                it.g = t[i].g; it.out = t[i].out; it.n = t[i].n; it.chunk0 = s.chunks;
                it.kinds = (t[i].dtype == HARTS_BF16 ? 1 : 0) | (t[i].out_dtype == HARTS_BF16 ? 2 : 0);
                s.chunks += static_cast<int32_t>(c);
            }
            s.span = span_of(s.chunks);
            s.spans = (s.chunks + s.span - 1) / s.span;
            const int grid = std::max(1, std::min(s.spans, grid_limit()));
            s.first = first;
            s.partials = partials;
            // the first scaling is set up while the last squares are summed
            const cudaError_t e = pass == 0 ? launch(grad_squares_kernel, grid, kThreads, 0, 1, false, st, s)
                                            : launch(grad_scale_kernel, grid, kThreads, 0, 1, first == 0, st, s);
            if (e != cudaSuccess) { set_error(std::string("gradient norm launch: ") + cudaGetErrorString(e)); return HARTS_ECUDA; }
            first += grid;
        } while (i < count);
        partials = first;
    }
    if (!clip) grad_norm_kernel<<<1, 32, 0, st>>>(s.part, partials, norm);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) { set_error(std::string("gradient norm launch: ") + cudaGetErrorString(e)); return HARTS_ECUDA; }
    set_error("");
    return HARTS_OK;
}

}  // namespace
}  // namespace harts

using namespace harts;

extern "C" {

size_t harts_grad_workspace_bytes(int32_t count) {
    if (count < 0) return 0;
    const size_t sets = std::max<int64_t>(1, (int64_t(count) + kSet - 1) / kSet);
    return std::max<size_t>(256, sets * grid_limit() * sizeof(double));
}

int harts_grad_norm(const harts_grad_tensor *t, int32_t count, float *norm, void *workspace, size_t workspace_bytes,
                    harts_stream_t stream) {
    return run(t, count, false, 0.f, norm, workspace, workspace_bytes, reinterpret_cast<cudaStream_t>(stream));
}

int harts_grad_clip(const harts_grad_tensor *t, int32_t count, float max_norm, float *norm, void *workspace,
                    size_t workspace_bytes, harts_stream_t stream) {
    return run(t, count, true, max_norm, norm, workspace, workspace_bytes, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
