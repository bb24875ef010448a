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
// sums.  Rows are copied ahead by cp.async.bulk into a ring in shared memory, whose bytes on their way
// do not depend on registers; short rows share a warp.  Blocks are persistent.  Forward, the weights of a thread's
// columns stay in its registers.  Backward, their gradients do, beside weights in shared memory (in registers too
// where rows are not whole vectors); above 4,096 channels the gradients are in shared memory and the weights are read
// where they are, through L1.  A block leaves one row of those gradients, a
// second kernel adds them in ascending order: no atomics, the same bits on every run.
//
// bf16, 65,536 rows of 2,048 channels with everything: forward 216 us (92 % of the copy's rate), backward 325 (97 %);
// 1,048,560 heads of 128 with norm and gate 132 (90 %) and 212 (93 %); fp32, 32,768 x 2,048: 222 (89 %) and 349 (91 %).
// Far from it are 8,192 channels backward (bf16 71 %, fp32 65 %: one row of a block at a time, on its way and in work)
// and bf16 rows that are not whole vectors, which instructions bound (see RAGGED).  One row of 2,048: 2.2 us on the device.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstring>
#include <type_traits>

#include "kda_common.cuh"
#include "launch_util.h"
#include "rows.cuh"
#include "tc_primitives.cuh"
#include "two.cuh"

namespace harts {
namespace {

using namespace rows;
using namespace two;

constexpr int kMaxDim = 8192;       // 512 threads x 16 values
constexpr int kMaxStages = 2;       // rows copied ahead

struct Fwd {
    const void *in[3];              // y; gate; residual
    const float *w1, *w2;
    void *h, *n;
    float *r1, *r2;
    int32_t *error;
    int64_t C, whole_end, whole_rows;   // values in whole vectors of a tensor, and the rows that end before that
    int32_t D, act;
    float scale, eps;
};

struct Bwd {
    const void *in[5];              // y; gate; dn; h; dh
    const float *w1, *w2, *r1, *r2;
    void *dy, *dgate, *dres;
    float *part;                    // [groups][2 D]: of w1, of w2
    int32_t *error;
    int64_t C, whole_end, whole_rows;
    int32_t D, act;
    float scale;
};

// A thread's values of one vector, in pairs.
template <int VEC> struct Vals {
    using E = Two;
    static constexpr int n = VEC / 2;
    E e[n];
};
template <int VEC> __device__ __forceinline__ typename Vals<VEC>::E all(float c) { return make_float2(c, c); }
template <typename T, int VEC> __device__ __forceinline__ void open(const Raw<T, VEC> &r, Vals<VEC> &v) {
    if constexpr (sizeof(T) == 2 && VEC == 8) {
        const uint32_t *u = &r.u.x;
#pragma unroll
        for (int i = 0; i < 4; ++i) v.e[i] = make_float2(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xffff0000u));
    } else {
        unpack(r, reinterpret_cast<float *>(v.e));
    }
}

// Rows that are not whole vectors (RAGGED) begin anywhere: they are copied with what shares their first
// and last 16 bytes, and a thread's "vector" is four words (one fp32 value or two of bf16) that lie R
// words apart.  A bf16 row that begins in the middle of a word has a first one that is half its own, and any
// row may have such a last one: the other half is taken as zero and not written.  (With everything,
// forward and backward: bf16 65,536 x 2,001 275 and 580 us, 131,072 x 1,001 302 and 580, 250,000 x 500 289 and 615,
// 1,000,000 x 131 479 and 903; fp32 32,768 x 2,001 231 and 358.  One value per thread at a time instead, straight from
// memory: 485 and 922, 736 and 1,391, 1,179 and 2,269, 713 and 1,013, 254 and 496.  Whole vectors, what is not the row's
// own masked out at the edges: 296 and 608, 365 and 567, 327 and 678, 773 and 1,400, 284 and 401.)
template <typename T> constexpr int kWord = 4 / sizeof(T);                        // values of a word
template <typename T, int VEC, int R, bool RAGGED> __device__ __forceinline__ int32_t col_of(int j, int t, int into) {
    return RAGGED ? j * VEC * R + t * kWord<T> - into : (j * R + t) * VEC;
}
template <typename T, int R, bool RAGGED> __device__ __forceinline__ int32_t value_of(int i) {   // a vector's i-th value, behind its first
    return RAGGED ? i / kWord<T> * R * kWord<T> + i % kWord<T> : i;
}
// Pairs of a vector that any of the R threads has something in; shape_of gives a row as few threads and
// values as it takes, so that a thread's first half is always its own (SURE).
template <typename T, int VEC, int R> __device__ __forceinline__ int pairs_of(int j, int32_t D) {
    return min(max((D + kWord<T> - 1 - j * VEC * R + 2 * R - 1) / (2 * R), 0), VEC / 2);
}
template <int VEC, int R, int NV, bool RAGGED> __device__ __forceinline__ constexpr bool sure(int j, int i) {
    return !RAGGED || (R > 8 && (j * VEC + 2 * i + 2) * 2 <= NV * VEC);
}
// at: the place of the row's first value; pairs: those of the vector
template <typename T, int VEC, int R, int NV, bool RAGGED> __device__ __forceinline__ void put(void *p, int64_t at, int j, int32_t col, int32_t D, int pairs, const Vals<VEC> &v) {
    if constexpr (RAGGED) {
        Raw<T, VEC> r;
        pack(r, reinterpret_cast<const float *>(v.e));
        const uint32_t *u = reinterpret_cast<const uint32_t *>(&r.u);
        uint32_t *words = reinterpret_cast<uint32_t *>(static_cast<T *>(p) + at + col);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int i = k * kWord<T> / 2;
            if (!sure<VEC, R, NV, true>(j, i) && i >= pairs) break;
            const int32_t c = col + k * R * kWord<T>;
            if constexpr (sizeof(T) == 4) {
                if (sure<VEC, R, NV, true>(j, i) || c < D) words[k * R] = u[k];
            } else {
                const bool first = j == 0 && k == 0 && c < 0;
                if (!first && (sure<VEC, R, NV, true>(j, i) || c + 1 < D)) words[k * R] = u[k];
                if (j == 0 && k == 0 && first) reinterpret_cast<uint16_t *>(words)[1] = static_cast<uint16_t>(u[k] >> 16);
                if (!sure<VEC, R, NV, true>(j, i) && !first && c + 1 == D) reinterpret_cast<uint16_t *>(words)[2 * k * R] = static_cast<uint16_t>(u[k]);
            }
        }
    } else {
        st<T, VEC>(p, at + col, reinterpret_cast<const float *>(v.e));
    }
}
// Of a tensor whose size is not a whole vector, the last values are not among what was copied: `in`, from memory.
template <typename T, int VEC, int R, int NV, bool RAGGED> __device__ __forceinline__ Raw<T, VEC> take(const T *buf, const T *in, bool last, int j, int32_t col, int32_t D, int pairs) {
    if constexpr (RAGGED) {
        Raw<T, VEC> r;
        uint32_t *u = reinterpret_cast<uint32_t *>(&r.u);
        const uint32_t *words = reinterpret_cast<const uint32_t *>(buf + col);
#pragma unroll
        for (int k = 0; k < 4; ++k) u[k] = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int i = k * kWord<T> / 2;
            const int32_t c = col + k * R * kWord<T>;
            if (sure<VEC, R, NV, true>(j, i)) {
                u[k] = words[k * R];
            } else {
                if (i >= pairs) break;
                if (c < D) u[k] = words[k * R];
                if (sizeof(T) == 2 && c + 1 >= D) u[k] &= 0xffffu;
            }
        }
        if (sizeof(T) == 2 && j == 0 && col < 0) u[0] &= 0xffff0000u;
        if (last) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const int32_t c = col + value_of<T, R, true>(i);
                if (c >= 0 && c < D && c > D - VEC) reinterpret_cast<T *>(u)[i] = in[c];
            }
        }
        return r;
    } else {
        return ld<T, VEC>(buf, col);
    }
}

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
// sigmoid(z) and sigmoid(-z).  For bf16 streams, where instructions are what the kernels are short
// of, by e^-z, which ends at 2^127: the reciprocal of that is below fp32's normal range, zero, so that
// gates below -87.3 count as none at all (the other factor, of no use beside a zero, is zero there too).  For
// fp32 by e^-|z|, which neither overflows nor is lost in a 1; __expf leaves it off by some (2 + |z|) u of itself, less
// than 2^-18 of a gate's value wherever that is not below 2^-60 (expf: heads of 128 141 us -> 148, gradients 224 -> 234).
template <typename T, typename E> __device__ __forceinline__ E sigmoid(E z, E &other) {
    if constexpr (sizeof(T) == 2) {
        const E e = each(z, [](float v) {
            float a;
            asm("min.NaN.f32 %0, %1, %2;" : "=f"(a) : "f"(v * -1.44269504f), "f"(127.f));
            return ex2(a);
        });
        const E q = each(e, [](float v) { return rcp(1.f + v); });
        other = mul(e, q);
        return q;
    } else {
        const E t = each(z, [](float v) { return __expf(-fabsf(v)); });
        const E big = each(t, [](float v) { return __fdividef(1.f, 1.f + v); }), small = mul(t, big);
        other = each(z, big, small, [](float v, float b, float s) { return v < 0.f ? b : s; });
        return each(z, big, small, [](float v, float b, float s) { return v < 0.f ? s : b; });
    }
}
// A gate's value, and its slope.
template <typename T, int VEC, int R, int NV, bool RAGGED> __device__ __forceinline__ void open_gate(Vals<VEC> &z, int act, int j, int pairs) {
    if (act == HARTS_GATE_LINEAR) return;
    const bool silu = act == HARTS_GATE_SILU;
#pragma unroll
    for (int i = 0; i < Vals<VEC>::n; ++i) {
        if (!sure<VEC, R, NV, RAGGED>(j, i) && i >= pairs) break;
        typename Vals<VEC>::E rest;
        const auto q = sigmoid<T>(z.e[i], rest);
        z.e[i] = silu ? mul(z.e[i], q) : q;
    }
}
template <typename T, int VEC, int R, int NV, bool RAGGED> __device__ __forceinline__ void open_gate(Vals<VEC> &z, Vals<VEC> &slope, int act, int j, int pairs) {
    const bool silu = act == HARTS_GATE_SILU;
#pragma unroll
    for (int i = 0; i < Vals<VEC>::n; ++i) {
        if (!sure<VEC, R, NV, RAGGED>(j, i) && i >= pairs) break;
        typename Vals<VEC>::E rest;
        const auto q = sigmoid<T>(z.e[i], rest);
        slope.e[i] = mul(q, silu ? fma(z.e[i], rest, all<VEC>(1.f)) : rest);
        z.e[i] = silu ? mul(z.e[i], q) : q;
    }
}

// The R threads of a row, or the warp that several rows share, are a team: it takes its rows, or
// twice as many where they are short, at a time, which lie one behind another in memory, and has them copied ahead into a ring of
// its own, without a look at other teams.
template <int R, int VALUES, bool RAGGED> struct Team {
    static constexpr int threads = R < 32 ? 32 : R, side = threads / R;        // rows side by side
    static constexpr int batch = R <= (RAGGED ? 16 : 32) && VALUES <= 8 ? 2 : 1, rows = side * batch, count = block_of(R) / threads;
};

// Bytes of a team's rows of one tensor in a stage.
template <typename T, bool RAGGED> __host__ __device__ __forceinline__ uint32_t room_of(int rows, int32_t D) {
    return RAGGED ? (static_cast<uint32_t>(rows) * D * sizeof(T) + 30) / 16 * 16 : static_cast<uint32_t>(rows) * D * sizeof(T);
}

// The N tensors' rows on their way, one tensor behind another.  The team's first thread fetches; a
// wait that runs out is reported once and never waited for again, and the block goes on with what
// its shared memory holds, so that its barriers stay matched.
template <typename T, int N, bool ONCE, bool RAGGED> struct Ahead {
    uint8_t *mem;
    uint64_t *full;
    int *fail;
    uint32_t tensor, stage;         // bytes of a stage and of one tensor in it
    int stages, s;
    uint32_t phase;
    // rows from `row` on, whose first value is `first`
    __device__ __forceinline__ void fetch(const void *const (&in)[N], int64_t row, int64_t first, int rows, int64_t C, int64_t whole_end, int32_t D, int slot) {
        if (row >= C) return;
        const uint32_t values = static_cast<uint32_t>(C - row < rows ? C - row : rows) * D;
        uint32_t bytes = values * sizeof(T);
        if (RAGGED) {                                           // from the vector that the first row begins in to the end of the last one's
            constexpr int64_t kMask = 16 / sizeof(T) - 1;
            const int64_t end = min((first + values + kMask) & ~kMask, whole_end);
            first &= ~kMask;
            bytes = static_cast<uint32_t>(end - first) * sizeof(T);
            if (bytes == 0) { tc::mbar_expect_tx(&full[slot], 0); return; }
        }
        uint8_t *dst = mem + slot * stage;
        uint32_t total = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) total += in[i] ? bytes : 0;
        tc::mbar_expect_tx(&full[slot], total);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if (!in[i]) continue;
            if (ONCE) bulk_load_once(dst, static_cast<const T *>(in[i]) + first, bytes, &full[slot]);
            else bulk_load(dst, static_cast<const T *>(in[i]) + first, bytes, &full[slot]);
            dst += tensor;
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

// Weights of a thread's columns: in its registers, from shared memory, or from where they are.
enum Place { kRegs, kShared, kMemory };
template <typename T, int NV, int VEC, int R, int PLACE, bool RAGGED> struct Weights {
    Vals<VEC> kept[PLACE == kRegs ? NV : 1];
    const float *from;
    int32_t width;
    __device__ __forceinline__ void one(const float *w, int32_t col, Vals<VEC> &v) const {
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            const int32_t c = col + value_of<T, R, true>(i);
            reinterpret_cast<float *>(v.e)[i] = c >= 0 && c < width ? __ldg(w + c) : 0.f;
        }
    }
    __device__ __forceinline__ void take(const float *w, float *sh, int t, int into, int32_t D) {
        width = D;
        from = PLACE == kShared ? sh : w;
        if (!w) return;
        if constexpr (PLACE == kRegs) {
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int32_t col = col_of<T, VEC, R, RAGGED>(j, t, into);
                if (RAGGED) one(w, col, kept[j]);
                else if (col < D) ld_w<VEC>(w, col, *reinterpret_cast<float (*)[VEC]>(kept[j].e));
            }
        } else if constexpr (PLACE == kShared) {
            for (int32_t c = threadIdx.x; c < D; c += blockDim.x) sh[c] = w[c];
        }
    }
    __device__ __forceinline__ Vals<VEC> get(int j, int32_t col) const {
        Vals<VEC> v;
        if constexpr (PLACE == kRegs) v = kept[j];
        else if constexpr (RAGGED) one(from, col, v);
        else
#pragma unroll
        for (int i = 0; i < Vals<VEC>::n; i += 2)            // vectors hold four values, or eight
            *reinterpret_cast<float4 *>(&v.e[i]) = *reinterpret_cast<const float4 *>(from + col + 2 * i);
        return v;
    }
};

// Blocks of an SM that registers are shared out for: by the values that a thread keeps.
constexpr int fwd_blocks(int R, int values) { return std::max(1, (values <= 8 ? 768 : 512) / block_of(R)); }
constexpr int bwd_blocks(int R) { return std::max(1, 512 / block_of(R)); }

// What there is beside y: known where it is what surrounds a block, with a gate or without, or a
// head's gated norm, and looked up otherwise.
enum Kind { kAny, kBlock, kHead, kUngated };

template <typename T, int VEC, int R, int NV, int PLACE, int KIND, bool RAGGED>
__global__ void __launch_bounds__(block_of(R), fwd_blocks(R, NV * VEC)) block_norm_fwd_kernel(const Fwd p, int stages) {
    using M = Team<R, NV * VEC, RAGGED>;
    constexpr int kBatch = M::batch, kTeamRows = M::side * kBatch;
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ float sm[2][2][rows_of(R)][R < 32 ? 1 : R / 32];
    __shared__ uint64_t full[M::count][kMaxStages];
    __shared__ int s_fail;
    constexpr bool block = KIND == kBlock || KIND == kUngated;
    const bool post = KIND != kAny || p.w1, gated = KIND == kBlock || KIND == kHead || (KIND == kAny && p.in[1]);
    const bool pre = block || (KIND == kAny && p.w2), added = block || (KIND == kAny && p.in[2]);
    auto there = [&](int i) { return i == 0 || (i == 1 ? gated : added); };
    const int t = threadIdx.x % R, sub = threadIdx.x / R, team = threadIdx.x / M::threads, tt = threadIdx.x % M::threads;
    const int32_t D = p.D;
    const int64_t step = static_cast<int64_t>(gridDim.x) * M::count * kTeamRows;
    int64_t row0 = (static_cast<int64_t>(blockIdx.x) * M::count + team) * kTeamRows;
    int64_t first = row0 * D;                                   // of row0's values
    const int64_t stride = step * D;
    const float inv_d = 1.f / static_cast<float>(D);
    Raw<T, VEC> a[3][NV];
    [[maybe_unused]] Ahead<T, 3, (R > 32), RAGGED> ahead;
    float *sh = reinterpret_cast<float *>(ring);
    int pairs[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) pairs[j] = RAGGED ? pairs_of<T, VEC, R>(j, D) : VEC / 2;
    // values by which the thread's rows begin into a word: the same for all, they are an even number apart
    const int into = RAGGED ? static_cast<int>(row0 + tt / R) & D & (kWord<T> - 1) : 0;
    Weights<T, NV, VEC, R, PLACE, RAGGED> w1, w2;
    w1.take(p.w1, sh, t, into, D);
    w2.take(p.w2, sh + D, t, into, D);
    ahead.tensor = room_of<T, RAGGED>(kTeamRows, D);
    ahead.stage = ahead.tensor * (1 + gated + added);
    ahead.mem = ring + (PLACE == kRegs ? 0 : (2 * D * sizeof(float) + 127) / 128 * 128) + static_cast<size_t>(team) * stages * ahead.stage;
    ahead.full = full[team]; ahead.fail = &s_fail; ahead.stages = stages; ahead.s = 0; ahead.phase = 0;
    if (threadIdx.x == 0) s_fail = 0;
    if (tt == 0) {
        for (int s = 0; s < stages; ++s) tc::mbar_init(&ahead.full[s], 1);
        tc::fence_mbar_init();
        for (int s = 0; s < stages; ++s) ahead.fetch(p.in, row0 + s * step, first + s * stride, kTeamRows, p.C, p.whole_end, D, s);
    }
    __syncthreads();
    for (int slot = 0; row0 < p.C; row0 += step, first += stride) {
        ahead.wait(p.error);
#pragma unroll 1
        for (int batch = 0; batch < kBatch; ++batch, slot ^= 1) {
            const int in_stage = batch * M::side + tt / R;
            const int64_t row = row0 + in_stage;
            const bool on = row < p.C;
            const T *buf = reinterpret_cast<const T *>(ring + (ahead.mem - ring) + ahead.s * ahead.stage) + in_stage * D + (RAGGED ? static_cast<int>(first) & (VEC - 1) : 0);
            const int64_t at = first + in_stage * D;
            const bool last = RAGGED && on && row >= p.whole_rows;
#pragma unroll
            for (int i = 0; i < 3; ++i) {
                if (!there(i)) continue;
#pragma unroll
                for (int j = 0; j < NV; ++j) {
                    const int32_t col = col_of<T, VEC, R, RAGGED>(j, t, into);
                    if (col < D) a[i][j] = take<T, VEC, R, NV, RAGGED>(buf, static_cast<const T *>(p.in[i]) + at, last, j, col, D, pairs[j]);
                }
                buf += ahead.tensor / sizeof(T);
            }
            // behind a sum's barrier, or the warp's own, the stage is free
            auto free_stage = [&] {
                if (tt == 0 && batch == kBatch - 1) ahead.fetch(p.in, row0 + stages * step, first + stages * stride, kTeamRows, p.C, p.whole_end, D, ahead.s);
            };
            if constexpr (R <= 32) {
                __syncwarp();
                free_stage();
            }
            Vals<VEC> v[NV], g[NV];
            Raw<T, VEC> res[NV];
            auto s = all<VEC>(0.f);
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                res[j] = a[2][j];
                if (col_of<T, VEC, R, RAGGED>(j, t, into) >= D) continue;
                open(a[0][j], v[j]);
                if (post) {
#pragma unroll
                    for (int i = 0; i < Vals<VEC>::n; ++i) s = fma(v[j].e[i], v[j].e[i], s);
                }
                if (gated) {
                    open(a[1][j], g[j]);
                    open_gate<T, VEC, R, NV, RAGGED>(g[j], p.act, j, pairs[j]);
                }
            }
            float factor = p.scale;
            if (post) {
                const float r1 = __frsqrt_rn(fmaf(row_sum<R>(total(s), sm[slot][0][sub]), inv_d, p.eps));
                factor *= r1;
                if constexpr (R > 32) free_stage();
                if (t == 0 && p.r1 && on) p.r1[row] = r1;
            }
            s = all<VEC>(0.f);
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int32_t col = col_of<T, VEC, R, RAGGED>(j, t, into);
                if (col >= D) continue;
                if (post) {
                    const Vals<VEC> w = w1.get(j, col);
#pragma unroll
                    for (int i = 0; i < Vals<VEC>::n; ++i) v[j].e[i] = mul(v[j].e[i], w.e[i]);
                }
                if (gated) {
#pragma unroll
                    for (int i = 0; i < Vals<VEC>::n; ++i) v[j].e[i] = mul(v[j].e[i], g[j].e[i]);
                }
                if (added) {
                    Vals<VEC> x;
                    open(res[j], x);
#pragma unroll
                    for (int i = 0; i < Vals<VEC>::n; ++i) v[j].e[i] = fma(v[j].e[i], all<VEC>(factor), x.e[i]);
                } else {
#pragma unroll
                    for (int i = 0; i < Vals<VEC>::n; ++i) v[j].e[i] = mul(v[j].e[i], all<VEC>(factor));
                }
                if (pre) {
#pragma unroll
                    for (int i = 0; i < Vals<VEC>::n; ++i) s = fma(v[j].e[i], v[j].e[i], s);
                }
                if (on) put<T, VEC, R, NV, RAGGED>(p.h, at, j, col, D, pairs[j], v[j]);
            }
            if (pre) {
                const float r2 = __frsqrt_rn(fmaf(row_sum<R>(total(s), sm[slot][1][sub]), inv_d, p.eps));
                if (!post) {
                    if constexpr (R > 32) free_stage();
                }
                if (t == 0 && p.r2 && on) p.r2[row] = r2;
#pragma unroll
                for (int j = 0; j < NV; ++j) {
                    const int32_t col = col_of<T, VEC, R, RAGGED>(j, t, into);
                    if (col >= D) continue;
                    const Vals<VEC> w = w2.get(j, col);
#pragma unroll
                    for (int i = 0; i < Vals<VEC>::n; ++i) v[j].e[i] = mul(mul(v[j].e[i], all<VEC>(r2)), w.e[i]);
                    if (on) put<T, VEC, R, NV, RAGGED>(p.n, at, j, col, D, pairs[j], v[j]);
                }
            }
        }
        ahead.next();
    }
    if (tt == 0) ahead.drain();
}

template <typename T, int VEC, int R, int NV, int PLACE, int KIND, bool RAGGED>
__global__ void __launch_bounds__(block_of(R), bwd_blocks(R)) block_norm_bwd_kernel(const Bwd p, int stages) {
    using M = Team<R, NV * VEC, RAGGED>;
    constexpr int kRows = rows_of(R);
    constexpr int kBatch = M::batch, kTeamRows = M::side * kBatch;
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ float sm[2][2][kRows][R < 32 ? 1 : R / 32];
    __shared__ uint64_t full[M::count][kMaxStages];
    __shared__ int s_fail;
    constexpr bool block = KIND == kBlock || KIND == kUngated;
    const bool post = KIND != kAny || p.w1, gated = KIND == kBlock || KIND == kHead || (KIND == kAny && p.in[1]);
    const bool pre = block || (KIND == kAny && p.w2), along = KIND != kAny || p.in[4];
    auto there = [&](int i) { return i == 0 || (i == 1 ? gated : i == 4 ? along : pre); };
    const int t = threadIdx.x % R, sub = threadIdx.x / R, team = threadIdx.x / M::threads, tt = threadIdx.x % M::threads;
    const int32_t D = p.D;
    const int64_t step = static_cast<int64_t>(gridDim.x) * M::count * kTeamRows;
    int64_t row0 = (static_cast<int64_t>(blockIdx.x) * M::count + team) * kTeamRows;
    int64_t first = row0 * D;                                   // of row0's values
    const int64_t stride = step * D;
    const float inv_d = 1.f / static_cast<float>(D);
    let_next_start();
    Raw<T, VEC> a[5][NV];
    [[maybe_unused]] Ahead<T, 5, false, RAGGED> ahead;
    float *sh = reinterpret_cast<float *>(ring);
    int pairs[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) pairs[j] = RAGGED ? pairs_of<T, VEC, R>(j, D) : VEC / 2;
    // values by which the thread's rows begin into a word: the same for all, they are an even number apart
    const int into = RAGGED ? static_cast<int>(row0 + tt / R) & D & (kWord<T> - 1) : 0;
    Weights<T, NV, VEC, R, PLACE, RAGGED> w1, w2;
    w1.take(p.w1, sh, t, into, D);
    w2.take(p.w2, sh + D, t, into, D);
    // the weights' gradients of a thread's columns: registers, but shared memory where 64 of them
    // are all that a thread has (then the weights stay where they are)
    constexpr bool kSums = PLACE == kMemory;
    Vals<VEC> dw1[kSums ? 1 : NV], dw2[kSums ? 1 : NV];
#pragma unroll
    for (int j = 0; j < (kSums ? 1 : NV); ++j) {
#pragma unroll
        for (int i = 0; i < Vals<VEC>::n; ++i) dw1[j].e[i] = dw2[j].e[i] = all<VEC>(0.f);
    }
    if constexpr (kSums)
        for (int32_t c = threadIdx.x; c < 2 * D; c += blockDim.x) sh[c] = 0.f;
    auto add_dw = [&](Vals<VEC> *dw, int which, int j, int32_t col, const Vals<VEC> &a, const Vals<VEC> &b) {
        if constexpr (kSums) {
            float *at = sh + which * D + col;
#pragma unroll
            for (int i = 0; i < Vals<VEC>::n; ++i) {
                if constexpr (RAGGED) {
                    const int32_t c = value_of<T, R, true>(2 * i), d = value_of<T, R, true>(2 * i + 1);
                    if (col + c >= 0 && col + c < D) at[c] = fmaf(a.e[i].x, b.e[i].x, at[c]);
                    if (col + d < D) at[d] = fmaf(a.e[i].y, b.e[i].y, at[d]);
                } else {
                    Two *pair = reinterpret_cast<Two *>(at) + i;
                    *pair = fma(a.e[i], b.e[i], *pair);
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < Vals<VEC>::n; ++i) dw[j].e[i] = fma(a.e[i], b.e[i], dw[j].e[i]);
        }
    };
    float next1 = 0.f, next2 = 0.f;
    auto load_roots = [&](int64_t r) {
        if (r >= p.C) return;
        if (post) next1 = __ldg(p.r1 + r);
        if (pre) next2 = __ldg(p.r2 + r);
    };
    ahead.tensor = room_of<T, RAGGED>(kTeamRows, D);
    ahead.stage = ahead.tensor * (1 + gated + 2 * pre + along);
    ahead.mem = ring + (PLACE == kRegs ? 0 : (2 * D * sizeof(float) + 127) / 128 * 128) + static_cast<size_t>(team) * stages * ahead.stage;
    ahead.full = full[team]; ahead.fail = &s_fail; ahead.stages = stages; ahead.s = 0; ahead.phase = 0;
    if (threadIdx.x == 0) s_fail = 0;
    if (tt == 0) {
        for (int s = 0; s < stages; ++s) tc::mbar_init(&ahead.full[s], 1);
        tc::fence_mbar_init();
        for (int s = 0; s < stages; ++s) ahead.fetch(p.in, row0 + s * step, first + s * stride, kTeamRows, p.C, p.whole_end, D, s);
    }
    load_roots(row0 + tt / R);
    __syncthreads();
    for (int slot = 0; row0 < p.C; row0 += step, first += stride) {
        ahead.wait(p.error);
#pragma unroll 1
        for (int batch = 0; batch < kBatch; ++batch, slot ^= 1) {
            const int in_stage = batch * M::side + tt / R;
            const int64_t row = row0 + in_stage;
            const bool on = row < p.C;
            const float r1 = next1, r2 = next2;
            load_roots(batch < kBatch - 1 ? row + M::side : row0 + step + tt / R);
            const T *buf = reinterpret_cast<const T *>(ring + (ahead.mem - ring) + ahead.s * ahead.stage) + in_stage * D + (RAGGED ? static_cast<int>(first) & (VEC - 1) : 0);
            const int64_t at = first + in_stage * D;
            const bool last = RAGGED && on && row >= p.whole_rows;
#pragma unroll
            for (int i = 0; i < 5; ++i) {
                if (!there(i)) continue;
#pragma unroll
                for (int j = 0; j < NV; ++j) {
                    const int32_t col = col_of<T, VEC, R, RAGGED>(j, t, into);
                    if (col < D) a[i][j] = take<T, VEC, R, NV, RAGGED>(buf, static_cast<const T *>(p.in[i]) + at, last, j, col, D, pairs[j]);
                }
                buf += ahead.tensor / sizeof(T);
            }
            auto free_stage = [&] {
                if (tt == 0 && batch == kBatch - 1) ahead.fetch(p.in, row0 + stages * step, first + stages * stride, kTeamRows, p.C, p.whole_end, D, ahead.s);
            };
            if constexpr (R <= 32) {
                __syncwarp();
                free_stage();
                if (!on) continue;                              // rows of a warp do not wait for each other from here on
            }
            Raw<T, VEC> y[NV], g[NV];
            Vals<VEC> d[NV], n[NV], f[NV];
            auto s = all<VEC>(0.f);
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                y[j] = a[0][j];
                g[j] = a[1][j];
                const int32_t col = col_of<T, VEC, R, RAGGED>(j, t, into);
                if (col >= D) continue;
                if (along) {
                    open(a[4][j], d[j]);
                } else {
#pragma unroll
                    for (int i = 0; i < Vals<VEC>::n; ++i) d[j].e[i] = all<VEC>(0.f);
                }
                if (pre) {
                    const Vals<VEC> w = w2.get(j, col);
                    open(a[2][j], f[j]);
                    open(a[3][j], n[j]);
#pragma unroll
                    for (int i = 0; i < Vals<VEC>::n; ++i) n[j].e[i] = mul(n[j].e[i], all<VEC>(r2));
                    add_dw(dw2, 1, j, col, f[j], n[j]);
#pragma unroll
                    for (int i = 0; i < Vals<VEC>::n; ++i) {
                        f[j].e[i] = mul(f[j].e[i], w.e[i]);
                        s = fma(f[j].e[i], n[j].e[i], s);
                    }
                }
            }
            if (pre) {
                const float m = row_sum<R>(total(s), sm[slot][0][sub]) * inv_d * -r2;
                if constexpr (R > 32) free_stage();
#pragma unroll
                for (int j = 0; j < NV; ++j) {
#pragma unroll
                    for (int i = 0; i < Vals<VEC>::n; ++i)
                        d[j].e[i] = fma(all<VEC>(r2), f[j].e[i], fma(n[j].e[i], all<VEC>(m), d[j].e[i]));
                }
            }
            s = all<VEC>(0.f);
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int32_t col = col_of<T, VEC, R, RAGGED>(j, t, into);
                if (col >= D) continue;
                if (p.dres && on) put<T, VEC, R, NV, RAGGED>(p.dres, at, j, col, D, pairs[j], d[j]);
                Vals<VEC> w;
                if (post) w = w1.get(j, col);
                open(y[j], n[j]);
#pragma unroll
                for (int i = 0; i < Vals<VEC>::n; ++i) {
                    d[j].e[i] = mul(d[j].e[i], all<VEC>(p.scale));
                    if (post) n[j].e[i] = mul(n[j].e[i], all<VEC>(r1));
                }
                if (gated) {
                    Vals<VEC> z, out;
                    open(g[j], z);
#pragma unroll
                    for (int i = 0; i < Vals<VEC>::n; ++i) {
                        out.e[i] = mul(d[j].e[i], n[j].e[i]);
                        if (post) out.e[i] = mul(out.e[i], w.e[i]);
                    }
                    if (p.act != HARTS_GATE_LINEAR) {
                        Vals<VEC> slope;
                        open_gate<T, VEC, R, NV, RAGGED>(z, slope, p.act, j, pairs[j]);
#pragma unroll
                        for (int i = 0; i < Vals<VEC>::n; ++i) out.e[i] = mul(out.e[i], slope.e[i]);
                    }
#pragma unroll
                    for (int i = 0; i < Vals<VEC>::n; ++i) d[j].e[i] = mul(d[j].e[i], z.e[i]);
                    if (p.dgate && on) put<T, VEC, R, NV, RAGGED>(p.dgate, at, j, col, D, pairs[j], out);
                }
                if (post) {
                    add_dw(dw1, 0, j, col, d[j], n[j]);
#pragma unroll
                    for (int i = 0; i < Vals<VEC>::n; ++i) {
                        d[j].e[i] = mul(d[j].e[i], w.e[i]);
                        s = fma(d[j].e[i], n[j].e[i], s);
                    }
                }
            }
            float m = 0.f;
            if (post) {
                m = -row_sum<R>(total(s), sm[slot][1][sub]) * inv_d;
                if (!pre) {
                    if constexpr (R > 32) free_stage();
                }
            }
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int32_t col = col_of<T, VEC, R, RAGGED>(j, t, into);
                if (col >= D) continue;
                if (post) {
#pragma unroll
                    for (int i = 0; i < Vals<VEC>::n; ++i) d[j].e[i] = mul(all<VEC>(r1), fma(n[j].e[i], all<VEC>(m), d[j].e[i]));
                }
                if (on) put<T, VEC, R, NV, RAGGED>(p.dy, at, j, col, D, pairs[j], d[j]);
            }
        }
        ahead.next();
    }
    if (tt == 0) ahead.drain();
    // the rows of a block leave one sum of either weight, added in ascending order
    __shared__ float all[kRows > 1 ? kRows : 1][kRows > 1 ? R * NV * VEC : 1];
    for (int which = 0; which < 2; ++which) {
        if (!(which ? pre : post)) continue;
        float *part = p.part + blockIdx.x * (2 * static_cast<int64_t>(D)) + which * D;
        if constexpr (kRows > 1) __syncthreads();
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int32_t col = col_of<T, VEC, R, RAGGED>(j, t, into);
            if (col >= D) continue;
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const int32_t at = col + value_of<T, R, RAGGED>(i);
                if (RAGGED && (at < 0 || at >= D)) continue;
                const float v = kSums ? sh[which * D + at] : reinterpret_cast<const float *>(which ? dw2[kSums ? 0 : j].e : dw1[kSums ? 0 : j].e)[i];
                if constexpr (kRows > 1) all[sub][at] = v;
                else part[at] = v;
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

// Threads of a row and values that each of them keeps.  The backward's rows above 4,096 channels have 16 values
// a thread, their sums in shared memory and the weights where they are.  Where shared memory holds them (launch_rows),
// two stages are on their way: with everything up to 7,314 channels in bf16 and 4,266 in fp32, without a gate up to
// 8,192 in bf16; wider rows have one, and more of L1 for the weights.  (bf16, 16,384 x 8,192 with everything: one stage 443
// us, two by leaving L1 no room 491, 1,024 threads with eight values, 64 registers each, 655.  fp32, 8,192 x
// 8,192, one stage: 471 - 497.  Two stages, bf16: 24,576 x 5,120 507, 20,000 x 6,144 459.)
struct Shape { int vec, r, values; bool ragged; };
Shape shape_of(int32_t dtype, int32_t D, bool backward) {
    const int full = dtype == HARTS_BF16 ? 8 : 4;
    Shape s{full, 8, 8, D % full != 0};
    if (s.ragged && full == 8) ++D;                      // a row's words, where it begins in the middle of one
    while (s.r < 16 && s.r * 8 < D) s.r *= 2;
    if (s.r * 8 < D && !backward) s.values = 16;
    if (D > 4096) s.values = 16;
    while (s.r * s.values < D) s.r *= 2;
    return s;
}

template <typename P> void set_whole(P &p, int32_t dtype) {
    const int vec = dtype == HARTS_BF16 ? 8 : 4;
    p.whole_end = p.C * p.D / vec * vec;
    p.whole_rows = p.whole_end / p.D;
}

// Most blocks that are resident at a time, whatever the kernel's registers.
int64_t blocks_of(const Shape &s, int64_t C) {
    return std::min<int64_t>((C + rows_of(s.r) - 1) / rows_of(s.r), int64_t(sm_count()) * (2048 / block_of(s.r)));
}

// Resident blocks of a persistent kernel, and the rows that each of them has on its way: `budget`
// bytes an SM.
template <typename T, int R, int VT, int PLACE, bool RAGGED, typename K, typename P>
cudaError_t launch_rows(K *kernel, const P &p, int tensors, size_t most, std::atomic<uint64_t> &allowed, std::atomic<int> &regs_fit, int64_t *groups, cudaStream_t st) {
    constexpr size_t kSmem = size_t(200) * 1024;
    using M = Team<R, VT, RAGGED>;
    int stages = 1, n = regs_fit.load(std::memory_order_relaxed);
    if (n == 0) {                                        // blocks that registers leave room for
        if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, block_of(R), 0) != cudaSuccess || n < 1) n = 1;
        regs_fit.store(n, std::memory_order_relaxed);
    }
    size_t smem = 0;
    const size_t weights = PLACE == kRegs ? 0 : (2 * size_t(p.D) * sizeof(float) + 127) / 128 * 128;
    const size_t stage = size_t(room_of<T, RAGGED>(M::rows, p.D)) * tensors * M::count;
    while (n > 1 && n * (weights + 2 * stage) > kSmem) --n;
    stages = static_cast<int>(std::min<size_t>(most, std::max<size_t>(1, (kSmem / n - std::min(weights, kSmem / n)) / stage)));
    smem = weights + stages * stage;
    const cudaError_t e = allow_smem(kernel, R >= 512 ? 226 * 1024 : kSmem, allowed);     // one stage of 8,192 fp32 values and sums: 224 KB
    if (e != cudaSuccess) return e;
    // an even number of blocks, so that a thread's rows are an even number apart
    const int64_t rows = rows_of(R), grid = std::min<int64_t>((p.C + rows - 1) / rows, std::max(int64_t(sm_count()) * n / 2 * 2, int64_t(1)));
    *groups = grid;
    return launch(kernel, grid, block_of(R), smem, 1, false, st, p, stages);
}

template <typename T, int VEC, int R, int VT, int KIND, bool RAGGED>
cudaError_t launch_kind(const Fwd &p, int tensors, int64_t *groups, cudaStream_t st) {
    static std::atomic<uint64_t> allowed{0};
    static std::atomic<int> fit{0};
    return launch_rows<T, R, VT, kRegs, RAGGED>(block_norm_fwd_kernel<T, VEC, R, VT / VEC, kRegs, KIND, RAGGED>, p, tensors, R <= 32 && VT > 8 ? 1 : kMaxStages, allowed, fit, groups, st);
}
template <typename T, int VEC, int R, int VT, int KIND, bool RAGGED>
cudaError_t launch_kind(const Bwd &p, int tensors, int64_t *groups, cudaStream_t st) {
    static std::atomic<uint64_t> allowed{0};
    static std::atomic<int> fit{0};
    constexpr int place = VT > 8 ? kMemory : RAGGED ? kRegs : kShared;
    return launch_rows<T, R, VT, place, RAGGED>(block_norm_bwd_kernel<T, VEC, R, VT / VEC, place, KIND, RAGGED>, p, tensors, kMaxStages, allowed, fit, groups, st);
}
Kind kind_of(const Fwd &p) {
    if (!p.w1 || (p.w2 == nullptr) != (p.in[2] == nullptr)) return kAny;
    return p.w2 ? (p.in[1] ? kBlock : kUngated) : p.in[1] ? kHead : kAny;
}
Kind kind_of(const Bwd &p) {
    if (!p.w1 || !p.in[4]) return kAny;
    return p.w2 ? (p.in[1] ? kBlock : kUngated) : p.in[1] ? kHead : kAny;
}
template <typename T, int VEC, int R, int VT, typename P>
cudaError_t launch_one(const P &p, bool ragged, int tensors, int64_t *groups, cudaStream_t st) {
    const Kind k = kind_of(p);
    if (k == kBlock) return ragged ? launch_kind<T, VEC, R, VT, kBlock, true>(p, tensors, groups, st) : launch_kind<T, VEC, R, VT, kBlock, false>(p, tensors, groups, st);
    if (k == kHead) return ragged ? launch_kind<T, VEC, R, VT, kHead, true>(p, tensors, groups, st) : launch_kind<T, VEC, R, VT, kHead, false>(p, tensors, groups, st);
    if (k == kUngated) return ragged ? launch_kind<T, VEC, R, VT, kUngated, true>(p, tensors, groups, st) : launch_kind<T, VEC, R, VT, kUngated, false>(p, tensors, groups, st);
    return ragged ? launch_kind<T, VEC, R, VT, kAny, true>(p, tensors, groups, st) : launch_kind<T, VEC, R, VT, kAny, false>(p, tensors, groups, st);
}

// The instances that shape_of names.
#define HARTS_CASE(V, R, VT) if (s.vec == V && s.r == R && s.values == VT) return launch_one<T, V, R, VT>(p, s.ragged, tensors, groups, st);
template <typename T, int VEC> cudaError_t run(const Shape &s, const Fwd &p, int tensors, int64_t *groups, cudaStream_t st) {
    HARTS_CASE(VEC, 8, 8) HARTS_CASE(VEC, 16, 8) HARTS_CASE(VEC, 16, 16) HARTS_CASE(VEC, 32, 16) HARTS_CASE(VEC, 64, 16)
    HARTS_CASE(VEC, 128, 16) HARTS_CASE(VEC, 256, 16) HARTS_CASE(VEC, 512, 16)
    return cudaErrorInvalidValue;
}
template <typename T, int VEC> cudaError_t run(const Shape &s, const Bwd &p, int tensors, int64_t *groups, cudaStream_t st) {
    HARTS_CASE(VEC, 8, 8) HARTS_CASE(VEC, 16, 8) HARTS_CASE(VEC, 32, 8) HARTS_CASE(VEC, 64, 8)
    HARTS_CASE(VEC, 128, 8) HARTS_CASE(VEC, 256, 8) HARTS_CASE(VEC, 512, 8) HARTS_CASE(VEC, 512, 16)
    return cudaErrorInvalidValue;
}
#undef HARTS_CASE

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
    set_whole(p, a->dtype);
    p.error = a->error ? a->error : own_error_word();
    if (!p.error) { set_error("the library's error word is not to be had"); return HARTS_ECUDA; }
    int64_t groups = 0;
    const int tensors = 1 + (a->gate != nullptr) + (a->residual != nullptr);
    const Shape s = shape_of(a->dtype, a->D, false);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = a->dtype == HARTS_BF16 ? run<__nv_bfloat16, 8>(s, p, tensors, &groups, st) : run<float, 4>(s, p, tensors, &groups, st);
    if (e != cudaSuccess) return cuda_fail(e, "block norm forward launch");
    set_error("");
    return HARTS_OK;
}

size_t harts_block_norm_bwd_workspace_bytes(int64_t C, int32_t D, int32_t dtype) {
    if (C < 0 || D < 1 || D > kMaxDim || (dtype != HARTS_FP32 && dtype != HARTS_BF16)) return 0;
    return std::max<size_t>(256, 2 * sizeof(float) * static_cast<size_t>(blocks_of(shape_of(dtype, D, true), C)) * D);
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
    set_whole(p, a->dtype);
    p.error = a->error ? a->error : own_error_word();
    if (!p.error) { set_error("the library's error word is not to be had"); return HARTS_ECUDA; }
    int tensors = 0;
    for (const void *q : p.in) tensors += q != nullptr;
    int64_t groups = 0;
    const Shape s = shape_of(a->dtype, a->D, true);
    cudaError_t e = a->dtype == HARTS_BF16 ? run<__nv_bfloat16, 8>(s, p, tensors, &groups, st) : run<float, 4>(s, p, tensors, &groups, st);
    if (e != cudaSuccess) return cuda_fail(e, "block norm backward launch");
    const Dw d{p.part, a->post_weight ? b->dpost_weight : nullptr, a->pre_weight ? b->dpre_weight : nullptr, a->D, static_cast<int32_t>(groups)};
    e = launch(block_norm_dw_kernel, 2 * ((a->D + 31) / 32), 1024, 0, 1, true, st, d);
    if (e != cudaSuccess) return cuda_fail(e, "block norm backward launch");
    set_error("");
    return HARTS_OK;
}

}  // extern "C"
