// What a persistent tile kernel of one block or of a pair of blocks is made of: bounded waits of its
// roles, copies and products whose barriers lie in the pair's leader, and rows of an output tile on
// their way out.
#pragma once
#include <cuda.h>

#include <cstdint>

#include "tc_primitives.cuh"

namespace harts {
namespace pairs {

__device__ __forceinline__ void arrive(uint64_t *bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" :: "r"(tc::smem_addr(bar)) : "memory");
}

__device__ __forceinline__ void store_3d(const void *map, int x, int y, int z, const void *src, bool add) {
    if (add)
        asm volatile("cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.tile.bulk_group [%0, {%1, %2, %3}], [%4];"
                     :: "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(tc::smem_addr(src)) : "memory");
    else
        asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];"
                     :: "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(tc::smem_addr(src)) : "memory");
}

// all but the last committed store of this thread have read their source
__device__ __forceinline__ void store_wait_read1() { asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory"); }

__device__ __forceinline__ bool failed(const int *f) { return *reinterpret_cast<const volatile int *>(f) != 0; }
// True once the phase completed; false, with the block marked, when the wait ran out or
// another role gave up.
__device__ __forceinline__ bool wait_or_fail(uint64_t *bar, uint32_t phase, int *f) {
    if (tc::mbar_try(bar, phase)) return true;
    if (failed(f)) return false;
    if (tc::mbar_wait(bar, phase)) return true;
    atomicExch(f, 1);
    return false;
}

// The same for a whole warp.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t phase, int *f) {
    return __all_sync(0xffffffffu, wait_or_fail(bar, phase, f)) != 0;
}

// ---- pairs of blocks: the leader (rank 0) issues the products of both, 256 tile rows ----

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// address of a barrier of this block in the pair's leader
__device__ __forceinline__ uint32_t leader_addr(const uint64_t *bar) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(a) : "r"(tc::smem_addr(bar)));
    return a;
}
template <int G> __device__ __forceinline__ void pair_alloc(uint32_t *dst) {
    if constexpr (G == 1) {
        tc::tmem_alloc(dst, 512);
    } else {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" :: "r"(tc::smem_addr(dst)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
}
template <int G> __device__ __forceinline__ void pair_dealloc(uint32_t t) {
    if constexpr (G == 1) tc::tmem_dealloc(t, 512);
    else asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" :: "r"(t) : "memory");
}
// One lane of the warp.
__device__ __forceinline__ uint32_t elect_lane() {
    uint32_t on;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(on));
    return on;
}
// The whole warp comes through these two, with the same operands in every lane (which the
// compiler then keeps in uniform registers, where the instruction wants them); the lane with
// `on` set issues.
template <int G> __device__ __forceinline__ void pair_mma(uint32_t on, uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t acc) {
    if constexpr (G == 1)
        asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
                     "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
                     :: "r"(d), "l"(a), "l"(b), "r"(id), "r"(acc), "r"(on) : "memory");
    else
        asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
                     "@q tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}"
                     :: "r"(d), "l"(a), "l"(b), "r"(id), "r"(acc), "r"(on) : "memory");
}
// Arrive, in every block of the pair, on the barrier at this offset once all products issued
// so far are done.
template <int G> __device__ __forceinline__ void pair_commit(uint32_t on, uint64_t *bar) {
    if constexpr (G == 1)
        asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
                     "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}"
                     :: "r"(tc::smem_addr(bar)), "r"(on) : "memory");
    else
        asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\t"
                     "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}"
                     :: "r"(tc::smem_addr(bar)), "h"(static_cast<uint16_t>(3)), "r"(on) : "memory");
}
// Copies into this block, issued by the lane with `on` set; the bytes count on `bar`, which in
// a pair lies in the leader.
template <int G> __device__ __forceinline__ void pair_load(uint32_t on, uint32_t dst, const void *map, int x, int y, uint32_t bar) {
    if constexpr (G == 1)
        asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %5, 0;\n\t"
                     "@q cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
                     " [%0], [%1, {%2, %3}], [%4];\n\t}"
                     :: "r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar), "r"(on) : "memory");
    else
        asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %5, 0;\n\t"
                     "@q cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
                     " [%0], [%1, {%2, %3}], [%4];\n\t}"
                     :: "r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar), "r"(on) : "memory");
}
__device__ __forceinline__ void prefetch_map(const CUtensorMap *map) {
    asm volatile("prefetch.tensormap [%0];" :: "l"(reinterpret_cast<uint64_t>(map)) : "memory");
}
template <int G>
__device__ __forceinline__ void pair_load3(uint32_t on, uint32_t dst, const void *map, int x, int y, int z, uint32_t bar) {
    if constexpr (G == 1)
        asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %6, 0;\n\t"
                     "@q cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
                     " [%0], [%1, {%2, %3, %4}], [%5];\n\t}"
                     :: "r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar), "r"(on)
                     : "memory");
    else
        asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %6, 0;\n\t"
                     "@q cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
                     " [%0], [%1, {%2, %3, %4}], [%5];\n\t}"
                     :: "r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar), "r"(on)
                     : "memory");
}
// The bytes that a phase of this block's barrier waits for, counted once.
__device__ __forceinline__ void expect(uint32_t on, uint32_t bar, uint32_t bytes) {
    asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\t"
                 "@q mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n\t}" :: "r"(bar), "r"(bytes), "r"(on) : "memory");
}
__device__ __forceinline__ void arrive_at(uint32_t cluster_addr) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" :: "r"(cluster_addr) : "memory");
}

// 64 values of one row of a 128-byte-swizzled tile, in bf16.
__device__ __forceinline__ void store_row(uint8_t *tile, int row, const float (&v)[64]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        uint4 w;
        w.x = tc::pack_bf16(v[8 * j], v[8 * j + 1]); w.y = tc::pack_bf16(v[8 * j + 2], v[8 * j + 3]);
        w.z = tc::pack_bf16(v[8 * j + 4], v[8 * j + 5]); w.w = tc::pack_bf16(v[8 * j + 6], v[8 * j + 7]);
        *reinterpret_cast<uint4 *>(tile + row * 128 + ((j ^ (row & 7)) << 4)) = w;
    }
}

}  // namespace pairs
}  // namespace harts
