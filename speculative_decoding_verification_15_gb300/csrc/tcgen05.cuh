// tcgen05.cuh -- fifth-generation tensor-core building blocks (sm_103a): tensor memory,
// fp8 products of shared-memory operands, tiled copies.
//
// Operand layouts used here (8-bit elements, a tile row of 128 bytes, shared-memory
// tiles 1024-byte aligned, 128-byte swizzle: 16-byte chunk c of row r lies at chunk
// c ^ (r & 7)):
//  - rows are M or N and the 128 bytes run along K ("K-major"): 8-row groups 1024 bytes
//    apart; a 32-element step along K is 32 bytes further into the swizzled row;
//  - rows are K and the 128 bytes run along M ("M-major", the transposed operand): 8-row
//    groups 1024 bytes apart; a step of 32 along K is 4096 bytes further.
// And one without swizzle for N-major B: blocks of 16 columns, in each the K rows 16
// bytes apart, so 8-row groups 128 bytes apart and blocks 16 * rows bytes apart.
#pragma once

#include <cuda.h>
#include <stdint.h>

#include "spec_common.cuh"

namespace specv {

// ------------------------------------------------------------------ tensor memory
// One warp allocates (a power of two of 32 .. 512 columns) and the same warp frees.
__device__ __forceinline__ void tmem_alloc(uint32_t *slot, uint32_t cols) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(slot)), "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}
__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t cols) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols));
}

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// Shared memory written by ordinary stores, before an arrive that lets the tensor
// cores or a bulk copy use it.
__device__ __forceinline__ void fence_async_shared() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// 16 consecutive columns of this warp's 32 lanes (a lane a thread) into registers.
__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t *r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(addr));
}
template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t addr, uint32_t (&r)[N]) {
    static_assert(N % 16 == 0, "columns come 16 at a time");
#pragma unroll
    for (int i = 0; i < N; i += 16) tmem_ld16(addr + i, r + i);
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// ------------------------------------------------------------------ descriptors
// Shared-memory operand: address, leading and stride byte offsets (16-byte units),
// version 1, swizzle mode (0 none, 2 128 bytes).
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lead, uint32_t stride, uint32_t swizzle) {
    return (uint64_t)((addr >> 4) & 0x3fff) | ((uint64_t)(lead >> 4) << 16) | ((uint64_t)(stride >> 4) << 32) |
           (1ull << 46) | ((uint64_t)swizzle << 61);
}
// e4m3 x e4m3 into fp32, M = 128; transposed operands as said.
__host__ __device__ constexpr uint32_t fp8_idesc(int n, bool a_transposed, bool b_transposed) {
    return (1u << 4) | ((a_transposed ? 1u : 0u) << 15) | ((b_transposed ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) |
           (8u << 24);
}

// True in one lane of a converged warp.  The instructions that one thread issues for the
// warp (products, commits, tiled copies) take their operands from uniform registers: a
// branch on elect.sync, inside code that the whole warp runs with the same values, tells
// the compiler so; a branch on the lane's number costs a loop over the lanes around each
// (130 cycles a product instead of 50).
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(p));
    return p != 0;
}

// D (+)= A B, issued by one thread.
__device__ __forceinline__ void mma_fp8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate ? 1u : 0u)
        : "memory");
}
// The barrier completes a phase's arrival when every product issued so far is done.
__device__ __forceinline__ void mma_commit(uint64_t *bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar))
                 : "memory");
}

// ------------------------------------------------------------------ tiled copies
__device__ __forceinline__ void tma_load_4d(void *dst, const CUtensorMap *map, int x0, int x1, int x2, int x3,
                                            uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
        "[%6];" ::"r"(smem_addr(dst)),
        "l"(map), "r"(x0), "r"(x1), "r"(x2), "r"(x3), "r"(smem_addr(bar))
        : "memory");
}

}  // namespace specv
