// tcgen05.cuh -- fifth-generation tensor core wrappers: tensor memory, operand
// descriptors and the products used by the prompt attention kernel.
#pragma once

#include "qasa_device.cuh"

namespace qasa {

__device__ __forceinline__ void tmem_alloc(uint32_t *dst, uint32_t columns) {   // a whole warp
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst)), "r"(columns)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t columns) {    // the same warp
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(columns) : "memory");
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// Shared memory written by ordinary stores, made visible to the tensor core.
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// `bar` is arrived on when every product issued so far by this thread is complete.
__device__ __forceinline__ void tc_commit(uint64_t *bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
                 : "memory");
}

// Instruction descriptor of kind::f16: fp32 accumulator, A and B both f16 or
// both bf16, A K-major, B K-major or N-major, M x N.
template <typename T>
constexpr uint32_t f16_idesc(int m, int n, bool b_n_major) {
    const uint32_t type = elem<T>::id == QASA_DTYPE_BF16 ? 1u : 0u;
    return (1u << 4) | (type << 7) | (type << 10) | ((b_n_major ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) |
           ((uint32_t)(m >> 4) << 24);
}

// Operand descriptor of a tile in 128-byte-swizzled shared memory: rows of 128
// bytes, groups of 8 rows `sbo` bytes apart; N-major operands wider than one row
// have their 64-element blocks `lbo` bytes apart.
__device__ __forceinline__ uint64_t swz128_desc(uint32_t addr, uint32_t lbo, uint32_t sbo) {
    return (uint64_t)((addr >> 4) & 0x3fffu) | ((uint64_t)((lbo >> 4) & 0x3fffu) << 16) |
           ((uint64_t)((sbo >> 4) & 0x3fffu) << 32) | (1ull << 46) | (2ull << 61);
}

// D[tmem] (+)= A[smem] B[smem], one k-step of 16.
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t add) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc),
                 "r"(add)
                 : "memory");
}
// D[tmem] (+)= A[tmem] B[smem].
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t add) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a), "l"(b), "r"(idesc),
                 "r"(add)
                 : "memory");
}

#define QASA_R8(o, i) o(r[i]), o(r[i + 1]), o(r[i + 2]), o(r[i + 3]), o(r[i + 4]), o(r[i + 5]), o(r[i + 6]), o(r[i + 7])
#define QASA_OUT(x) "=r"(x)
#define QASA_IN(x) "r"(x)

// 32 consecutive columns of this warp's 32 lanes: a lane's row, one register per column.
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t *r) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 "
                 "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
                 "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
                 : QASA_R8(QASA_OUT, 0), QASA_R8(QASA_OUT, 8), QASA_R8(QASA_OUT, 16), QASA_R8(QASA_OUT, 24)
                 : "r"(addr));
}
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t *r) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
                 "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
                 "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(addr),
                 QASA_R8(QASA_IN, 0), QASA_R8(QASA_IN, 8), QASA_R8(QASA_IN, 16), QASA_R8(QASA_IN, 24)
                 : "memory");
}

__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t *r) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 "
                 "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
                 : QASA_R8(QASA_OUT, 0), QASA_R8(QASA_OUT, 8) : "r"(addr));
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t *r) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
                 "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(addr),
                 QASA_R8(QASA_IN, 0), QASA_R8(QASA_IN, 8)
                 : "memory");
}

// Waits for the loads of 32 (16) registers, whose uses cannot move before it.
#define QASA_INOUT(x) "+r"(x)
__device__ __forceinline__ void tmem_wait_ld16(uint32_t *r) {
    asm volatile("tcgen05.wait::ld.sync.aligned;" : QASA_R8(QASA_INOUT, 0), QASA_R8(QASA_INOUT, 8) :: "memory");
}
__device__ __forceinline__ void tmem_wait_ld32(uint32_t *r) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : QASA_R8(QASA_INOUT, 0), QASA_R8(QASA_INOUT, 8), QASA_R8(QASA_INOUT, 16), QASA_R8(QASA_INOUT, 24)
                 :: "memory");
}
#undef QASA_INOUT

#undef QASA_R8
#undef QASA_OUT
#undef QASA_IN

}  // namespace qasa
