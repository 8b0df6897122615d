// The 5th-generation matrix unit (tcgen05) as the latent attention uses it:
// descriptors, issue, completion and tensor-memory access.
#pragma once

#include "kva_common.cuh"

namespace kvw {

// Shared-memory operand in 128-byte-swizzled lines, 8 lines to a 1024-byte
// group.  K-major: a line holds 64 contraction elements of one row and groups
// of 8 rows lie 1024 bytes apart (lead is not used).  MN-major: a line holds
// 64 rows' elements of one contraction index, groups of 8 indices lie 1024
// bytes apart, and the next 64 rows `lead` bytes away.  The descriptor's low
// word; the high one is the same for all.  An operand `bytes` further on has
// the low word plus bytes / 16.
constexpr uint32_t kOperandHigh = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t operand_low(uint32_t smem, uint32_t lead) {
    return ((lead >> 4) << 16) | ((smem & 0x3ffffu) >> 4);
}

// Instruction descriptor of kind::f16: fp32 accumulator, both operands bf16
// or both fp16, majorness (0: K), sizes.
constexpr uint32_t f16_instr(bool bf16, uint32_t a_mn, uint32_t b_mn, uint32_t m, uint32_t n) {
    return (1u << 4) | ((bf16 ? 1u : 0u) << 7) | ((bf16 ? 1u : 0u) << 10) | (a_mn << 15) |
           (b_mn << 16) | ((n >> 3) << 17) | ((m >> 4) << 24);
}

// The same with 64-byte-swizzled lines, 8 lines to a 512-byte group.
constexpr uint32_t kOperandHigh64 = (512u >> 4) | (1u << 14) | (4u << 29);

// Instruction descriptor of kind::f8f6f4: fp32 accumulator, both operands
// E4M3, K-major.
constexpr uint32_t e4m3_instr(uint32_t m, uint32_t n) {
    return (1u << 4) | ((n >> 3) << 17) | ((m >> 4) << 24);
}

// D (+)= A B, one k32 step of E4M3 operands; A_HIGH: A's high word.
template <uint32_t A_HIGH>
__device__ __forceinline__ void mma_e4m3_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t instr,
                                            bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "mov.b64 x, {%1, %5};\n\tmov.b64 y, {%2, %6};\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], x, y, %3, p;\n\t}"
        ::"r"(d), "r"(a), "r"(b), "r"(instr), "r"((uint32_t)accumulate), "n"(A_HIGH),
        "n"(kOperandHigh)
        : "memory");
}

// D (+)= A B, one k16 step, operands by their low words; one thread issues.
__device__ __forceinline__ void mma_f16_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t instr,
                                           bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "mov.b64 x, {%1, %5};\n\tmov.b64 y, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n\t}"
        ::"r"(d), "r"(a), "r"(b), "r"(instr), "r"((uint32_t)accumulate), "n"(kOperandHigh)
        : "memory");
}

// Arrive on `bar` when every MMA this thread issued so far has completed.
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
    asm volatile(
        "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
            smem_addr(bar))
        : "memory");
}

__device__ __forceinline__ void fence_before_sync() {
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void fence_after_sync() {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

// Tensor memory: one warp allocates and frees (all its lanes).
__device__ __forceinline__ void tmem_alloc(uint32_t* where, uint32_t columns) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_addr(where)),
                 "r"(columns)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}
__device__ __forceinline__ void tmem_free(uint32_t base, uint32_t columns) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(base), "r"(columns));
}
__device__ __forceinline__ void tmem_st_wait() {
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// The loads wait for their data in the same statement: until the wait the
// registers belong to the load, and the compiler must not move or reuse them.
// 16 lanes x 64 columns: thread t gets, for i = 0..7, columns 8i + 2(t%4) and
// + 1 of lane t/4 (r[4i], r[4i+1]) and of lane t/4 + 8 (r[4i+2], r[4i+3]).
__device__ __forceinline__ void tmem_ld_16x64(float (&r)[32], uint32_t addr) {
    uint32_t* u = reinterpret_cast<uint32_t*>(r);
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x8.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]),
          "=r"(u[7]), "=r"(u[8]), "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]),
          "=r"(u[14]), "=r"(u[15]), "=r"(u[16]), "=r"(u[17]), "=r"(u[18]), "=r"(u[19]),
          "=r"(u[20]), "=r"(u[21]), "=r"(u[22]), "=r"(u[23]), "=r"(u[24]), "=r"(u[25]),
          "=r"(u[26]), "=r"(u[27]), "=r"(u[28]), "=r"(u[29]), "=r"(u[30]), "=r"(u[31])
        : "r"(addr)
        : "memory");
}

// 32 lanes x 16 columns: thread t gets 16 columns of lane t.
__device__ __forceinline__ void tmem_ld_32x16(float (&r)[16], uint32_t addr) {
    uint32_t* u = reinterpret_cast<uint32_t*>(r);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]),
          "=r"(u[7]), "=r"(u[8]), "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]),
          "=r"(u[14]), "=r"(u[15])
        : "r"(addr)
        : "memory");
}
__device__ __forceinline__ void tmem_st_32x16(uint32_t addr, const float (&r)[16]) {
    const uint32_t* u = reinterpret_cast<const uint32_t*>(r);
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};"
        ::"r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7]),
        "r"(u[8]), "r"(u[9]), "r"(u[10]), "r"(u[11]), "r"(u[12]), "r"(u[13]), "r"(u[14]),
        "r"(u[15]), "r"(addr)
        : "memory");
}

}  // namespace kvw
