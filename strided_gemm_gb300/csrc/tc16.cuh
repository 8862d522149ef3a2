// tcgen05 helpers of the 16-bit kernels: kind::f16 products (bf16 or fp16
// operands, fp32 accumulation), their instruction descriptors, and
// shared-memory descriptors of 128-byte swizzled tiles in either major order.
#pragma once

#include "half_util.cuh"
#include "ptx.cuh"

namespace sbg {

// kind::f16, D fp32, M = 128: N columns; *_mn: the operand's unit stride in
// shared memory runs along M or N instead of K.
__host__ __device__ constexpr uint32_t idesc16(bool bf16, int n, bool a_mn, bool b_mn) {
    return (1u << 4) | ((bf16 ? 1u : 0u) << 7) | ((bf16 ? 1u : 0u) << 10) | ((a_mn ? 1u : 0u) << 15) |
           ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) | ((128u >> 4) << 24);
}

// Shared-memory descriptor of a tile whose rows of 128 bytes (64 elements) are
// swizzled in groups of 8 rows (1024 bytes).  K-major: a row is one index of M
// or N with 64 of K.  MN-major: a row is one index of K with 64 of M or N, and
// `lbo` is the distance in bytes to the next 64 of them.
__device__ __forceinline__ uint64_t desc16(uint32_t smem_addr, uint32_t lbo = 16) {
    return ((uint64_t)kDescHiSw128 << 32) | ((lbo >> 4) << 16) | ((smem_addr >> 4) & 0x3FFF);
}
// A K step of 16 elements further: 32 bytes of a K-major row, 16 rows of an
// MN-major tile.  In descriptor units of 16 bytes.
constexpr uint32_t kStepK = 32 >> 4, kStepMN = 16 * 128 >> 4;

// D[tmem] (+)= A B, both from shared memory.
__device__ __forceinline__ void mma16_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
        ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}

// The same with A in TMEM: 128 lanes from address `a`, two elements of K a column.
__device__ __forceinline__ void mma16_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
        ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}

}  // namespace sbg
