// Two fp32 values in a 64-bit register, for the instructions that work on both.
#pragma once

#include <cstdint>

namespace sbg {

__device__ __forceinline__ uint64_t pair_of(uint32_t lo, uint32_t hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
    return r;
}
__device__ __forceinline__ uint64_t pair_of(float lo, float hi) { return pair_of(__float_as_uint(lo), __float_as_uint(hi)); }
__device__ __forceinline__ float lower(uint64_t v) { return __uint_as_float((uint32_t)v); }
__device__ __forceinline__ float upper(uint64_t v) { return __uint_as_float((uint32_t)(v >> 32)); }

// acc += v f, rounded once.
__device__ __forceinline__ void fma2(uint64_t& acc, uint64_t v, uint64_t f) {
    asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc) : "l"(v), "l"(f));
}
// a b + c, rounded once.
__device__ __forceinline__ uint64_t mad2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

}  // namespace sbg
