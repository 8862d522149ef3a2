// 8-bit floats on the device: conversions and their types' properties.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <cstdint>

#include "sbgemm.h"

namespace sbg {

// The largest finite value of a type.
__host__ __device__ constexpr float fp8_largest(int type) { return type == SBGEMM_TYPE_E4M3 ? 448.0f : 57344.0f; }

__device__ __forceinline__ float fp8_to_float(uint8_t v, bool e4m3) {
    return __half2float(__half(__nv_cvt_fp8_to_halfraw(v, e4m3 ? __NV_E4M3 : __NV_E5M2)));
}

// Two values rounded to nearest even and packed, `lo` in the low byte; what is
// larger than the largest value becomes it, NaN stays NaN.
__device__ __forceinline__ uint32_t pack_fp8x2(float lo, float hi, bool e4m3) {
    uint16_t r;
    if (e4m3) asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    else asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

}  // namespace sbg
