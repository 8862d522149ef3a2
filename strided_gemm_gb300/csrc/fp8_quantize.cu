// Quantisation to 8-bit floats with a scale for each group x 128 elements
// (sbgemm_quantize_fp8):
//     scale = max(fl(amax / largest), 2^-126),   y = fl8(fl(x / scale))
// amax over the block's finite elements.  Both quotients are IEEE divisions:
// where 7 divides amax's mantissa, x / scale is a tie of e4m3 for common x, and
// one ulp of either quotient would decide it.
//
// Bound: the bytes of X and Y.  A warp takes a block of one row, 4 elements a
// lane; a CTA one of 128 rows, in two passes over them.  Any strides; the loads
// run along X's unit stride only where that is K.
#include <algorithm>

#include "debug_check.cuh"
#include "fp8_util.cuh"
#include "half_util.cuh"
#include "layers.h"

namespace sbg {
namespace {

__device__ unsigned int g_status = 0;
constexpr float kSmallest = 1.1754943508222875e-38f;    // 2^-126
constexpr int kThreads = 256;

__device__ __forceinline__ float value(float v) { return v; }
template <typename T> __device__ __forceinline__ float value(T v) { return to_float(v); }

// |x| of a finite x, else 0.
__device__ __forceinline__ float finite_size(float x) { return fabsf(x) < INFINITY ? fabsf(x) : 0.0f; }
// x / scale, NaN for what is not finite.
__device__ __forceinline__ float quotient(float x, float scale) {
    return fabsf(x) < INFINITY ? __fdiv_rn(x, scale) : NAN;
}
__device__ __forceinline__ float scale_of(float amax, float largest) {
    return fmaxf(__fdiv_rn(amax, largest), kSmallest);
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(~0u, v, o));
    return v;
}

template <typename T>
struct Element {
    const QuantizeProblem& p;
    bool e4m3;
    __device__ __forceinline__ float load(int64_t b, int64_t m, int64_t k) const {
        const T* x = static_cast<const T*>(p.X) + b * p.bsX + m * p.rsX + k * p.csX;
        return dbg_in_bytes(x, sizeof(T), p.sx, &g_status) ? value(*x) : 0.0f;
    }
    __device__ __forceinline__ void store(int64_t b, int64_t m, int64_t k, float v) const {
        uint8_t* y = p.Y + b * p.bsY + m * p.rsY + k * p.ksY;
        if (dbg_in_bytes(y, 1, p.sy, &g_status)) *y = (uint8_t)pack_fp8x2(v, 0.0f, e4m3);
    }
    __device__ __forceinline__ void store_scale(int64_t b, int64_t r, int64_t j, float v) const {
        float* s = p.S + b * p.bsS + r * p.rsS + j * p.ksS;
        if (dbg_in_bytes(s, 4, p.ss, &g_status)) *s = v;
    }
};

template <typename T>
__global__ void __launch_bounds__(kThreads) rows_any_kernel(const __grid_constant__ QuantizeProblem p) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const Element<T> x{p, p.type_y == SBGEMM_TYPE_E4M3};
    const int lane = threadIdx.x & 31;
    const int64_t kb = (p.K + kScaleBlock - 1) / kScaleBlock, items = p.batch * p.M * kb;
    const float largest = fp8_largest(p.type_y);
    for (int64_t i = (int64_t)blockIdx.x * (kThreads / 32) + threadIdx.x / 32; i < items;
         i += (int64_t)gridDim.x * (kThreads / 32)) {
        const int64_t j = i % kb, m = i / kb % p.M, b = i / kb / p.M;
        float v[4], top = 0.0f;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int64_t k = j * kScaleBlock + lane + 32 * q;
            v[q] = k < p.K ? x.load(b, m, k) : 0.0f;
            top = fmaxf(top, finite_size(v[q]));
        }
        const float s = scale_of(warp_max(top), largest);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int64_t k = j * kScaleBlock + lane + 32 * q;
            if (k < p.K) x.store(b, m, k, quotient(v[q], s));
        }
        if (lane == 0) x.store_scale(b, m, j, s);
    }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) blocks_any_kernel(const __grid_constant__ QuantizeProblem p) {
    __shared__ float tops[kThreads / 32];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const Element<T> x{p, p.type_y == SBGEMM_TYPE_E4M3};
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t kb = (p.K + kScaleBlock - 1) / kScaleBlock, mb = (p.M + 127) / 128;
    const float largest = fp8_largest(p.type_y);
    // The unit-stride index, if any, runs across the threads.
    const bool along_m = p.rsX == 1 && p.csX != 1;
    for (int64_t i = blockIdx.x; i < p.batch * mb * kb; i += gridDim.x) {
        const int64_t j = i % kb, r = i / kb % mb, b = i / kb / mb;
        auto at = [&](int e, int64_t* m, int64_t* k) {
            *m = r * 128 + (along_m ? e & 127 : e >> 7);
            *k = j * kScaleBlock + (along_m ? e >> 7 : e & 127);
            return *m < p.M && *k < p.K;
        };
        float top = 0.0f;
        int64_t m, k;
        for (int e = threadIdx.x; e < 128 * kScaleBlock; e += kThreads)
            if (at(e, &m, &k)) top = fmaxf(top, finite_size(x.load(b, m, k)));
        top = warp_max(top);
        if (lane == 0) tops[warp] = top;
        __syncthreads();
        for (int w = 0; w < kThreads / 32; ++w) top = fmaxf(top, tops[w]);
        __syncthreads();
        const float s = scale_of(top, largest);
        for (int e = threadIdx.x; e < 128 * kScaleBlock; e += kThreads)
            if (at(e, &m, &k)) x.store(b, m, k, quotient(x.load(b, m, k), s));
        if (threadIdx.x == 0) x.store_scale(b, r, j, s);
    }
}

template <typename T>
void launch(const QuantizeProblem& p, cudaStream_t stream) {
    const int64_t kb = (p.K + kScaleBlock - 1) / kScaleBlock;
    const int64_t most = 1 << 20;
    if (p.group == 1) {
        const int64_t items = p.batch * p.M * kb, per = kThreads / 32;
        rows_any_kernel<T><<<(unsigned)std::min((items + per - 1) / per, most), kThreads, 0, stream>>>(p);
    } else {
        const int64_t items = p.batch * ((p.M + 127) / 128) * kb;
        blocks_any_kernel<T><<<(unsigned)std::min(items, most), kThreads, 0, stream>>>(p);
    }
}

}  // namespace

cudaError_t launch_quantize(const QuantizeProblem& p, cudaStream_t stream) {
    if (p.type_x == SBGEMM_TYPE_BF16) launch<__nv_bfloat16>(p, stream);
    else if (p.type_x == SBGEMM_TYPE_FP16) launch<__half>(p, stream);
    else launch<float>(p, stream);
    return cudaGetLastError();
}

unsigned int* status_word_fp8_quantize() { return word_address(&g_status); }

}  // namespace sbg
