// The product of 8-bit floats with block scales for any layout (sbgemm_fp8):
// every operand read element by element through its strides.
//
// 64 x 64 tiles of C, K in steps of 16 through shared memory, 256 threads of
// 4 x 4 outputs each; a block of 128 elements of K is summed on its own and
// joins the output's sum times its two scales.  This is the kernel of layouts
// without a tensor map (no unit stride along K, odd alignments), bound by its
// byte loads, conversions and FFMA issue.
#include <algorithm>

#include "debug_check.cuh"
#include "fp8_util.cuh"
#include "half_util.cuh"
#include "layers.h"

namespace sbg {
namespace {

constexpr int BM = 64, BN = 64, BK = 16;
__device__ unsigned int g_status = 0;

__device__ __forceinline__ void put(float& o, float v) { o = v; }
template <typename T> __device__ __forceinline__ void put(T& o, float v) { o = from_float<T>(v); }
__device__ __forceinline__ float get(float v) { return v; }
template <typename T> __device__ __forceinline__ float get(T v) { return to_float(v); }

template <typename T>
__global__ void __launch_bounds__(256) fp8_gather_kernel(const __grid_constant__ Fp8Problem p, int64_t tiles_n) {
    __shared__ float sa[BK][BM + 1], sb[BK][BN + 1];
    const int t = threadIdx.x, tx = t & 15, ty = t >> 4;
    const int64_t m0 = (int64_t)(blockIdx.x / tiles_n) * BM, n0 = (int64_t)(blockIdx.x % tiles_n) * BN;
    const bool ea = p.a.type == SBGEMM_TYPE_E4M3, eb = p.b.type == SBGEMM_TYPE_E4M3;
    // One element, 0 outside the operand.
    auto load = [&](const Fp8Operand& o, bool e4m3, int64_t b, int64_t r, int64_t k) {
        const uint8_t* at = o.data + b * o.bs + r * o.rs + k * o.ks;
        return r < o.rows && k < p.K && dbg_in_bytes(at, 1, o.sd, &g_status) ? fp8_to_float(*at, e4m3) : 0.0f;
    };
    auto scale = [&](const Fp8Operand& o, int64_t b, int64_t r, int64_t k0) {
        const float* at = o.scale + b * o.bsS + r / o.group * o.rsS + k0 / kScaleBlock * o.ksS;
        return r < o.rows && dbg_in_bytes(at, 4, o.ss, &g_status) ? *at : 0.0f;
    };
    for (int64_t b = blockIdx.y; b < p.batch; b += gridDim.y) {
        float sum[4][4] = {};
        for (int64_t kb = 0; kb < p.K; kb += kScaleBlock) {
            float acc[4][4] = {};
            for (int64_t k0 = kb; k0 < p.K && k0 < kb + kScaleBlock; k0 += BK) {
#pragma unroll
                for (int i = t; i < BK * BM; i += 256) {
                    // The unit-stride index, if any, runs across the threads.
                    const int ka = p.a.ks == 1 ? i % BK : i / BM, ma = p.a.ks == 1 ? i / BK : i % BM;
                    const int kc = p.b.ks == 1 ? i % BK : i / BN, nb = p.b.ks == 1 ? i / BK : i % BN;
                    sa[ka][ma] = load(p.a, ea, b, m0 + ma, k0 + ka);
                    sb[kc][nb] = load(p.b, eb, b, n0 + nb, k0 + kc);
                }
                __syncthreads();
#pragma unroll
                for (int k = 0; k < BK; ++k) {
                    float a[4], c[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) { a[i] = sa[k][ty + 16 * i]; c[i] = sb[k][tx + 16 * i]; }
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(a[i], c[j], acc[i][j]);
                }
                __syncthreads();
            }
            float fa[4], fb[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                fa[i] = scale(p.a, b, m0 + ty + 16 * i, kb);
                fb[i] = scale(p.b, b, n0 + tx + 16 * i, kb);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) sum[i][j] = fmaf(acc[i][j], fa[i] * fb[j], sum[i][j]);
        }
        T* C = static_cast<T*>(p.C) + b * p.bsC;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int64_t m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
                if (m < p.a.rows && n < p.b.rows) {
                    T* c = C + m * p.rsC + n * p.csC;
                    if (!dbg_in_bytes(c, sizeof(T), p.sc, &g_status)) continue;
                    put(*c, p.accumulate ? fmaf(p.alpha, sum[i][j], get(*c)) : p.alpha * sum[i][j]);
                }
            }
    }
}

}  // namespace

cudaError_t launch_fp8_gather(const Fp8Problem& p, cudaStream_t stream) {
    const int64_t tn = (p.b.rows + BN - 1) / BN, tiles = (p.a.rows + BM - 1) / BM * tn;
    if (tiles >= ((int64_t)1 << 31)) return cudaErrorInvalidValue;
    const dim3 grid((unsigned)tiles, (unsigned)std::min<int64_t>(p.batch, 65535));
    if (p.type_c == SBGEMM_TYPE_BF16) fp8_gather_kernel<__nv_bfloat16><<<grid, 256, 0, stream>>>(p, tn);
    else if (p.type_c == SBGEMM_TYPE_FP16) fp8_gather_kernel<__half><<<grid, 256, 0, stream>>>(p, tn);
    else fp8_gather_kernel<float><<<grid, 256, 0, stream>>>(p, tn);
    return cudaGetLastError();
}

unsigned int* status_word_fp8_gather() { return word_address(&g_status); }

}  // namespace sbg
