// The 16-bit strided product for any layout (sbgemm_half): C = alpha A B (+ C)
// with every operand read element by element through its strides, fp32 sums,
// one rounding at the end.
//
// 64 x 64 tiles of C, K in steps of 16 through shared memory, 256 threads of
// 4 x 4 outputs each.  This is the kernel of layouts without a tensor map
// (no unit stride, odd alignments); it is bound by its scalar loads and by
// FFMA issue, an order below the tensor cores.
#include <algorithm>

#include "debug_check.cuh"
#include "half_util.cuh"
#include "serving.h"

namespace sbg {
namespace {

constexpr int BM = 64, BN = 64, BK = 16;
__device__ unsigned int g_status = 0;

template <typename T>
__global__ void __launch_bounds__(256)
half_gather_kernel(const HalfProblem p, int64_t tiles_n) {
    __shared__ float sa[BK][BM + 1], sb[BK][BN + 1];
    const int t = threadIdx.x, tx = t & 15, ty = t >> 4;
    const int64_t m0 = (int64_t)(blockIdx.x / tiles_n) * BM, n0 = (int64_t)(blockIdx.x % tiles_n) * BN;
    for (int64_t b = blockIdx.y; b < p.batch; b += gridDim.y) {
        const T* A = static_cast<const T*>(p.A) + b * p.bsA;
        const T* B = static_cast<const T*>(p.B) + b * p.bsB;
        T* C = static_cast<T*>(p.C) + b * p.bsC;
        float acc[4][4] = {};
        for (int64_t k0 = 0; k0 < p.K; k0 += BK) {
#pragma unroll
            for (int i = t; i < BK * BM; i += 256) {
                // The unit-stride index, if any, runs across the threads.
                const int ka = p.csA == 1 ? i % BK : i / BM, ma = p.csA == 1 ? i / BK : i % BM;
                const int kb = p.csB == 1 ? i / BN : i % BK, nb = p.csB == 1 ? i % BN : i / BK;
                const T* a = A + (m0 + ma) * p.rsA + (k0 + ka) * p.csA;
                const T* bb = B + (k0 + kb) * p.rsB + (n0 + nb) * p.csB;
                sa[ka][ma] = m0 + ma < p.M && k0 + ka < p.K && dbg_in_bytes(a, sizeof(T), p.sa, &g_status)
                                 ? to_float(*a) : 0.0f;
                sb[kb][nb] = n0 + nb < p.N && k0 + kb < p.K && dbg_in_bytes(bb, sizeof(T), p.sb, &g_status)
                                 ? to_float(*bb) : 0.0f;
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
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int64_t m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
                if (m < p.M && n < p.N) {
                    T* c = C + m * p.rsC + n * p.csC;
                    if (!dbg_in_bytes(c, sizeof(T), p.sc, &g_status)) continue;
                    *c = from_float<T>(p.accumulate ? fmaf(p.alpha, acc[i][j], to_float(*c)) : p.alpha * acc[i][j]);
                }
            }
    }
}

}  // namespace

cudaError_t launch_half_gather(const HalfProblem& p, cudaStream_t stream) {
    const int64_t tn = (p.N + BN - 1) / BN, tiles = (p.M + BM - 1) / BM * tn;
    if (tiles >= ((int64_t)1 << 31)) return cudaErrorInvalidValue;
    const dim3 grid((unsigned)tiles, (unsigned)std::min<int64_t>(p.batch, 65535));
    if (p.type == SBGEMM_TYPE_BF16)
        half_gather_kernel<__nv_bfloat16><<<grid, 256, 0, stream>>>(p, tn);
    else
        half_gather_kernel<__half><<<grid, 256, 0, stream>>>(p, tn);
    return cudaGetLastError();
}

unsigned int* status_word_half_gather() { return word_address(&g_status); }

}  // namespace sbg
