// Norms of queries, keys and latents with the rotation of their positions in
// one pass, and the gradient (sbgemm_norm_rope, sbgemm_norm_rope_backward).
//
// Angles.  A pair turns by position * step of 2^-64 turns.  The product modulo
// 2^64 is the angle modulo a turn without any error, for every position; its
// top two bits are the quadrant and the rest, exact to fp32's 24 bits, an angle
// of at most an eighth of a turn either side.
//
// rows_kernel: a CTA a row, any sizes and alignments.  A first pass over the
// row makes its sums, a second one the outputs; a thread has a pair, or an
// element that is not rotated, to itself in both, so that y may be x.  Bound by
// its scalar loads and by an angle a pair and row.
#include <algorithm>

#include "debug_check.cuh"
#include "half_util.cuh"
#include "layers.h"

namespace sbg {
namespace {

__device__ unsigned int g_status = 0;
constexpr int kRowThreads = 128;
// Blocks of the backward kernels an SM, each with its partial sums of dweight.
constexpr int kGradBlocks = 4;

__device__ __forceinline__ float value(float v) { return v; }
template <typename T> __device__ __forceinline__ float value(T v) { return to_float(v); }
__device__ __forceinline__ void put(float& o, float v) { o = v; }
template <typename T> __device__ __forceinline__ void put(T& o, float v) { o = from_float<T>(v); }

// magnitude * cosine and sine of position * step.
__device__ __forceinline__ float2 turn(int position, uint64_t step, float magnitude) {
    const uint64_t phase = (uint64_t)(int64_t)position * step;
    const uint32_t q = (uint32_t)((phase + (1ull << 61)) >> 62);         // the nearest quarter turn
    const float x = (float)(int64_t)(phase - ((uint64_t)q << 62)) * 1.0842021724855044e-19f;   // half turns: 2^-63
    float s, c;
    sincospif(x, &s, &c);
    const float cs = q & 1 ? s : c, sn = q & 1 ? c : s;
    return make_float2(q == 1 || q == 2 ? -magnitude * cs : magnitude * cs, q & 2 ? -magnitude * sn : magnitude * sn);
}

// Sum over the CTA's threads, the same in all of them.
__device__ __forceinline__ float block_sum(float v, float* shared) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) shared[threadIdx.x >> 5] = v;
    __syncthreads();
    float r = 0.0f;
#pragma unroll
    for (int w = 0; w < kRowThreads / 32; ++w) r += shared[w];
    return r;
}

// Items of a row: first its pairs, then the elements that are not rotated.
struct Items {
    int pairs, dims, start, interleaved, count;
    __device__ __forceinline__ Items(const RopeProblem& p, const RopePart& a)
        : pairs(p.dims / 2), dims(p.dims), start(a.start), interleaved(p.interleaved), count(a.D - p.dims / 2) {}
    __device__ __forceinline__ int first(int i) const {
        if (i < pairs) return interleaved ? start + 2 * i : start + i;
        const int e = i - pairs;
        return e < start ? e : e + dims;
    }
    __device__ __forceinline__ int second(int i) const { return first(i) + (interleaved ? 1 : pairs); }
};

template <typename T, bool kBackward>
__global__ void __launch_bounds__(kRowThreads) rows_kernel(const __grid_constant__ RopeProblem p, int64_t norm_total) {
    __shared__ float shared[kRowThreads / 32];
    const int tid = threadIdx.x;
    int64_t rows = 0;
    for (int n = 0; n < p.n_parts; ++n) rows += p.tokens * p.part[n].heads;
    float* slot = kBackward && p.workspace ? p.workspace + blockIdx.x * norm_total : nullptr;
    if (slot)
        for (int64_t e = tid; e < norm_total; e += kRowThreads) slot[e] = 0.0f;
    __syncthreads();
    for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
        int64_t r = row, before = 0;
        int n = 0;
        while (r >= p.tokens * p.part[n].heads) {
            r -= p.tokens * p.part[n].heads;
            before += p.part[n].norm;
            ++n;
        }
        const RopePart& a = p.part[n];
        const int64_t t = r / a.heads, h = r % a.heads;
        const int position = p.positions ? p.positions[t] : 0;
        const T* x = static_cast<const T*>(a.x) + t * a.tsX + h * a.hsX;
        const T* dy = static_cast<const T*>(a.dy) + t * a.tsD + h * a.hsD;
        T* y = static_cast<T*>(a.y) + t * a.tsY + h * a.hsY;
        auto load = [](const T* at, const ByteSpan& s) {
            return dbg_in_bytes(at, sizeof(T), s, &g_status) ? value(*at) : 0.0f;
        };
        auto weight = [&](int e) { return a.weight ? load(static_cast<const T*>(a.weight) + e, a.sw) : 1.0f; };
        const Items items(p, a);
        // The gradient of item i's elements before the rotation.
        auto gradient = [&](int i) {
            if (i >= items.pairs) return make_float2(load(dy + items.first(i), a.sd), 0.0f);
            const float2 cs = turn(position, p.steps[i], p.magnitude);
            const float u = load(dy + items.first(i), a.sd), v = load(dy + items.second(i), a.sd);
            return make_float2(fmaf(u, cs.x, v * cs.y), fmaf(v, cs.x, -u * cs.y));
        };
        float r_norm = 1.0f, mean = 0.0f;
        if (a.norm) {
            float ss = 0.0f, dot = 0.0f;
            for (int e = tid; e < a.norm; e += kRowThreads) {
                const float v = load(x + e, a.sx);
                ss = fmaf(v, v, ss);
            }
            r_norm = rsqrtf(block_sum(ss, shared) / a.norm + p.eps);
            if constexpr (kBackward) {
                for (int i = tid; i < items.count; i += kRowThreads) {
                    const float2 g = gradient(i);
                    const int e = items.first(i), f = items.second(i);
                    if (e < a.norm) dot = fmaf(g.x * weight(e), load(x + e, a.sx), dot);
                    if (i < items.pairs && f < a.norm) dot = fmaf(g.y * weight(f), load(x + f, a.sx), dot);
                }
                mean = block_sum(dot, shared) * r_norm / a.norm;
            }
        }
        // One element of the output, given its gradient going backward.
        auto element = [&](int e, float g) {
            if constexpr (!kBackward) {
                const float v = load(x + e, a.sx);
                return e < a.norm ? v * r_norm * weight(e) : v;
            } else {
                if (e >= a.norm) return g;
                const float v = load(x + e, a.sx) * r_norm;
                if (slot && a.dweight) slot[before + e] += g * v;
                return r_norm * (g * weight(e) - v * mean);
            }
        };
        for (int i = tid; i < items.count; i += kRowThreads) {
            const int e = items.first(i), f = items.second(i);
            const float2 g = kBackward ? gradient(i) : make_float2(0.0f, 0.0f);
            float u = element(e, g.x), v = i < items.pairs ? element(f, g.y) : 0.0f;
            if (!kBackward && i < items.pairs) {
                const float2 cs = turn(position, p.steps[i], p.magnitude);
                const float a0 = u, b0 = v;
                u = fmaf(a0, cs.x, -b0 * cs.y);
                v = fmaf(a0, cs.y, b0 * cs.x);
            }
            if (dbg_in_bytes(y + e, sizeof(T), a.sy, &g_status)) put(y[e], u);
            if (i < items.pairs && dbg_in_bytes(y + f, sizeof(T), a.sy, &g_status)) put(y[f], v);
        }
        __syncthreads();
    }
}

// dweight: the blocks' partial sums in order, in 64 bits (131072 rows of fp32
// sums keep an error of some 2^-22 of theirs then).
__global__ void __launch_bounds__(256) sum_kernel(const __grid_constant__ RopeProblem p, int64_t norm_total, int blocks) {
    __shared__ double sums[8][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t e = (int64_t)blockIdx.x * 32 + lane;
    double s = 0.0;
    if (e < norm_total)
        for (int b = warp; b < blocks; b += 8) s += (double)p.workspace[b * norm_total + e];
    sums[warp][lane] = s;
    __syncthreads();
    if (warp != 0 || e >= norm_total) return;
    for (int w = 1; w < 8; ++w) s += sums[w][lane];
    int64_t at = e;
    int n = 0;
    while (at >= p.part[n].norm) at -= p.part[n++].norm;
    float* out = p.part[n].dweight;
    if (!out || !dbg_in_bytes(out + at, 4, p.part[n].sdw, &g_status)) return;
    out[at] = (float)(p.accumulate ? s + (double)out[at] : s);
}

int64_t norm_total(const RopeProblem& p) {
    int64_t n = 0;
    for (int i = 0; i < p.n_parts; ++i) n += p.part[i].norm;
    return n;
}

template <typename T>
cudaError_t launch(const RopeProblem& p, bool backward, int sms, cudaStream_t stream) {
    int64_t rows = 0;
    for (int i = 0; i < p.n_parts; ++i) rows += p.tokens * p.part[i].heads;
    const int64_t total = norm_total(p);
    if (!backward) {
        rows_kernel<T, false><<<(unsigned)std::min<int64_t>(rows, 1 << 20), kRowThreads, 0, stream>>>(p, total);
        return cudaGetLastError();
    }
    const int blocks = (int)std::min<int64_t>(rows, (int64_t)sms * kGradBlocks);
    rows_kernel<T, true><<<blocks, kRowThreads, 0, stream>>>(p, total);
    if (p.workspace) sum_kernel<<<(unsigned)((total + 31) / 32), 256, 0, stream>>>(p, total, blocks);
    return cudaGetLastError();
}

cudaError_t launch_any(const RopeProblem& p, bool backward, int sms, cudaStream_t stream) {
    if (p.type == SBGEMM_TYPE_BF16) return launch<__nv_bfloat16>(p, backward, sms, stream);
    if (p.type == SBGEMM_TYPE_FP16) return launch<__half>(p, backward, sms, stream);
    return launch<float>(p, backward, sms, stream);
}

}  // namespace

cudaError_t launch_norm_rope(const RopeProblem& p, int sms, cudaStream_t stream) {
    return launch_any(p, false, sms, stream);
}
cudaError_t launch_norm_rope_backward(const RopeProblem& p, int sms, cudaStream_t stream) {
    return launch_any(p, true, sms, stream);
}
size_t norm_rope_workspace_bytes(int sms, int64_t norm_total) {
    return ((size_t)sms * kGradBlocks * (size_t)norm_total * 4 + 255) / 256 * 256;
}

unsigned int* status_word_norm_rope() { return word_address(&g_status); }

}  // namespace sbg
