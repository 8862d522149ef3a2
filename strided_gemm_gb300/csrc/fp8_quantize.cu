// Quantisation to 8-bit floats with a scale for each group x 128 elements
// (sbgemm_quantize_fp8):
//     scale = max(fl(amax / largest), 2^-126),   y = fl8(fl(x / scale))
// amax over the block's finite elements.  Both quotients are IEEE divisions:
// where 7 divides amax's mantissa, x / scale is a tie of e4m3 for common x, and
// one ulp of either quotient would decide it.
//
// Bound: the bytes of X and Y. Kernels, by where X and Y have their unit strides:
//   rows       K in both: 16 lanes a block, 8 elements a lane, one pass
//   tiles      K in both, 128 rows a scale: a CTA a block, held in registers
//   turned     X's along its rows (a transposed matrix), Y's along K: a CTA takes
//              128 x 128 elements, 8 rows by 8 of K a thread, and turns the 8-bit
//              values in shared memory, where 8-byte pieces change places by their
//              row's number, so that neither side meets a bank twice
//   any        any strides, a warp or a CTA a block, element by element
//
// Quotients. With r = fl(1 / scale), q0 = fl(x r) and the exact remainder x - q0
// scale from a fused multiply-add, fl(q0 + remainder r) is the correctly rounded
// quotient (P. Markstein, Computation of elementary functions on the IBM RISC
// System/6000 processor, 1990) as long as nothing underflows: below a scale of
// 2^-70 both x and the scale are multiplied by 2^60 first. Infinities and NaN come
// out as NaN. (64 divisions a thread take 26 us for 7100 x 4096 fp16, their code
// alone being more than the instruction cache holds.)
//
// Measured on a GB300, device time in a graph whose replays find these arrays in L2,
// and behind a flushed L2: rows 4099 x 4096 bf16 12.9 and 16.3 us (3.1 TB/s from memory),
// fp32 14.0 and 18.8 (4.5 TB/s); tiles 7100 x 4096 fp16 16.3 and 22 (4.0 TB/s); turned
// 2560 x 8192 bf16 19.7 and 25 (2.5 TB/s); any 4099 x 4095 bf16 45 and 46. Bound: by what
// is in flight. Of bf16 rows from memory the counters show 53 % of the SMs' peak, 25 % of
// DRAM's and 42 % of the warps, which wait for their own loads and for fixed latencies; a
// thread of the turned kernel loads nothing while its CTA converts and stores.
#include <algorithm>
#include <type_traits>

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

// fl(x / y) from inverse = fl(1 / y).
__device__ __forceinline__ float divided(float x, float y, float inverse) {
    const float q = x * inverse;
    return fmaf(fmaf(-q, y, x), inverse, q);
}
constexpr float kLow = 8.470329472543003e-22f, kLift = 1152921504606846976.0f;     // 2^-70, 2^60

// What a block's elements are divided by, and its scale.
struct Divisor {
    float scale, lift, lifted, inverse;
    __device__ __forceinline__ float of(float x) const { return divided(x, lifted, inverse); }      // of an x times lift
    __device__ __forceinline__ bool low() const { return lift != 1.0f; }
};
__device__ __forceinline__ Divisor divisor(float amax, float largest) {
    Divisor d;
    // (A quotient of this size below fp32's normals becomes the least scale anyway.)
    const float up = amax < kLow ? kLift : 1.0f;
    d.scale = fmaxf(divided(amax * up, largest, largest == 448.0f ? 1.0f / 448.0f : 1.0f / 57344.0f) * (1.0f / up), kSmallest);
    d.lift = d.scale < kLow ? kLift : 1.0f;
    d.lifted = d.scale * d.lift;
    d.inverse = __frcp_rn(d.lifted);
    return d;
}

// 8 consecutive elements as floats; those from `n` on are 0.
__device__ __forceinline__ void load8(const float* x, int n, const ByteSpan& span, float (&v)[8]) {
    if (n >= 8 && dbg_in_bytes(x, 32, span, &g_status)) {
        const float4 a = *reinterpret_cast<const float4*>(x), b = *reinterpret_cast<const float4*>(x + 4);
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < n && dbg_in_bytes(x + i, 4, span, &g_status) ? x[i] : 0.0f;
}
// Raw vectors of 8, to be held: the 16-bit types stay packed.
template <typename T> struct Raw8 {
    uint4 w;
    __device__ __forceinline__ void load(const T* x, int n, const ByteSpan& span) {
        if (n >= 8 && dbg_in_bytes(x, 16, span, &g_status)) {
            w = *reinterpret_cast<const uint4*>(x);
            return;
        }
        uint32_t h[4] = {0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n && dbg_in_bytes(x + i, 2, span, &g_status))
                h[i / 2] |= (uint32_t)*reinterpret_cast<const uint16_t*>(x + i) << (16 * (i & 1));
        w = make_uint4(h[0], h[1], h[2], h[3]);
    }
    __device__ __forceinline__ void get(float (&v)[8]) const {
        const uint32_t h[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = unpack2<T>(h[i]);
            v[2 * i] = f.x;
            v[2 * i + 1] = f.y;
        }
    }
};
template <> struct Raw8<float> {
    float v[8];
    __device__ __forceinline__ void load(const float* x, int n, const ByteSpan& span) { load8(x, n, span, v); }
    __device__ __forceinline__ void get(float (&o)[8]) const {
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = v[i];
    }
};
// Largest finite magnitudes, element by element, of vectors of 8.  The bits of a
// magnitude order as integers, so 16-bit types need no conversion.
template <typename T> struct Top8 {
    uint32_t w[4] = {};
    static constexpr uint32_t kInf2 = std::is_same<T, __half>::value ? 0x7c007c00u : 0x7f807f80u;
    template <int n> __device__ __forceinline__ void take(const Raw8<T> (&r)[n]) {
#pragma unroll
        for (int q = 0; q < n; ++q) {
            w[0] = __vmaxu2(w[0], r[q].w.x & 0x7fff7fffu);
            w[1] = __vmaxu2(w[1], r[q].w.y & 0x7fff7fffu);
            w[2] = __vmaxu2(w[2], r[q].w.z & 0x7fff7fffu);
            w[3] = __vmaxu2(w[3], r[q].w.w & 0x7fff7fffu);
        }
        const uint32_t m = __vmaxu2(__vmaxu2(w[0], w[1]), __vmaxu2(w[2], w[3]));
        if ((m & 0xffffu) < (kInf2 & 0xffffu) && m < (kInf2 & 0xffff0000u)) return;
        // Something is not finite: again, without what is not.
        w[0] = w[1] = w[2] = w[3] = 0;
#pragma unroll 1
        for (int i = 0; i < 4; ++i) {
            uint32_t t = 0;
#pragma unroll
            for (int q = 0; q < n; ++q) {
                const uint32_t a = (i == 0 ? r[q].w.x : i == 1 ? r[q].w.y : i == 2 ? r[q].w.z : r[q].w.w) & 0x7fff7fffu;
                t = __vmaxu2(t, a & __vcmpltu2(a, kInf2));
            }
            if (i == 0) w[0] = t;
            else if (i == 1) w[1] = t;
            else if (i == 2) w[2] = t;
            else w[3] = t;
        }
    }
    __device__ __forceinline__ void get(float (&v)[8]) const {
        Raw8<T> r;
        r.w = make_uint4(w[0], w[1], w[2], w[3]);
        r.get(v);
    }
    __device__ __forceinline__ float all() const {
        const float2 f = unpack2<T>(__vmaxu2(__vmaxu2(w[0], w[1]), __vmaxu2(w[2], w[3])));
        return fmaxf(f.x, f.y);
    }
};
template <> struct Top8<float> {
    float v[8] = {};
    template <int n> __device__ __forceinline__ void take(const Raw8<float> (&r)[n]) {
#pragma unroll
        for (int q = 0; q < n; ++q)
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = fmaxf(v[i], finite_size(r[q].v[i]));
    }
    __device__ __forceinline__ void get(float (&o)[8]) const {
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = v[i];
    }
    __device__ __forceinline__ float all() const {
        return fmaxf(fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3])), fmaxf(fmaxf(v[4], v[5]), fmaxf(v[6], v[7])));
    }
};
__device__ __forceinline__ uint2 pack8(float (&v)[8], const Divisor& d, bool e4m3) {
    if (d.low()) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] *= d.lift;
    }
    uint32_t h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = pack_fp8x2(d.of(v[2 * i]), d.of(v[2 * i + 1]), e4m3);
    return make_uint2(__byte_perm(h[0], h[1], 0x5410), __byte_perm(h[2], h[3], 0x5410));
}
// 8 values of a row of Y, the first n of them.
__device__ __forceinline__ void store8(uint8_t* y, uint2 w, int n, const ByteSpan& span) {
    if (n >= 8) {
        if (dbg_in_bytes(y, 8, span, &g_status)) *reinterpret_cast<uint2*>(y) = w;
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < n && dbg_in_bytes(y + i, 1, span, &g_status)) y[i] = (uint8_t)((i < 4 ? w.x : w.y) >> (8 * (i & 3)));
}

// A warp takes 2 n blocks of a row, 16 lanes each.
template <typename T, int n>
__global__ void __launch_bounds__(kThreads) rows_kernel(const __grid_constant__ QuantizeProblem p) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const bool e4m3 = p.type_y == SBGEMM_TYPE_E4M3;
    const float largest = fp8_largest(p.type_y);
    const int lane = threadIdx.x & 31, half = lane >> 4, piece = lane & 15, K = (int)p.K;
    const int kb = (K + kScaleBlock - 1) / kScaleBlock, per_row = (kb + 2 * n - 1) / (2 * n);
    const int64_t items = p.batch * p.M * per_row;
    for (int64_t it = (int64_t)blockIdx.x * (kThreads / 32) + threadIdx.x / 32; it < items;
         it += (int64_t)gridDim.x * (kThreads / 32)) {
        const int64_t r = it / per_row, m = r % p.M, b = r / p.M;
        const int j0 = (int)(it - r * per_row) * 2 * n + half, k0 = j0 * kScaleBlock + piece * 8;
        const T* x = static_cast<const T*>(p.X) + b * p.bsX + m * p.rsX + k0;
        uint8_t* y = p.Y + b * p.bsY + m * p.rsY + k0;
        float* s = p.S + b * p.bsS + m * p.rsS + j0 * p.ksS;
        Raw8<T> raw[n][1];
#pragma unroll
        for (int q = 0; q < n; ++q) raw[q][0].load(x + 2 * q * kScaleBlock, K - k0 - 2 * q * kScaleBlock, p.sx);
#pragma unroll
        for (int q = 0; q < n; ++q) {
            Top8<T> tops;
            tops.take(raw[q]);
            float top = tops.all();
#pragma unroll
            for (int o = 8; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
            const Divisor d = divisor(top, largest);
            float v[8];
            raw[q][0].get(v);
            store8(y + 2 * q * kScaleBlock, pack8(v, d, e4m3), K - k0 - 2 * q * kScaleBlock, p.sy);
            float* at = s + 2 * q * p.ksS;
            if (piece == 0 && j0 + 2 * q < kb && dbg_in_bytes(at, 4, p.ss, &g_status)) *at = d.scale;
        }
    }
}

// Maximum over the CTA's threads, the same in all of them.
__device__ __forceinline__ float block_max(float v, float* shared) {
    v = warp_max(v);
    if ((threadIdx.x & 31) == 0) shared[threadIdx.x >> 5] = v;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) v = fmaxf(v, shared[w]);
    return v;
}

// A CTA a block of 128 x 128.
template <typename T>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 3 : 2) tiles_kernel(const __grid_constant__ QuantizeProblem p) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    __shared__ float shared[kThreads / 32];
    const int64_t kb = (p.K + kScaleBlock - 1) / kScaleBlock, mb = (p.M + 127) / 128;
    const int64_t j = blockIdx.x % kb, r = blockIdx.x / kb % mb, b = blockIdx.x / kb / mb;
    const int64_t k = j * kScaleBlock + (threadIdx.x & 15) * 8, m0 = r * 128 + (threadIdx.x >> 4);
    const int n = k < p.K ? (int)min((int64_t)8, p.K - k) : 0;
    const T* x = static_cast<const T*>(p.X) + b * p.bsX + k;
    Raw8<T> raw[8];
    Top8<T> top;
#pragma unroll
    for (int q = 0; q < 8; ++q) raw[q].load(x + (m0 + 16 * q) * p.rsX, m0 + 16 * q < p.M ? n : 0, p.sx);
    top.take(raw);
    const Divisor d = divisor(block_max(top.all(), shared), fp8_largest(p.type_y));
#pragma unroll
    for (int q = 0; q < 8; ++q) {
        float v[8];
        raw[q].get(v);
        const uint2 w = pack8(v, d, p.type_y == SBGEMM_TYPE_E4M3);
        if (n > 0 && m0 + 16 * q < p.M) store8(p.Y + b * p.bsY + (m0 + 16 * q) * p.rsY + k, w, n, p.sy);
    }
    float* s = p.S + b * p.bsS + r * p.rsS + j * p.ksS;
    if (threadIdx.x == 0 && dbg_in_bytes(s, 4, p.ss, &g_status)) *s = d.scale;
}

// 128 rows by 128 elements of K of an X with unit stride along its rows.
template <typename T>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 3 : 2) turned_kernel(const __grid_constant__ QuantizeProblem p) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    __shared__ alignas(16) float tops[kThreads / 32][128];
    __shared__ float shared[kThreads / 32];
    __shared__ alignas(16) uint2 out[128][16];
    const bool e4m3 = p.type_y == SBGEMM_TYPE_E4M3;
    const float largest = fp8_largest(p.type_y);
    const int64_t kb = (p.K + kScaleBlock - 1) / kScaleBlock, mb = (p.M + 127) / 128;
    // (Tiles side by side along the rows read the same rows of memory.)
    const int64_t r = blockIdx.x % mb, j = blockIdx.x / mb % kb, b = blockIdx.x / mb / kb;
    const int mi = threadIdx.x & 15, ki = threadIdx.x >> 4, warp = threadIdx.x >> 5;
    const int64_t m0 = r * 128 + mi * 8, k0 = j * kScaleBlock + ki * 8;
    const int n = m0 < p.M ? (int)min((int64_t)8, p.M - m0) : 0;
    const T* x = static_cast<const T*>(p.X) + b * p.bsX + m0;
    Raw8<T> raw[8];                       // [element of K]: 8 rows
#pragma unroll
    for (int q = 0; q < 8; ++q) raw[q].load(x + (k0 + q) * p.csX, k0 + q < p.K ? n : 0, p.sx);
    float top[8];
    {
        Top8<T> each;
        each.take(raw);
        each.get(top);
    }
    if (p.group == 1) {
#pragma unroll
        for (int i = 0; i < 8; ++i) top[i] = fmaxf(top[i], __shfl_xor_sync(~0u, top[i], 16));
        if ((threadIdx.x & 16) == 0) {
            *reinterpret_cast<float4*>(&tops[warp][mi * 8]) = make_float4(top[0], top[1], top[2], top[3]);
            *reinterpret_cast<float4*>(&tops[warp][mi * 8 + 4]) = make_float4(top[4], top[5], top[6], top[7]);
        }
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) {
            const float4 a = *reinterpret_cast<const float4*>(&tops[w][mi * 8]);
            const float4 c = *reinterpret_cast<const float4*>(&tops[w][mi * 8 + 4]);
            top[0] = fmaxf(top[0], a.x); top[1] = fmaxf(top[1], a.y); top[2] = fmaxf(top[2], a.z); top[3] = fmaxf(top[3], a.w);
            top[4] = fmaxf(top[4], c.x); top[5] = fmaxf(top[5], c.y); top[6] = fmaxf(top[6], c.z); top[7] = fmaxf(top[7], c.w);
        }
    } else {
        float all = top[0];
#pragma unroll
        for (int i = 1; i < 8; ++i) all = fmaxf(all, top[i]);
        all = block_max(all, shared);
#pragma unroll
        for (int i = 0; i < 8; ++i) top[i] = all;
    }
    float* s = p.S + b * p.bsS + j * p.ksS;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const Divisor d = divisor(top[i], largest);
        // Row m0 + i: its 8 elements of K.
        uint32_t h[4];
#pragma unroll
        for (int q = 0; q < 8; q += 2) {
            float u[8], v[8];
            raw[q].get(u);
            raw[q + 1].get(v);
            h[q / 2] = pack_fp8x2(d.of(u[i] * d.lift), d.of(v[i] * d.lift), e4m3);
        }
        out[mi * 8 + i][ki ^ mi] = make_uint2(__byte_perm(h[0], h[1], 0x5410), __byte_perm(h[2], h[3], 0x5410));
        if (ki == 0 && i < n && (p.group == 1 || (mi == 0 && i == 0))) {
            float* at = s + (p.group == 1 ? m0 + i : r) * p.rsS;
            if (dbg_in_bytes(at, 4, p.ss, &g_status)) *at = d.scale;
        }
    }
    __syncthreads();
    const int64_t k = j * kScaleBlock + mi * 8;
    if (k >= p.K) return;
#pragma unroll
    for (int q = 0; q < 8; ++q) {
        const int row = ki + 16 * q;
        const int64_t m = r * 128 + row;
        if (m < p.M)
            store8(p.Y + b * p.bsY + m * p.rsY + k, out[row][mi ^ (row >> 3)], (int)min((int64_t)8, p.K - k), p.sy);
    }
}

template <typename... Args>
cudaError_t start(void (*kernel)(Args...), int64_t blocks, cudaStream_t stream, const QuantizeProblem& p) {
    // Launched while the kernel before may still run, for which the kernels wait themselves.
    cudaLaunchAttribute early{};
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cfg.attrs = &early;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

// The kernel for a layout: whole vectors of 8 along X's unit stride and along K of Y.
template <typename T>
cudaError_t launch(const QuantizeProblem& p, cudaStream_t stream) {
    const int64_t kb = (p.K + kScaleBlock - 1) / kScaleBlock, mb = (p.M + 127) / 128, most = 1 << 20;
    auto whole = [](const void* base, int64_t bytes, int64_t s, int64_t n, int64_t bs, int64_t batch, int64_t each) {
        return reinterpret_cast<uintptr_t>(base) % bytes == 0 && (n <= 1 || s % each == 0) && (batch <= 1 || bs % each == 0);
    };
    const bool y = (p.ksY == 1 || p.K == 1) && whole(p.Y, 8, p.rsY, p.M, p.bsY, p.batch, 8);
    const bool along_k = (p.csX == 1 || p.K == 1) && whole(p.X, 16, p.rsX, p.M, p.bsX, p.batch, 8);
    const bool along_m = p.rsX == 1 && whole(p.X, 16, p.csX, p.K, p.bsX, p.batch, 8);
    if (y && along_k && p.group == 1 && p.K < ((int64_t)1 << 30)) {        // (its indexes are ints)
        // 8 blocks a warp where a row has them, else 2: short rows and few of them want more warps.
        const int n = kb >= 8 && p.batch * p.M * kb >= 8192 ? 4 : 1;
        const int64_t items = p.batch * p.M * ((kb + 2 * n - 1) / (2 * n)), blocks = std::min((items + 7) / 8, most);
        return n == 4 ? start(rows_kernel<T, 4>, blocks, stream, p) : start(rows_kernel<T, 1>, blocks, stream, p);
    }
    const int64_t tiles = p.batch * mb * kb;
    if (y && tiles < ((int64_t)1 << 31)) {
        if (along_k) return start(tiles_kernel<T>, tiles, stream, p);
        if (along_m) return start(turned_kernel<T>, tiles, stream, p);
    }
    if (p.group == 1) {
        const int64_t items = p.batch * p.M * kb, per = kThreads / 32;
        rows_any_kernel<T><<<(unsigned)std::min((items + per - 1) / per, most), kThreads, 0, stream>>>(p);
    } else {
        blocks_any_kernel<T><<<(unsigned)std::min(tiles, most), kThreads, 0, stream>>>(p);
    }
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_quantize(const QuantizeProblem& p, cudaStream_t stream) {
    if (p.type_x == SBGEMM_TYPE_BF16) return launch<__nv_bfloat16>(p, stream);
    if (p.type_x == SBGEMM_TYPE_FP16) return launch<__half>(p, stream);
    return launch<float>(p, stream);
}

unsigned int* status_word_fp8_quantize() { return word_address(&g_status); }

}  // namespace sbg
