// Norms of queries, keys and latents with the rotation of their positions in
// one pass, and the gradient (sbgemm_norm_rope, sbgemm_norm_rope_backward).
//
// Angles.  A pair turns by position * step of 2^-64 turns.  The product modulo
// 2^64 is the angle modulo a turn without any error, for every position; its
// top two bits are the quadrant and the rest, exact to fp32's 24 bits, an angle
// of at most an eighth of a turn either side.
//
// vectors_kernel: rows whose elements come in whole vectors.  A unit is two
// vectors: the two members of V pairs (i, i + dims / 2), or V interleaved pairs
// one behind the other, or two vectors that are not rotated.  L lanes (a power of
// two) take a row's units, one to four each, held in registers, and walk through
// several heads of a token with its cosines, sines and weights.  Norms are sums
// over the L lanes.  A lane alone reads and writes its elements, so that y may be
// x (what neither changes is then not touched).  The backward kernel's groups of
// lanes walk through (token, heads) items and keep their share of dweight in
// registers; a CTA adds its groups' in a fixed order and leaves one partial sum.
// Bound by the bytes of x and y.
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

// ---- rows in vectors -----------------------------------------------------------------

constexpr int kVecThreads = 256;

// How a launch goes through one array.
struct PartPlan {
    int first_block, blocks;         // its CTAs
    int log_lanes;                   // lanes a row, log2
    int rotated, units;              // units that are rotated, and all
    int heads_each, chunks;          // heads an item, items a token
    int column;                      // of its first normed element among all arrays'
    int in_place;                    // y is x (dx is dy)
};
struct VecPlan { PartPlan part[SBGEMM_MAX_ROPE_PARTS]; int columns; };

// V elements as they lie in memory.
template <typename T, int V> struct alignas(V * sizeof(T)) Vec {
    uint32_t w[V * sizeof(T) / 4];
    __device__ __forceinline__ void get(float (&f)[V]) const {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < V; ++i) f[i] = __uint_as_float(w[i]);
        } else {
#pragma unroll
            for (int i = 0; i < V / 2; ++i) {
                const float2 x = unpack2<T>(w[i]);
                f[2 * i] = x.x;
                f[2 * i + 1] = x.y;
            }
        }
    }
    __device__ __forceinline__ void set(const float (&f)[V]) {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < V; ++i) w[i] = __float_as_uint(f[i]);
        } else {
#pragma unroll
            for (int i = 0; i < V / 2; ++i) w[i] = pack2<T>(f[2 * i], f[2 * i + 1]);
        }
    }
};

// (a, b) turned by the angles of V pairs, or back: b's members are the pairs'
// second ones, or each vector holds V / 2 pairs of its own.
template <int V, bool kBack>
__device__ __forceinline__ void rotate(float (&a)[V], float (&b)[V], const float2 (&cs)[V], bool interleaved) {
    auto pair = [&](float& u, float& v, const float2& c) {
        const float x = u, y = v, s = kBack ? -c.y : c.y;
        u = fmaf(x, c.x, -y * s);
        v = fmaf(x, s, y * c.x);
    };
    if (interleaved) {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            pair(a[2 * i], a[2 * i + 1], cs[i]);
            pair(b[2 * i], b[2 * i + 1], cs[V / 2 + i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) pair(a[i], b[i], cs[i]);
    }
}

template <typename T, int V, int KU, bool kBackward>
__global__ void __launch_bounds__(kVecThreads) vectors_kernel(const __grid_constant__ RopeProblem p,
                                                              const __grid_constant__ VecPlan plan) {
    using W = Vec<T, V>;
    extern __shared__ float dsum[];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    int n = 0;
    while (n + 1 < p.n_parts && (int)blockIdx.x >= plan.part[n + 1].first_block) ++n;
    const RopePart& a = p.part[n];
    const PartPlan& q = plan.part[n];
    const int L = 1 << q.log_lanes, lane = threadIdx.x & (L - 1), warp = threadIdx.x >> 5;
    const unsigned group_mask = L == 32 ? ~0u : ((1u << L) - 1) << (threadIdx.x & 31 & ~(L - 1));
    const float inv_norm = a.norm ? 1.0f / a.norm : 0.0f;
    // This lane's units: where their vectors lie, and what happens to them.
    int o1[KU], o2[KU];
    bool turned[KU], has1[KU], has2[KU], norm1[KU], norm2[KU];
    W w1[KU], w2[KU];
    float sw1[kBackward ? KU : 1][V], sw2[kBackward ? KU : 1][V];      // shares of dweight
    asm volatile("griddepcontrol.wait;" ::: "memory");
#pragma unroll
    for (int k = 0; k < KU; ++k) {
        const int u = lane + (k << q.log_lanes);
        turned[k] = u < q.rotated;
        if (turned[k]) {
            o1[k] = a.start + u * (p.interleaved ? 2 * V : V);
            o2[k] = o1[k] + (p.interleaved ? V : p.dims / 2);
            has1[k] = has2[k] = true;
        } else {
            const int e1 = 2 * (u - q.rotated) * V, e2 = e1 + V, rest = a.D - p.dims;
            o1[k] = e1 < a.start ? e1 : e1 + p.dims;
            o2[k] = e2 < a.start ? e2 : e2 + p.dims;
            has1[k] = u < q.units && e1 < rest;
            has2[k] = u < q.units && e2 < rest;
        }
        norm1[k] = has1[k] && o1[k] < a.norm;
        norm2[k] = has2[k] && o2[k] < a.norm;
        if (q.in_place && !turned[k]) {      // what stays as it is, where it is
            has1[k] = norm1[k];
            has2[k] = norm2[k];
        }
        const T* w = static_cast<const T*>(a.weight);
        if (w && norm1[k] && dbg_in_bytes(w + o1[k], sizeof(W), a.sw, &g_status)) w1[k] = *reinterpret_cast<const W*>(w + o1[k]);
        if (w && norm2[k] && dbg_in_bytes(w + o2[k], sizeof(W), a.sw, &g_status)) w2[k] = *reinterpret_cast<const W*>(w + o2[k]);
        if constexpr (kBackward) {
#pragma unroll
            for (int i = 0; i < V; ++i) sw1[k][i] = sw2[k][i] = 0.0f;
        }
    }
    // Sum over a row's lanes, the same in all of them.
    auto row_sum = [&](float v) {
        for (int o = L >> 1; o; o >>= 1) v += __shfl_xor_sync(group_mask, v, o);
        return v;
    };
    auto load = [&](const T* at, const ByteSpan& s, bool there, W& v) {
        if (there && dbg_in_bytes(at, sizeof(W), s, &g_status)) v = *reinterpret_cast<const W*>(at);
        else
#pragma unroll
            for (uint32_t& x : v.w) x = 0;
    };
    auto store = [&](T* at, bool there, const float (&f)[V]) {
        W v;
        v.set(f);
        if (there && dbg_in_bytes(at, sizeof(W), a.sy, &g_status)) *reinterpret_cast<W*>(at) = v;
    };

    const int64_t items = p.tokens * q.chunks, groups = (int64_t)q.blocks * (kVecThreads >> q.log_lanes);
    for (int64_t it = (int64_t)(blockIdx.x - q.first_block) * (kVecThreads >> q.log_lanes) + (threadIdx.x >> q.log_lanes);
         it < items; it += groups) {
        const int64_t t = it / q.chunks;
        const int h0 = (int)(it - t * q.chunks) * q.heads_each, h1 = min(a.heads, h0 + q.heads_each);
        float2 cs[KU][V];
        if (q.rotated) {
            const int position = p.positions[t];
#pragma unroll
            for (int k = 0; k < KU; ++k) {
                if (!turned[k]) continue;
                const uint64_t* steps = p.steps + (lane + (k << q.log_lanes)) * V;
#pragma unroll
                for (int i = 0; i < V; ++i) cs[k][i] = turn(position, steps[i], p.magnitude);
            }
        }
        const T* in = kBackward ? static_cast<const T*>(a.dy) + t * a.tsD : static_cast<const T*>(a.x) + t * a.tsX;
        const int64_t hs = kBackward ? a.hsD : a.hsX;
        const ByteSpan& span = kBackward ? a.sd : a.sx;
        const T* x = static_cast<const T*>(a.x) + t * a.tsX;
        T* y = static_cast<T*>(a.y) + t * a.tsY;
        W r1[KU], r2[KU], x1[kBackward ? KU : 1], x2[kBackward ? KU : 1];
        auto fetch = [&](int h) {
#pragma unroll
            for (int k = 0; k < KU; ++k) {
                load(in + h * hs + o1[k], span, has1[k], r1[k]);
                load(in + h * hs + o2[k], span, has2[k], r2[k]);
                if constexpr (kBackward) {
                    load(x + h * a.hsX + o1[k], a.sx, norm1[k], x1[k]);
                    load(x + h * a.hsX + o2[k], a.sx, norm2[k], x2[k]);
                }
            }
        };
        fetch(h0);
        for (int h = h0; h < h1; ++h) {
            float f1[KU][V], f2[KU][V], g1[kBackward ? KU : 1][V], g2[kBackward ? KU : 1][V];
#pragma unroll
            for (int k = 0; k < KU; ++k) {
                r1[k].get(f1[k]);
                r2[k].get(f2[k]);
                if constexpr (kBackward) {
                    x1[k].get(g1[k]);
                    x2[k].get(g2[k]);
                }
            }
            // The next head's loads under this one's work.
            if (h + 1 < h1) fetch(h + 1);
            if constexpr (!kBackward) {
                if (a.norm) {
                    float ss = 0.0f;
#pragma unroll
                    for (int k = 0; k < KU; ++k)
#pragma unroll
                        for (int i = 0; i < V; ++i) {
                            if (norm1[k]) ss = fmaf(f1[k][i], f1[k][i], ss);
                            if (norm2[k]) ss = fmaf(f2[k][i], f2[k][i], ss);
                        }
                    const float r = rsqrtf(fmaf(row_sum(ss), inv_norm, p.eps));
#pragma unroll
                    for (int k = 0; k < KU; ++k) {
                        float u[V], v[V];
                        w1[k].get(u);
                        w2[k].get(v);
#pragma unroll
                        for (int i = 0; i < V; ++i) {
                            if (norm1[k]) f1[k][i] *= a.weight ? r * u[i] : r;
                            if (norm2[k]) f2[k][i] *= a.weight ? r * v[i] : r;
                        }
                    }
                }
#pragma unroll
                for (int k = 0; k < KU; ++k)
                    if (turned[k]) rotate<V, false>(f1[k], f2[k], cs[k], p.interleaved);
            } else {
#pragma unroll
                for (int k = 0; k < KU; ++k)
                    if (turned[k]) rotate<V, true>(f1[k], f2[k], cs[k], p.interleaved);
                if (a.norm) {
                    // x (in g) to the normed x, and the mean of g w x.
                    float ss = 0.0f, dot = 0.0f;
#pragma unroll
                    for (int k = 0; k < KU; ++k) {
                        float u[V], v[V];
                        w1[k].get(u);
                        w2[k].get(v);
#pragma unroll
                        for (int i = 0; i < V; ++i) {
                            if (norm1[k]) {
                                ss = fmaf(g1[k][i], g1[k][i], ss);
                                dot = fmaf(a.weight ? f1[k][i] * u[i] : f1[k][i], g1[k][i], dot);
                            }
                            if (norm2[k]) {
                                ss = fmaf(g2[k][i], g2[k][i], ss);
                                dot = fmaf(a.weight ? f2[k][i] * v[i] : f2[k][i], g2[k][i], dot);
                            }
                        }
                    }
                    const float r = rsqrtf(fmaf(row_sum(ss), inv_norm, p.eps));
                    const float mean = row_sum(dot) * r * inv_norm;
#pragma unroll
                    for (int k = 0; k < KU; ++k) {
                        float u[V], v[V];
                        w1[k].get(u);
                        w2[k].get(v);
#pragma unroll
                        for (int i = 0; i < V; ++i) {
                            if (norm1[k]) {
                                const float z = g1[k][i] * r;
                                sw1[k][i] = fmaf(f1[k][i], z, sw1[k][i]);
                                f1[k][i] = r * fmaf(-z, mean, a.weight ? f1[k][i] * u[i] : f1[k][i]);
                            }
                            if (norm2[k]) {
                                const float z = g2[k][i] * r;
                                sw2[k][i] = fmaf(f2[k][i], z, sw2[k][i]);
                                f2[k][i] = r * fmaf(-z, mean, a.weight ? f2[k][i] * v[i] : f2[k][i]);
                            }
                        }
                    }
                }
            }
#pragma unroll
            for (int k = 0; k < KU; ++k) {
                store(y + h * a.hsY + o1[k], has1[k], f1[k]);
                store(y + h * a.hsY + o2[k], has2[k], f2[k]);
            }
        }
    }
    if constexpr (kBackward) {
        if (!p.workspace || !a.norm || !a.dweight) return;
        // A warp's groups in a tree, then the warps one behind the other.
#pragma unroll
        for (int k = 0; k < KU; ++k)
#pragma unroll
            for (int i = 0; i < V; ++i)
                for (int o = L; o < 32; o <<= 1) {
                    sw1[k][i] += __shfl_xor_sync(~0u, sw1[k][i], o);
                    sw2[k][i] += __shfl_xor_sync(~0u, sw2[k][i], o);
                }
        for (int w = 0; w < kVecThreads / 32; ++w) {
            if (warp == w && (threadIdx.x & 31) < L) {
#pragma unroll
                for (int k = 0; k < KU; ++k)
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        if (norm1[k]) dsum[o1[k] + i] = (w ? dsum[o1[k] + i] : 0.0f) + sw1[k][i];
                        if (norm2[k]) dsum[o2[k] + i] = (w ? dsum[o2[k] + i] : 0.0f) + sw2[k][i];
                    }
            }
            __syncthreads();
        }
        float* slot = p.workspace + (int64_t)blockIdx.x * plan.columns + q.column;
        for (int e = threadIdx.x; e < a.norm; e += kVecThreads) slot[e] = dsum[e];
    }
}

// dweight: the blocks' partial sums in order, in 64 bits (131072 rows of fp32
// sums keep an error of some 2^-22 of theirs then).
__global__ void __launch_bounds__(256) sum_kernel(const __grid_constant__ RopeProblem p, const __grid_constant__ VecPlan plan) {
    __shared__ double sums[8][32];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int e = blockIdx.x * 32 + lane;
    double s = 0.0;
    int n = 0;
    if (e < plan.columns) {
        while (n + 1 < p.n_parts && e >= plan.part[n + 1].column) ++n;
        const int last = plan.part[n].first_block + plan.part[n].blocks;
        if (p.part[n].dweight)
            for (int b = plan.part[n].first_block + warp; b < last; b += 8)
                s += (double)p.workspace[(int64_t)b * plan.columns + e];
    }
    sums[warp][lane] = s;
    __syncthreads();
    if (warp != 0 || e >= plan.columns || !p.part[n].dweight) return;
    for (int w = 1; w < 8; ++w) s += sums[w][lane];
    float* out = p.part[n].dweight + (e - plan.part[n].column);
    if (dbg_in_bytes(out, 4, p.part[n].sdw, &g_status)) *out = (float)(p.accumulate ? s + (double)*out : s);
}

template <typename... Args, typename... Given>
cudaError_t start(void (*kernel)(Args...), int64_t blocks, int threads, size_t smem, cudaStream_t stream, const Given&... given) {
    // Launched while the kernel before may still run, for which the kernels wait themselves.
    cudaLaunchAttribute early{};
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = &early;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, given...);
}

// Whether all arrays' rows come in vectors of v elements.
bool whole_vectors(const RopeProblem& p, bool backward, int v, size_t esize) {
    auto whole = [&](const void* base, int64_t ts, int64_t hs, int64_t heads) {
        return reinterpret_cast<uintptr_t>(base) % (v * esize) == 0 && (p.tokens <= 1 || ts % v == 0) && (heads <= 1 || hs % v == 0);
    };
    if (p.dims / 2 % v != 0) return false;
    for (int i = 0; i < p.n_parts; ++i) {
        const RopePart& a = p.part[i];
        if (a.D % v != 0 || a.start % v != 0 || a.norm % v != 0) return false;
        if (!whole(a.y, a.tsY, a.hsY, a.heads) || (a.weight && !whole(a.weight, 0, 0, 1))) return false;
        if ((!backward || a.norm) && !whole(a.x, a.tsX, a.hsX, a.heads)) return false;
        if (backward && !whole(a.dy, a.tsD, a.hsD, a.heads)) return false;
    }
    return true;
}

int columns_of(const RopeProblem& p, VecPlan* plan) {
    plan->columns = 0;
    for (int i = 0; i < p.n_parts; ++i) {
        plan->part[i].column = plan->columns;
        plan->columns += p.part[i].norm;
    }
    return plan->columns;
}

cudaError_t launch_sum(const RopeProblem& p, const VecPlan& plan, cudaStream_t stream) {
    if (!p.workspace) return cudaSuccess;
    return start(sum_kernel, (plan.columns + 31) / 32, 256, 0, stream, p, plan);
}

template <typename T, int V, int KU>
cudaError_t launch_vectors(const RopeProblem& p, bool backward, const VecPlan& plan, int64_t blocks, cudaStream_t stream) {
    if (!backward) return start(vectors_kernel<T, V, KU, false>, blocks, kVecThreads, 0, stream, p, plan);
    int most = 0;
    for (int i = 0; i < p.n_parts; ++i) most = std::max(most, p.part[i].norm);
    if (const cudaError_t e = start(vectors_kernel<T, V, KU, true>, blocks, kVecThreads, most * sizeof(float), stream, p, plan))
        return e;
    return launch_sum(p, plan, stream);
}

// Lays the arrays out over CTAs; false when a row has more units than its lanes hold.
template <typename T, int V>
bool try_vectors(const RopeProblem& p, bool backward, int sms, cudaStream_t stream, cudaError_t* err) {
    VecPlan plan{};
    columns_of(p, &plan);
    int most = 1;
    int64_t threads = 0;             // lanes of all rows
    for (int i = 0; i < p.n_parts; ++i) {
        const RopePart& a = p.part[i];
        PartPlan& q = plan.part[i];
        q.rotated = p.dims / 2 / V;
        q.units = q.rotated + ((a.D - p.dims) / V + 1) / 2;
        q.log_lanes = 0;
        while (q.log_lanes < 5 && (1 << q.log_lanes) < q.units) ++q.log_lanes;
        most = std::max(most, (q.units + 31) / 32);
        q.in_place = backward ? a.y == a.dy : a.y == a.x;
        threads += (p.tokens * a.heads) << q.log_lanes;
    }
    if (most > 4) return false;
    // Heads an item: as many as leave every SM its threads, since each item works out
    // its angles anew (at most 16, all of a token's rows in flight being enough).
    const int64_t want = (int64_t)sms * (backward ? kGradBlocks * kVecThreads : 2048);
    const int64_t each = std::max<int64_t>(1, std::min<int64_t>(16, threads / want));
    int64_t blocks = 0;
    for (int i = 0; i < p.n_parts; ++i) {
        const RopePart& a = p.part[i];
        PartPlan& q = plan.part[i];
        q.chunks = (int)((a.heads + std::min<int64_t>(each, a.heads) - 1) / std::min<int64_t>(each, a.heads));
        q.heads_each = (a.heads + q.chunks - 1) / q.chunks;
        const int64_t per = kVecThreads >> q.log_lanes;
        int64_t mine = (p.tokens * q.chunks + per - 1) / per;
        if (backward) {
            // Its share of the partial sums' slots, by its rows' lanes.
            const int64_t share = (int64_t)((double)sms * kGradBlocks * (double)((p.tokens * a.heads) << q.log_lanes) / (double)threads);
            mine = std::min(mine, std::max<int64_t>(1, share - 1));
        }
        if (blocks + mine >= ((int64_t)1 << 31)) return false;
        q.first_block = (int)blocks;
        q.blocks = (int)mine;
        blocks += mine;
    }
    *err = most == 1 ? launch_vectors<T, V, 1>(p, backward, plan, blocks, stream)
         : most == 2 ? launch_vectors<T, V, 2>(p, backward, plan, blocks, stream)
                     : launch_vectors<T, V, 4>(p, backward, plan, blocks, stream);
    return true;
}

template <typename T>
cudaError_t launch(const RopeProblem& p, bool backward, int sms, cudaStream_t stream) {
    constexpr int V = 16 / sizeof(T);
    cudaError_t e = cudaSuccess;
    if (whole_vectors(p, backward, V, sizeof(T)) && try_vectors<T, V>(p, backward, sms, stream, &e)) return e;
    if (whole_vectors(p, backward, V / 2, sizeof(T)) && try_vectors<T, V / 2>(p, backward, sms, stream, &e)) return e;
    int64_t rows = 0;
    for (int i = 0; i < p.n_parts; ++i) rows += p.tokens * p.part[i].heads;
    VecPlan plan{};
    const int64_t total = columns_of(p, &plan);
    if (!backward) {
        rows_kernel<T, false><<<(unsigned)std::min<int64_t>(rows, 1 << 20), kRowThreads, 0, stream>>>(p, total);
        return cudaGetLastError();
    }
    const int blocks = (int)std::min<int64_t>(rows, (int64_t)sms * kGradBlocks);
    for (int i = 0; i < p.n_parts; ++i) plan.part[i].blocks = blocks;      // every CTA has a share of every array
    rows_kernel<T, true><<<blocks, kRowThreads, 0, stream>>>(p, total);
    if (const cudaError_t r = cudaGetLastError()) return r;
    return launch_sum(p, plan, stream);
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
