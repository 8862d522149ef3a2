// Norms of queries, keys and latents with the rotation of their positions in
// one pass, and the gradient (sbgemm_norm_rope, sbgemm_norm_rope_backward).
//
// Angles.  A pair turns by position * step of 2^-64 turns.  The product modulo
// 2^64 is the angle modulo a turn without any error, for every position; its
// top bits are the nearest quarter turn and the rest, exact to fp32's 24 bits, an
// angle of at most an eighth of a turn either side.
//
// vectors_kernel: rows whose elements come in whole vectors.  A lane holds one
// unit of a row, two vectors: the two members of V pairs (i, i + dims / 2), or V
// interleaved pairs one behind the other, or two vectors that are not rotated.  L
// lanes (a power of two, up to the whole CTA) take a row and walk through several
// heads of a token, with its angles: forward as the 2 x 2 coefficients of a pair
// with the members' weights in them, so that a normed and rotated element costs
// three operations.  Norms are sums over the L lanes.  A lane alone reads and
// writes its elements, so that y may be x (what neither changes is then not
// touched).  The backward kernel's lanes keep their share of dweight in registers;
// a CTA adds its groups' in a fixed order and leaves one partial sum.
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
constexpr int kGradBlocks = 2;

__device__ __forceinline__ float value(float v) { return v; }
template <typename T> __device__ __forceinline__ float value(T v) { return to_float(v); }
__device__ __forceinline__ void put(float& o, float v) { o = v; }
template <typename T> __device__ __forceinline__ void put(T& o, float v) { o = from_float<T>(v); }

// magnitude * cosine and sine of position * step.  Within an eighth of a turn the
// Taylor polynomials of degree 9 and 10 are exact to 2^-29.
__device__ __forceinline__ float2 turn(int position, uint64_t step, float magnitude) {
    const uint64_t phase = (uint64_t)(int64_t)position * step;
    const uint32_t q = (uint32_t)((phase + (1ull << 61)) >> 62);         // the nearest quarter turn
    // What is left, in radians: 2 pi / 2^64.
    const float x = (float)(int64_t)(phase - ((uint64_t)q << 62)) * 3.4061215800304626e-19f;
    const float z = x * x;
    float s = fmaf(z, 2.7557319223985893e-6f, -1.9841269841269841e-4f);  // 1/9!, 1/7!, 1/5!, 1/3!
    s = fmaf(z, s, 8.3333333333333332e-3f);
    s = fmaf(z, s, -1.6666666666666666e-1f);
    s = fmaf(z * x, s, x);
    float c = fmaf(z, -2.7557319223985888e-7f, 2.4801587301587302e-5f);  // 1/10!, 1/8!, 1/6!, 1/4!, 1/2!
    c = fmaf(z, c, -1.3888888888888889e-3f);
    c = fmaf(z, c, 4.1666666666666664e-2f);
    c = fmaf(z, c, -0.5f);
    c = fmaf(z, c, 1.0f);
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

__device__ __forceinline__ float plus(float a, float b) { return a + b; }
__device__ __forceinline__ float2 plus(float2 a, float2 b) { return make_float2(a.x + b.x, a.y + b.y); }
__device__ __forceinline__ float other(float v, int o) { return __shfl_xor_sync(~0u, v, o); }
__device__ __forceinline__ float2 other(float2 v, int o) { return make_float2(other(v.x, o), other(v.y, o)); }
// The sum (or two sums) over a row's lanes, the same in all of them.  Rows of more
// than a warp meet in shared memory, in one of two buffers in turns.
template <typename F>
__device__ __forceinline__ F row_sums(F v, int L, float2 (&shared)[2][kVecThreads / 32], int& turns) {
    for (int o = min(L, 32) >> 1; o; o >>= 1) v = plus(v, other(v, o));
    if (L > 32) {
        float2* now = shared[turns++ & 1];
        const int warp = threadIdx.x >> 5, first = warp & ~((L >> 5) - 1);
        if ((threadIdx.x & 31) == 0) *reinterpret_cast<F*>(&now[warp]) = v;
        __syncthreads();
        v = *reinterpret_cast<const F*>(&now[first]);
        for (int w = 1; w < L >> 5; ++w) v = plus(v, *reinterpret_cast<const F*>(&now[first + w]));
    }
    return v;
}

template <typename T, int V, bool kBackward>
__global__ void __launch_bounds__(kVecThreads, kBackward ? 2 : 3) vectors_kernel(const __grid_constant__ RopeProblem p,
                                                                                 const __grid_constant__ VecPlan plan) {
    using W = Vec<T, V>;
    extern __shared__ float dsum[];
    __shared__ float2 meet[2][kVecThreads / 32];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    int n = 0, turns = 0;
    while (n + 1 < p.n_parts && (int)blockIdx.x >= plan.part[n + 1].first_block) ++n;
    const RopePart& a = p.part[n];
    const PartPlan& q = plan.part[n];
    const int L = 1 << q.log_lanes, u = threadIdx.x & (L - 1), warp = threadIdx.x >> 5;
    const float inv_norm = a.norm ? 1.0f / a.norm : 0.0f;
    const bool interleaved = p.interleaved;
    // This lane's unit: where its vectors lie, and what happens to them.
    const bool turned = u < q.rotated;
    int o1, o2;
    bool has1, has2;
    if (turned) {
        o1 = a.start + u * (interleaved ? 2 * V : V);
        o2 = o1 + (interleaved ? V : p.dims / 2);
        has1 = has2 = true;
    } else {
        const int e1 = 2 * (u - q.rotated) * V, e2 = e1 + V, rest = a.D - p.dims;
        o1 = e1 < a.start ? e1 : e1 + p.dims;
        o2 = e2 < a.start ? e2 : e2 + p.dims;
        has1 = u < q.units && e1 < rest;
        has2 = u < q.units && e2 < rest;
    }
    const bool norm1 = has1 && o1 < a.norm, norm2 = has2 && o2 < a.norm;
    if (q.in_place && !turned) {             // what stays as it is, where it is
        has1 = norm1;
        has2 = norm2;
    }
    // One member of a pair normed, the other not: norms before the rotation.
    const bool mixed = turned && !interleaved && norm1 != norm2;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    float w1[V], w2[V];                      // weights, 1 where there are none
    {
        const T* w = static_cast<const T*>(a.weight);
#pragma unroll
        for (int i = 0; i < V; ++i) w1[i] = w2[i] = 1.0f;
        if (w && norm1 && dbg_in_bytes(w + o1, sizeof(W), a.sw, &g_status)) reinterpret_cast<const W*>(w + o1)->get(w1);
        if (w && norm2 && dbg_in_bytes(w + o2, sizeof(W), a.sw, &g_status)) reinterpret_cast<const W*>(w + o2)->get(w2);
    }
    float sw1[V] = {}, sw2[V] = {};          // shares of dweight
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

    // (All of a CTA's groups go the same number of times round, as they meet at barriers.)
    const int64_t items = p.tokens * q.chunks;
    const int per = kVecThreads >> q.log_lanes, mine = threadIdx.x >> q.log_lanes;
    for (int64_t i0 = (int64_t)(blockIdx.x - q.first_block) * per; i0 < items; i0 += (int64_t)q.blocks * per) {
        const int64_t it = min(i0 + mine, items - 1), t = it / q.chunks;
        const int h0 = (int)(it - t * q.chunks) * q.heads_each, h1 = i0 + mine < items ? min(a.heads, h0 + q.heads_each) : h0;
        // A pair's first member is x.x a + x.y b, its second one x.z a + x.w b.
        float4 m[kBackward ? 1 : V];
        float2 cs[kBackward ? V : 1];
        if (turned) {
            const int position = p.positions[t];
            const uint64_t* steps = p.steps + u * V;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float2 c = turn(position, steps[i], p.magnitude);
                if constexpr (kBackward) {
                    cs[i] = c;
                } else {
                    constexpr int H = V / 2;
                    const float wa = mixed ? 1.0f : !interleaved ? w1[i] : i < H ? w1[2 * i] : w2[2 * (i - H)];
                    const float wb = mixed ? 1.0f : !interleaved ? w2[i] : i < H ? w1[2 * i + 1] : w2[2 * (i - H) + 1];
                    m[i] = make_float4(c.x * wa, -c.y * wb, c.y * wa, c.x * wb);
                }
            }
        }
        // Places of this head's vectors, moved on head by head.
        const int64_t hs = kBackward ? a.hsD : a.hsX;
        const T* in = (kBackward ? static_cast<const T*>(a.dy) + t * a.tsD : static_cast<const T*>(a.x) + t * a.tsX) + h0 * hs;
        const T *in1 = in + o1, *in2 = in + o2;
        const T* x = static_cast<const T*>(a.x) + t * a.tsX + h0 * a.hsX;
        const T *xn1 = x + o1, *xn2 = x + o2;
        T* y = static_cast<T*>(a.y) + t * a.tsY + h0 * a.hsY;
        T *out1 = y + o1, *out2 = y + o2;
        const ByteSpan& span = kBackward ? a.sd : a.sx;
        W r1, r2, x1, x2;
        auto fetch = [&](bool there) {
            load(in1, span, has1 && there, r1);
            load(in2, span, has2 && there, r2);
            in1 += hs;
            in2 += hs;
            if constexpr (kBackward) {
                load(xn1, a.sx, norm1 && there, x1);
                load(xn2, a.sx, norm2 && there, x2);
                xn1 += a.hsX;
                xn2 += a.hsX;
            }
        };
        const int count = h1 - h0;
        fetch(count > 0);
        for (int h = 0; h < q.heads_each; ++h) {
            const bool live = h < count;
            float f1[V], f2[V];
            r1.get(f1);
            r2.get(f2);
            if constexpr (!kBackward) {
                // The next head's loads under this one's work.
                if (h + 1 < q.heads_each) fetch(h + 1 < count);
                float r = 1.0f;
                if (a.norm) {
                    float ss = 0.0f;
                    if (norm1)
#pragma unroll
                        for (int i = 0; i < V; ++i) ss = fmaf(f1[i], f1[i], ss);
                    if (norm2)
#pragma unroll
                        for (int i = 0; i < V; ++i) ss = fmaf(f2[i], f2[i], ss);
                    r = rsqrtf(fmaf(row_sums(ss, L, meet, turns), inv_norm, p.eps));
                }
                if (mixed || !turned) {
                    // (In both cases each vector is normed with its weights or not.)
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        if (norm1) f1[i] *= r * w1[i];
                        if (norm2) f2[i] *= r * w2[i];
                    }
                }
                if (turned) {
                    const float ra = norm1 && !mixed ? r : 1.0f, rb = norm2 && !mixed ? r : 1.0f;
                    if (interleaved) {
#pragma unroll
                        for (int i = 0; i < V / 2; ++i) {
                            const float4 c = m[i], d = m[V / 2 + i];
                            const float a0 = f1[2 * i], a1 = f1[2 * i + 1], b0 = f2[2 * i], b1 = f2[2 * i + 1];
                            f1[2 * i] = ra * fmaf(a0, c.x, a1 * c.y);
                            f1[2 * i + 1] = ra * fmaf(a0, c.z, a1 * c.w);
                            f2[2 * i] = rb * fmaf(b0, d.x, b1 * d.y);
                            f2[2 * i + 1] = rb * fmaf(b0, d.z, b1 * d.w);
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < V; ++i) {
                            const float4 c = m[i];
                            const float a0 = f1[i], b0 = f2[i];
                            f1[i] = ra * fmaf(a0, c.x, b0 * c.y);
                            f2[i] = rb * fmaf(a0, c.z, b0 * c.w);
                        }
                    }
                }
            } else {
                float g1[V], g2[V];
                x1.get(g1);
                x2.get(g2);
                if (h + 1 < q.heads_each) fetch(h + 1 < count);
                if (turned) {
                    auto back = [](float& c, float& d, const float2& z) {
                        const float u0 = c, v0 = d;
                        c = fmaf(u0, z.x, v0 * z.y);
                        d = fmaf(v0, z.x, -u0 * z.y);
                    };
#pragma unroll
                    for (int i = 0; i < V / 2; ++i) {
                        if (interleaved) {
                            back(f1[2 * i], f1[2 * i + 1], cs[i]);
                            back(f2[2 * i], f2[2 * i + 1], cs[V / 2 + i]);
                        } else {
                            back(f1[i], f2[i], cs[i]);
                            back(f1[V / 2 + i], f2[V / 2 + i], cs[V / 2 + i]);
                        }
                    }
                }
                if (a.norm) {
                    // Sums of x^2 and g w x; then dweight's share and dx.
                    float2 sums = make_float2(0.0f, 0.0f);
                    if (norm1)
#pragma unroll
                        for (int i = 0; i < V; ++i) {
                            sums.x = fmaf(g1[i], g1[i], sums.x);
                            sums.y = fmaf(f1[i] * w1[i], g1[i], sums.y);
                        }
                    if (norm2)
#pragma unroll
                        for (int i = 0; i < V; ++i) {
                            sums.x = fmaf(g2[i], g2[i], sums.x);
                            sums.y = fmaf(f2[i] * w2[i], g2[i], sums.y);
                        }
                    sums = row_sums(sums, L, meet, turns);
                    const float r = rsqrtf(fmaf(sums.x, inv_norm, p.eps)), mean = sums.y * r * inv_norm;
                    if (norm1)
#pragma unroll
                        for (int i = 0; i < V; ++i) {
                            const float z = g1[i] * r;
                            sw1[i] = fmaf(f1[i], z, sw1[i]);
                            f1[i] = r * fmaf(-z, mean, f1[i] * w1[i]);
                        }
                    if (norm2)
#pragma unroll
                        for (int i = 0; i < V; ++i) {
                            const float z = g2[i] * r;
                            sw2[i] = fmaf(f2[i], z, sw2[i]);
                            f2[i] = r * fmaf(-z, mean, f2[i] * w2[i]);
                        }
                }
            }
            store(out1, has1 && live, f1);
            store(out2, has2 && live, f2);
            out1 += a.hsY;
            out2 += a.hsY;
        }
    }
    if constexpr (kBackward) {
        if (!p.workspace || !a.norm || !a.dweight) return;
        // A warp's groups in a tree, then the warps one behind the other.
#pragma unroll
        for (int i = 0; i < V; ++i)
            for (int o = L; o < 32; o <<= 1) {
                sw1[i] += __shfl_xor_sync(~0u, sw1[i], o);
                sw2[i] += __shfl_xor_sync(~0u, sw2[i], o);
            }
        const int row_warps = max(1, L >> 5);
        for (int w = 0; w < kVecThreads / 32; w += row_warps) {
            if (warp / row_warps * row_warps == w && (threadIdx.x & 31) < L) {
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    if (norm1) dsum[o1 + i] = (w ? dsum[o1 + i] : 0.0f) + sw1[i];
                    if (norm2) dsum[o2 + i] = (w ? dsum[o2 + i] : 0.0f) + sw2[i];
                }
            }
            __syncthreads();
        }
        float* slot = p.workspace + (int64_t)blockIdx.x * plan.columns + q.column;
        for (int e = threadIdx.x; e < a.norm; e += kVecThreads) slot[e] = dsum[e];
    }
}

// A sum and what its rounding lost (Knuth's two-sum): 48 bits without the slow
// 64-bit units, whose latency 300 partial sums in order would pay.
struct Sum {
    float hi = 0.0f, lo = 0.0f;
    __device__ __forceinline__ void add(float v) {
        const float s = __fadd_rn(hi, v), b = __fsub_rn(s, hi);
        lo = __fadd_rn(lo, __fadd_rn(__fsub_rn(hi, __fsub_rn(s, b)), __fsub_rn(v, b)));
        hi = s;
    }
};

// dweight: the blocks' partial sums in order.
constexpr int kSumWarps = 32;
__global__ void __launch_bounds__(kSumWarps * 32) sum_kernel(const __grid_constant__ RopeProblem p,
                                                             const __grid_constant__ VecPlan plan) {
    __shared__ float2 sums[kSumWarps][32];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int e = blockIdx.x * 32 + lane;
    Sum s;
    int n = 0;
    if (e < plan.columns) {
        while (n + 1 < p.n_parts && e >= plan.part[n + 1].column) ++n;
        const int last = plan.part[n].first_block + plan.part[n].blocks;
        const float* at = p.workspace + e;
        if (p.part[n].dweight)
            for (int b = plan.part[n].first_block + warp; b < last; b += 4 * kSumWarps) {
                float v[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = b + i * kSumWarps < last ? at[(int64_t)(b + i * kSumWarps) * plan.columns] : 0.0f;
#pragma unroll
                for (int i = 0; i < 4; ++i) s.add(v[i]);
            }
    }
    sums[warp][lane] = make_float2(s.hi, s.lo);
    __syncthreads();
    if (warp != 0 || e >= plan.columns || !p.part[n].dweight) return;
#pragma unroll 8
    for (int w = 1; w < kSumWarps; ++w) {
        const float2 v = sums[w][lane];
        s.add(v.x);
        s.add(v.y);
    }
    float* out = p.part[n].dweight + (e - plan.part[n].column);
    if (!dbg_in_bytes(out, 4, p.part[n].sdw, &g_status)) return;
    if (p.accumulate) s.add(*out);
    *out = fabsf(s.hi) < INFINITY ? s.hi + s.lo : s.hi;
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
    return start(sum_kernel, (plan.columns + 31) / 32, kSumWarps * 32, 0, stream, p, plan);
}

template <typename T, int V>
cudaError_t launch_vectors(const RopeProblem& p, bool backward, const VecPlan& plan, int64_t blocks, cudaStream_t stream) {
    if (!backward) return start(vectors_kernel<T, V, false>, blocks, kVecThreads, 0, stream, p, plan);
    int most = 0;
    for (int i = 0; i < p.n_parts; ++i) most = std::max(most, p.part[i].norm);
    if (const cudaError_t e = start(vectors_kernel<T, V, true>, blocks, kVecThreads, most * sizeof(float), stream, p, plan))
        return e;
    return launch_sum(p, plan, stream);
}

// Lays the arrays out over CTAs; false when a row has more units than a CTA has lanes.
template <typename T, int V>
bool try_vectors(const RopeProblem& p, bool backward, int sms, cudaStream_t stream, cudaError_t* err) {
    VecPlan plan{};
    columns_of(p, &plan);
    int64_t threads = 0;             // lanes of all rows
    for (int i = 0; i < p.n_parts; ++i) {
        const RopePart& a = p.part[i];
        PartPlan& q = plan.part[i];
        q.rotated = p.dims / 2 / V;
        q.units = q.rotated + ((a.D - p.dims) / V + 1) / 2;
        if (q.units > kVecThreads) return false;
        q.log_lanes = 0;
        while ((1 << q.log_lanes) < q.units) ++q.log_lanes;
        q.in_place = backward ? a.y == a.dy : a.y == a.x;
        threads += (p.tokens * a.heads) << q.log_lanes;
    }
    // Heads an item: as many as leave every SM its resident threads, since each item
    // works out its angles anew.
    const int64_t want = (int64_t)sms * (backward ? kGradBlocks : 3) * kVecThreads;
    // (Backward at most 4: 4096 tokens of 40 heads take 39 us so, 44 with up to 16.)
    const int64_t each = std::max<int64_t>(1, std::min<int64_t>(backward ? 4 : 16, threads / want));
    int64_t blocks = 0;
    for (int i = 0; i < p.n_parts; ++i) {
        const RopePart& a = p.part[i];
        PartPlan& q = plan.part[i];
        q.chunks = (int)((a.heads + std::min<int64_t>(each, a.heads) - 1) / std::min<int64_t>(each, a.heads));
        q.heads_each = (a.heads + q.chunks - 1) / q.chunks;
        const int64_t per = kVecThreads >> q.log_lanes;
        int64_t mine = (p.tokens * q.chunks + per - 1) / per;
        if (backward) {
            // Its share of the partial sums' slots, by its rows' lanes, one at least: so
            // that all of them are no more than there are, but for one each to spare.
            const int64_t slots = (int64_t)sms * kGradBlocks - p.n_parts;
            const int64_t share = (int64_t)((double)slots * (double)((p.tokens * a.heads) << q.log_lanes) / (double)threads);
            mine = std::min(mine, std::max<int64_t>(1, share));
        }
        if (blocks + mine >= ((int64_t)1 << 31)) return false;
        q.first_block = (int)blocks;
        q.blocks = (int)mine;
        blocks += mine;
    }
    *err = launch_vectors<T, V>(p, backward, plan, blocks, stream);
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
