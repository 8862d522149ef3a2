// Norms of queries, keys and latents with the rotation of their positions in
// one pass, and the gradient (sbgemm_norm_rope, sbgemm_norm_rope_backward).
//
// Angles.  A pair turns by position * step of 2^-64 turns.  The product modulo
// 2^64 is the angle modulo a turn, for every position; its top 32 bits leave out
// less than 2^-29 radians.  They are the nearest quarter turn and the rest, an angle
// of at most an eighth of a turn either side.
//
// vectors_kernel: rows whose elements come in whole vectors.  A lane holds one
// unit of a row, two vectors: the two members of V pairs (i, i + dims / 2), or V
// interleaved pairs one behind the other, or two vectors that are not rotated.  L
// lanes (a power of two, up to the whole CTA) take a row and walk through a run of
// rows, head by head and token by token, with a token's angles: forward as the 2 x 2
// coefficients of a pair with the members' weights in them, so that a normed and
// rotated element costs three operations, two elements an instruction.  Norms are
// sums over the L lanes.  A lane alone reads and writes its elements, so that y may be
// x (what neither changes is then not touched).  The backward kernel's lanes keep
// their share of dweight in registers; a CTA adds its warps' in a fixed order and
// leaves one partial sum.
//
// Measured on a GB300, device time in a graph and behind a flushed L2: 8192 tokens of 40
// heads of 128, bf16, normed and rotated, 37 and 39 us, 4.5 and 4.3 TB/s (20000 tokens
// without norms 74 us, 5.5 TB/s); the gradient of 4096 of them 31.8 and 34.8 us, 4.0 and 3.6
// TB/s, where one element an instruction, angles from 64-bit arithmetic and a walk of
// four heads took 39.  Bound by what is in flight: the counters show 49 % of the SMs' peak
// and 40 % of DRAM's, the gradient's 52 and 52, with 23 % of the warps, since two CTAs of
// 118 and 128 registers a thread fill an SM.  (Angles made once a warp in shared memory,
// for rows taken in the order of memory: 45 and 44 us, by its bookkeeping.)
//
// rows_kernel: a CTA a row, any sizes and alignments.  A first pass over the
// row makes its sums, a second one the outputs; a thread has a pair, or an
// element that is not rotated, to itself in both, so that y may be x.  Bound by
// its scalar loads and by an angle a pair and row.
#include <algorithm>

#include "debug_check.cuh"
#include "f32x2.cuh"
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

// A token's position without its sign, and the factors of cosine and sine (which the
// sign belongs to).
struct Place {
    uint32_t at;
    float c, s;
    __device__ __forceinline__ Place(int position, float magnitude)
        : at(position < 0 ? 0u - (uint32_t)position : (uint32_t)position), c(magnitude), s(position < 0 ? -magnitude : magnitude) {}
};
// Cosine and sine of position * step, times their factors.  Within an eighth of a turn
// the Taylor polynomials of degree 9 and 10 are exact to 2^-29.
__device__ __forceinline__ float2 turn(const Place& p, uint64_t step) {
    const uint32_t phase = p.at * (uint32_t)(step >> 32) + __umulhi(p.at, (uint32_t)step);   // in 2^-32 turns
    const uint32_t q = phase + (1u << 29);                               // the nearest quarter turn on top
    // What is left, in radians: 2 pi / 2^32.
    const float x = (float)(int)(phase - (q & 0xc0000000u)) * 1.4629180792671596e-09f;
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
    const bool odd = q & 0x40000000u;
    const uint32_t cs = __float_as_uint(odd ? s : c) ^ ((q + 0x40000000u) & 0x80000000u);    // minus in quarters 1 and 2
    const uint32_t sn = __float_as_uint(odd ? c : s) ^ (q & 0x80000000u);                    // ... 2 and 3
    return make_float2(p.c * __uint_as_float(cs), p.s * __uint_as_float(sn));
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

// A sum and what its rounding lost (Knuth's two-sum): 48 bits without the slow
// 64-bit units, whose latency 300 partial sums in order would pay.
struct Sum {
    float hi = 0.0f, lo = 0.0f;
    __device__ __forceinline__ void add(float v) {
        const float s = __fadd_rn(hi, v), b = __fsub_rn(s, hi);
        lo = __fadd_rn(lo, __fadd_rn(__fsub_rn(hi, __fsub_rn(s, b)), __fsub_rn(v, b)));
        hi = s;
    }
    __device__ __forceinline__ float all() const { return fabsf(hi) < INFINITY ? hi + lo : hi; }
};

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
    // This CTA's sums of dweight, and behind all CTAs' what their roundings lost: it
    // adds up rows / CTAs of them one behind the other.
    float* slot = kBackward && p.workspace ? p.workspace + blockIdx.x * norm_total : nullptr;
    float* lost = slot + gridDim.x * norm_total;
    if (slot)
        for (int64_t e = tid; e < norm_total; e += kRowThreads) slot[e] = lost[e] = 0.0f;
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
        const Place place(p.positions ? p.positions[t] : 0, p.magnitude);
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
            const float2 cs = turn(place, p.steps[i]);
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
                if (slot && a.dweight) {
                    Sum sum{slot[before + e], lost[before + e]};
                    sum.add(g * v);
                    slot[before + e] = sum.hi;
                    lost[before + e] = sum.lo;
                }
                return r_norm * (g * weight(e) - v * mean);
            }
        };
        for (int i = tid; i < items.count; i += kRowThreads) {
            const int e = items.first(i), f = items.second(i);
            const float2 g = kBackward ? gradient(i) : make_float2(0.0f, 0.0f);
            float u = element(e, g.x), v = i < items.pairs ? element(f, g.y) : 0.0f;
            if (!kBackward && i < items.pairs) {
                const float2 cs = turn(place, p.steps[i]);
                const float a0 = u, b0 = v;
                u = fmaf(a0, cs.x, -b0 * cs.y);
                v = fmaf(a0, cs.y, b0 * cs.x);
            }
            if (dbg_in_bytes(y + e, sizeof(T), a.sy, &g_status)) put(y[e], u);
            if (i < items.pairs && dbg_in_bytes(y + f, sizeof(T), a.sy, &g_status)) put(y[f], v);
        }
        __syncthreads();
    }
    if (slot)
        for (int64_t e = tid; e < norm_total; e += kRowThreads) slot[e] = Sum{slot[e], lost[e]}.all();
}

// ---- rows in vectors -----------------------------------------------------------------

constexpr int kVecThreads = 256;
// Rows on their way to a group of lanes, and CTAs an SM, forward.
constexpr int kForwardAhead = 3, kForwardBlocks = 2;

// How a launch goes through one array.
struct PartPlan {
    int first_block, blocks;         // its CTAs
    int log_lanes;                   // lanes a row, log2
    int rotated, units;              // units that are rotated, and all
    int span;                        // rows, head by head, that a group of lanes walks through
    int column;                      // of its first normed element among all arrays'
    int in_place;                    // y is x (dx is dy)
};
struct VecPlan { PartPlan part[SBGEMM_MAX_ROPE_PARTS]; int columns; };

// V elements as they lie in memory.
template <typename T, int V> struct alignas(V * sizeof(T)) Vec {
    uint32_t w[V * sizeof(T) / 4];
    __device__ __forceinline__ void get(uint64_t (&f)[V / 2]) const {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            if constexpr (sizeof(T) == 4) {
                f[i] = pair_of(w[2 * i], w[2 * i + 1]);
            } else {
                const float2 x = unpack2<T>(w[i]);
                f[i] = pair_of(x.x, x.y);
            }
        }
    }
    __device__ __forceinline__ void set(const uint64_t (&f)[V / 2]) {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            if constexpr (sizeof(T) == 4) {
                w[2 * i] = __float_as_uint(lower(f[i]));
                w[2 * i + 1] = __float_as_uint(upper(f[i]));
            } else {
                w[i] = pack2<T>(lower(f[i]), upper(f[i]));
            }
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
__global__ void __launch_bounds__(kVecThreads, kBackward ? 2 : kForwardBlocks) vectors_kernel(const __grid_constant__ RopeProblem p,
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
    constexpr int H = V / 2;                 // pairs of elements a vector
    const uint64_t one = pair_of(1.0f, 1.0f);
    // Weights, 1 where there are none.
    auto weights = [&](uint64_t (&w1)[H], uint64_t (&w2)[H]) {
        const T* w = static_cast<const T*>(a.weight);
#pragma unroll
        for (int i = 0; i < H; ++i) w1[i] = w2[i] = one;
        if (w && norm1 && dbg_in_bytes(w + o1, sizeof(W), a.sw, &g_status)) reinterpret_cast<const W*>(w + o1)->get(w1);
        if (w && norm2 && dbg_in_bytes(w + o2, sizeof(W), a.sw, &g_status)) reinterpret_cast<const W*>(w + o2)->get(w2);
    };
    uint64_t w1[kBackward ? H : 1], w2[kBackward ? H : 1];
    if constexpr (kBackward) weights(w1, w2);
    uint64_t sw1[H] = {}, sw2[H] = {};       // shares of dweight
    auto load = [&](const T* at, const ByteSpan& s, bool there, W& v) {
        if (there && dbg_in_bytes(at, sizeof(W), s, &g_status)) v = *reinterpret_cast<const W*>(at);
        else
#pragma unroll
            for (uint32_t& x : v.w) x = 0;
    };
    auto store = [&](T* at, bool there, const uint64_t (&f)[H]) {
        W v;
        v.set(f);
        if (there && dbg_in_bytes(at, sizeof(W), a.sy, &g_status)) *reinterpret_cast<W*>(at) = v;
    };

    // This group's rows, a token's heads one behind the other. (All of a CTA's groups
    // go the same number of times round, as they meet at barriers.)
    const int per = kVecThreads >> q.log_lanes;
    const int64_t lo = ((int64_t)(blockIdx.x - q.first_block) * per + (threadIdx.x >> q.log_lanes)) * q.span;
    const int count = (int)max((int64_t)0, min(p.tokens * a.heads - lo, (int64_t)q.span));
    int64_t t = count > 0 ? lo / a.heads : 0;
    int h = count > 0 ? (int)(lo - t * a.heads) : 0;
    // Places of the next row to come in and of the next one to go out, moved on row by
    // row: by a head, or from the last one to the next token's first.
    const int64_t hs = kBackward ? a.hsD : a.hsX, ts = kBackward ? a.tsD : a.tsX;
    const T* in = (kBackward ? static_cast<const T*>(a.dy) : static_cast<const T*>(a.x)) + t * ts + h * hs;
    const T* x = static_cast<const T*>(a.x) + t * a.tsX + h * a.hsX;
    T* out = static_cast<T*>(a.y) + t * a.tsY + h * a.hsY;
    const int64_t in_wrap = ts - (a.heads - 1) * hs, x_wrap = a.tsX - (a.heads - 1) * a.hsX, out_wrap = a.tsY - (a.heads - 1) * a.hsY;
    const ByteSpan& span = kBackward ? a.sd : a.sx;
    constexpr int kAhead = kBackward ? 1 : kForwardAhead;
    W r1[kAhead], r2[kAhead], x1, x2;
    int hf = h, left = count;
    auto fetch = [&](W& r1, W& r2) {
        const bool there = left > 0, wrap = hf + 1 == a.heads;
        load(in + o1, span, has1 && there, r1);
        load(in + o2, span, has2 && there, r2);
        if constexpr (kBackward) {
            load(x + o1, a.sx, norm1 && there, x1);
            load(x + o2, a.sx, norm2 && there, x2);
            x += wrap ? x_wrap : a.hsX;
        }
        in += wrap ? in_wrap : hs;
        hf = wrap ? 0 : hf + 1;
        --left;
    };
    // A token's rotation.  Forward, with the weights in it: the elements i of the two
    // vectors (or the two elements of a pair i) are m[i] a + n[i] b and m[H + i] a +
    // n[H + i] b; of vectors that are not turned m and n are the weights.  Backward:
    // cosines and sines by elements (or by pairs).
    // (Zeros for groups without rows, which go round with the others.)
    uint64_t m[V] = {}, n2[kBackward ? 1 : V] = {};
    if constexpr (!kBackward) {
        if (!turned) {
            uint64_t v1[H], v2[H];
            weights(v1, v2);
#pragma unroll
            for (int i = 0; i < H; ++i) {
                m[i] = v1[i];
                n2[i] = v2[i];
            }
        }
    }
    int next = turned && count > 0 ? p.positions[t] : 0;     // (the next token's, ahead of its rows)
    bool fresh = true;
#pragma unroll
    for (int k = 0; k < kAhead; ++k) fetch(r1[k], r2[k]);
    for (int i0 = 0; i0 < q.span; i0 += kAhead)
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
        if (kAhead > 1 && i0 + k >= q.span) break;
        const bool live = i0 + k < count;
        if (turned && live && fresh) {
            const Place place(next, p.magnitude);
            next = t + 1 < p.tokens ? p.positions[t + 1] : 0;
            const uint64_t* steps = p.steps + u * V;
            // (Two angles at a time: all of them would not leave their registers free.)
            uint64_t v1[H], v2[H];
            if constexpr (!kBackward) weights(v1, v2);
#pragma unroll
            for (int i = 0; i < H; ++i) {
                const float2 c = turn(place, steps[interleaved ? i : 2 * i]);
                const float2 d = turn(place, steps[interleaved ? H + i : 2 * i + 1]);
                if (interleaved) {
                    if constexpr (kBackward) {
                        m[i] = pair_of(c.x, c.y);
                        m[H + i] = pair_of(d.x, d.y);
                    } else {
                        m[i] = mul2(pair_of(c.x, c.y), pair_of(lower(v1[i]), lower(v1[i])));
                        n2[i] = mul2(pair_of(-c.y, c.x), pair_of(upper(v1[i]), upper(v1[i])));
                        m[H + i] = mul2(pair_of(d.x, d.y), pair_of(lower(v2[i]), lower(v2[i])));
                        n2[H + i] = mul2(pair_of(-d.y, d.x), pair_of(upper(v2[i]), upper(v2[i])));
                    }
                } else {
                    m[i] = pair_of(c.x, d.x);
                    m[H + i] = pair_of(c.y, d.y);
                    if constexpr (!kBackward) {
                        const uint64_t wa = mixed ? one : v1[i], wb = mixed ? one : v2[i];
                        n2[i] = mul2(pair_of(-c.y, -d.y), wb);
                        n2[H + i] = mul2(m[i], wb);
                        m[i] = mul2(m[i], wa);
                        m[H + i] = mul2(m[H + i], wa);
                    }
                }
            }
        }
        uint64_t f1[H], f2[H];
        r1[k].get(f1);
        r2[k].get(f2);
        if constexpr (!kBackward) {
            fetch(r1[k], r2[k]);             // rows ahead on their way under this one's work
            float r = 1.0f;
            if (a.norm) {
                uint64_t ss = 0;
                if (norm1)
#pragma unroll
                    for (int i = 0; i < H; ++i) fma2(ss, f1[i], f1[i]);
                if (norm2)
#pragma unroll
                    for (int i = 0; i < H; ++i) fma2(ss, f2[i], f2[i]);
                r = rsqrtf(fmaf(row_sums(lower(ss) + upper(ss), L, meet, turns), inv_norm, p.eps));
            }
            const uint64_t rr = pair_of(r, r);
            if (!turned) {
#pragma unroll
                for (int i = 0; i < H; ++i) {
                    if (norm1) f1[i] = mul2(f1[i], mul2(rr, m[i]));
                    if (norm2) f2[i] = mul2(f2[i], mul2(rr, n2[i]));
                }
            } else if (mixed) {
                uint64_t w1[H], w2[H];
                weights(w1, w2);
#pragma unroll
                for (int i = 0; i < H; ++i) {
                    if (norm1) f1[i] = mul2(f1[i], mul2(rr, w1[i]));
                    if (norm2) f2[i] = mul2(f2[i], mul2(rr, w2[i]));
                }
            }
            if (turned) {
                const uint64_t ra = norm1 && !mixed ? rr : one, rb = norm2 && !mixed ? rr : one;
                if (interleaved) {
#pragma unroll
                    for (int i = 0; i < H; ++i) {
                        auto both = [](float v) { return pair_of(v, v); };
                        f1[i] = mul2(ra, mad2(m[i], both(lower(f1[i])), mul2(n2[i], both(upper(f1[i])))));
                        f2[i] = mul2(rb, mad2(m[H + i], both(lower(f2[i])), mul2(n2[H + i], both(upper(f2[i])))));
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < H; ++i) {
                        const uint64_t c = f1[i], d = f2[i];
                        f1[i] = mul2(ra, mad2(m[i], c, mul2(n2[i], d)));
                        f2[i] = mul2(rb, mad2(m[H + i], c, mul2(n2[H + i], d)));
                    }
                }
            }
        } else {
            uint64_t g1[H], g2[H];
            x1.get(g1);
            x2.get(g2);
            fetch(r1[k], r2[k]);
            if (turned) {
                if (interleaved) {
                    auto back = [](uint64_t f, uint64_t z) {
                        return pair_of(fmaf(lower(f), lower(z), upper(f) * upper(z)), fmaf(upper(f), lower(z), -lower(f) * upper(z)));
                    };
#pragma unroll
                    for (int i = 0; i < H; ++i) {
                        f1[i] = back(f1[i], m[i]);
                        f2[i] = back(f2[i], m[H + i]);
                    }
                } else {
                    const uint64_t minus = pair_of(-1.0f, -1.0f);
#pragma unroll
                    for (int i = 0; i < H; ++i) {
                        const uint64_t c = f1[i], d = f2[i];
                        f1[i] = mad2(c, m[i], mul2(d, m[H + i]));
                        f2[i] = mad2(mul2(c, m[H + i]), minus, mul2(d, m[i]));
                    }
                }
            }
            if (a.norm) {
                // Sums of x^2 and g w x; then dweight's share and dx.
                uint64_t xx = 0, gx = 0;
                if (norm1)
#pragma unroll
                    for (int i = 0; i < H; ++i) {
                        fma2(xx, g1[i], g1[i]);
                        fma2(gx, mul2(f1[i], w1[i]), g1[i]);
                    }
                if (norm2)
#pragma unroll
                    for (int i = 0; i < H; ++i) {
                        fma2(xx, g2[i], g2[i]);
                        fma2(gx, mul2(f2[i], w2[i]), g2[i]);
                    }
                const float2 sums = row_sums(make_float2(lower(xx) + upper(xx), lower(gx) + upper(gx)), L, meet, turns);
                const float r = rsqrtf(fmaf(sums.x, inv_norm, p.eps)), mean = sums.y * r * inv_norm;
                const uint64_t rr = pair_of(r, r), mm = pair_of(-mean, -mean);
                if (norm1)
#pragma unroll
                    for (int i = 0; i < H; ++i) {
                        const uint64_t z = mul2(g1[i], rr);
                        fma2(sw1[i], f1[i], z);
                        f1[i] = mul2(rr, mad2(z, mm, mul2(f1[i], w1[i])));
                    }
                if (norm2)
#pragma unroll
                    for (int i = 0; i < H; ++i) {
                        const uint64_t z = mul2(g2[i], rr);
                        fma2(sw2[i], f2[i], z);
                        f2[i] = mul2(rr, mad2(z, mm, mul2(f2[i], w2[i])));
                    }
            }
        }
        store(out + o1, has1 && live, f1);
        store(out + o2, has2 && live, f2);
        fresh = h + 1 == a.heads;
        out += fresh ? out_wrap : a.hsY;
        t += fresh;
        h = fresh ? 0 : h + 1;
    }
    if constexpr (kBackward) {
        if (!p.workspace || !a.norm || !a.dweight) return;
        // A warp's groups in a tree, then the warps one behind the other.
        float s1[V], s2[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            s1[i] = i & 1 ? upper(sw1[i / 2]) : lower(sw1[i / 2]);
            s2[i] = i & 1 ? upper(sw2[i / 2]) : lower(sw2[i / 2]);
            for (int o = L; o < 32; o <<= 1) {
                s1[i] += __shfl_xor_sync(~0u, s1[i], o);
                s2[i] += __shfl_xor_sync(~0u, s2[i], o);
            }
        }
        const int row_warps = max(1, L >> 5), sets = kVecThreads / 32 / row_warps;
        float* mine = dsum + warp / row_warps * a.norm;
        if ((threadIdx.x & 31) < L) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                if (norm1) mine[o1 + i] = s1[i];
                if (norm2) mine[o2 + i] = s2[i];
            }
        }
        __syncthreads();
        float* slot = p.workspace + (int64_t)blockIdx.x * plan.columns + q.column;
        for (int e = threadIdx.x; e < a.norm; e += kVecThreads) {
            float sum = dsum[e];
            for (int w = 1; w < sets; ++w) sum += dsum[w * a.norm + e];
            slot[e] = sum;
        }
    }
}

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
    *out = s.all();
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
    for (int i = 0; i < p.n_parts; ++i)      // (a warp's lanes hold 32 x 2 V elements at most: 16 KB in all)
        most = std::max(most, p.part[i].norm * (kVecThreads / 32 / std::max(1, (1 << plan.part[i].log_lanes) / 32)));
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
    // As many CTAs as are resident, so that a group has the angles of a token for all
    // the heads that it has of it; the arrays' shares by their rows' lanes, one at
    // least, which for the gradient all fit the partial sums' slots.  Forward, groups
    // that would have more than 16 rows take some 8, a part of a token or some tokens,
    // and the CTAs come in waves: 8192 tokens of 40 heads of 128 take 37 us so, 39 with
    // 16 rows each and 47 in one wave of 45.
    const int64_t slots = (int64_t)sms * (backward ? kGradBlocks : kForwardBlocks) - p.n_parts;
    int64_t blocks = 0;
    for (int i = 0; i < p.n_parts; ++i) {
        const RopePart& a = p.part[i];
        PartPlan& q = plan.part[i];
        const int64_t per = kVecThreads >> q.log_lanes, rows = p.tokens * a.heads;
        const int64_t share = std::max<int64_t>(1, (int64_t)((double)slots * (double)(rows << q.log_lanes) / (double)threads));
        int64_t span = (rows + share * per - 1) / (share * per);
        if (!backward && span > 16) {
            const int64_t pieces = (a.heads + 9) / 10;
            span = a.heads < 8 ? 8 / a.heads * a.heads : (a.heads + pieces - 1) / pieces;
        }
        if (span >= ((int64_t)1 << 31)) return false;
        q.span = (int)span;
        const int64_t mine = (rows + span * per - 1) / (span * per);
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
    // (Twice: the kernel of any alignment keeps what its sums' roundings lost.)
    return ((size_t)sms * kGradBlocks * (size_t)norm_total * 8 + 255) / 256 * 256;
}

unsigned int* status_word_norm_rope() { return word_address(&g_status); }

}  // namespace sbg
