// Latent attention for any sizes and alignments, one warp a query row, paged
// or packed (include/sbgemm.h).  One pass over the keys with the running
// maximum and sum of the softmax: lanes hold the row's query and output
// elements lane, lane + 32, ...; a key's score is a warp sum, and its weight
// scales the sums held so far only when the maximum rises.  Loads are scalar
// (2 bytes a lane) and every query row reads its keys again, which bounds it;
// the tensor-core kernels take the sizes they can.
#include <algorithm>

#include "debug_check.cuh"
#include "half_util.cuh"
#include "ptx.cuh"
#include "serving.h"

namespace sbg {
namespace {

constexpr int kWarps = 4;
constexpr int XQ = (int)kLatentMaxQK / 32, XV = (int)kLatentMaxV / 32;
__device__ unsigned int g_status = 0;

// Running softmax of one row over keys; `key(n, K, K2, V)` gives the key's nope
// part, rope part and value rows, or false for a row of zeros.  (No pointer
// says so: a part of no elements may lie anywhere, at address 0 too.)
// What the operands occupy, for the checks of debug builds.
struct Spans { ByteSpan q, k, r, v, o; };

template <typename T, typename Key>
__device__ __forceinline__ void attend_row(const T* q, int dn, int dr, int dv, int64_t keys, float scale_log2,
                                           T* o, const Spans& in, Key key) {
    auto load = [](const T* x, const ByteSpan& span) {
        return dbg_in_bytes(x, sizeof(T), span, &g_status) ? to_float(*x) : 0.0f;
    };
    const int lane = threadIdx.x & 31;
    float qf[XQ], acc[XV];
#pragma unroll
    for (int x = 0; x < XQ; ++x) qf[x] = lane + 32 * x < dn + dr ? load(q + lane + 32 * x, in.q) : 0.0f;
#pragma unroll
    for (int x = 0; x < XV; ++x) acc[x] = 0.0f;
    float top = -INFINITY, sum = 0.0f;
    for (int64_t n = 0; n < keys; ++n) {
        const T *kn, *kr, *v;
        const bool there = key(n, &kn, &kr, &v);
        float z = 0.0f;
        if (there) {
#pragma unroll
            for (int x = 0; x < XQ; ++x) {
                const int d = lane + 32 * x;
                if (d < dn + dr) z = fmaf(qf[x], d < dn ? load(kn + d, in.k) : load(kr + (d - dn), in.r), z);
            }
        }
#pragma unroll
        for (int s = 16; s; s >>= 1) z += __shfl_xor_sync(~0u, z, s);
        z *= scale_log2;
        if (z > top) {
            const float f = exp2f(top - z);      // 0 for the first key
            sum *= f;
#pragma unroll
            for (int x = 0; x < XV; ++x) acc[x] *= f;
            top = z;
        }
        // A score of -infinity weighs nothing, also as the first one.
        const float w = z == -INFINITY ? 0.0f : exp2f(z - top);
        sum += w;
        if (there) {
#pragma unroll
            for (int x = 0; x < XV; ++x)
                if (lane + 32 * x < dv) acc[x] = fmaf(w, load(v + lane + 32 * x, in.v), acc[x]);
        }
    }
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;   // no key: zeros
#pragma unroll
    for (int x = 0; x < XV; ++x)
        if (lane + 32 * x < dv && dbg_in_bytes(o + lane + 32 * x, sizeof(T), in.o, &g_status))
            o[lane + 32 * x] = from_float<T>(acc[x] * inv);
}

template <typename T>
__global__ void __launch_bounds__(kWarps * 32)
rows_paged_kernel(const LatentPaged a, float scale_log2) {
    const int64_t rows = a.n_seqs * a.q_len * a.heads;
    for (int64_t r = (int64_t)blockIdx.x * kWarps + threadIdx.x / 32; r < rows; r += (int64_t)gridDim.x * kWarps) {
        const int64_t h = r % a.heads, t = r / a.heads % a.q_len, s = r / a.heads / a.q_len;
        int64_t len = a.seq_lens ? a.seq_lens[s] : a.N;
        if (len < 0 || len > a.N) {
            record_status(&g_status, kPagedInput);
            len = len < 0 ? 0 : a.N;
        }
        const int64_t keys = a.causal ? min(len, max((int64_t)0, len - a.q_len + t + 1)) : len;
        const T* base = static_cast<const T*>(a.cache);
        attend_row<T>(static_cast<const T*>(a.Q) + s * a.bsQ + t * a.tsQ + h * a.hsQ, (int)a.R, (int)a.P, (int)a.R,
                      keys, scale_log2, static_cast<T*>(a.O) + s * a.bsO + t * a.tsO + h * a.hsO,
                      Spans{a.sq, a.sc, a.sc, a.sc, a.so},
                      [&](int64_t n, const T** kn, const T** kr, const T** v) {
                          const int64_t page = a.table[s * a.max_blocks + n / a.block_size];
                          if (page < 0 || page >= a.num_blocks) {
                              record_status(&g_status, kPagedInput);
                              return false;
                          }
                          *kn = *v = base + page * a.psC + n % a.block_size * a.rsC;
                          *kr = *kn + a.R;
                          return true;
                      });
    }
}

template <typename T>
__global__ void __launch_bounds__(kWarps * 32)
rows_shared_kernel(const __grid_constant__ LatentShared g, float scale_log2) {
    const LatentPaged& a = g.paged;
    const int64_t rows = a.n_seqs * a.q_len * a.heads;
    for (int64_t r = (int64_t)blockIdx.x * kWarps + threadIdx.x / 32; r < rows; r += (int64_t)gridDim.x * kWarps) {
        const int64_t h = r % a.heads, t = r / a.heads % a.q_len, s = r / a.heads / a.q_len;
        int64_t len = a.seq_lens ? a.seq_lens[s] : a.N;
        len = min(max(len, (int64_t)0), a.N);            // (reported by the plan)
        const int64_t keys = a.causal ? min(len, max((int64_t)0, len - a.q_len + t + 1)) : len;
        const int64_t first = g.first[s], prefix = g.prefix[s];
        const T* base = static_cast<const T*>(a.cache);
        attend_row<T>(static_cast<const T*>(a.Q) + s * a.bsQ + t * a.tsQ + h * a.hsQ, (int)a.R, (int)a.P, (int)a.R,
                      keys, scale_log2, static_cast<T*>(a.O) + s * a.bsO + t * a.tsO + h * a.hsO,
                      Spans{a.sq, a.sc, a.sc, a.sc, a.so},
                      [&](int64_t n, const T** kn, const T** kr, const T** v) {
                          const int64_t page = a.table[(n < prefix ? first : s) * a.max_blocks + n / a.block_size];
                          if (page < 0 || page >= a.num_blocks) {
                              record_status(&g_status, kPagedInput);
                              return false;
                          }
                          *kn = *v = base + page * a.psC + n % a.block_size * a.rsC;
                          *kr = *kn + a.R;
                          return true;
                      });
    }
}

// starts[s], starts[s + 1] as a range inside [0, total], reported when they are not.
__device__ __forceinline__ void packed_range(const int32_t* starts, int64_t s, int64_t total, int64_t most,
                                             int64_t* lo, int64_t* n) {
    const int64_t a = starts[s], b = starts[s + 1];
    const int64_t x = min(max(a, (int64_t)0), total), y = min(max(b, x), total);
    *lo = x;
    *n = min(y - x, most);
    if (a != x || b != y || *n != y - x) record_status(&g_status, kPagedInput);
}

template <typename T>
__global__ void __launch_bounds__(kWarps * 32)
rows_packed_kernel(const LatentPacked a, float scale_log2) {
    const int64_t s = blockIdx.y;
    int64_t q0, nq, k0, nk;
    packed_range(a.q_starts, s, a.total_q, a.max_q, &q0, &nq);
    packed_range(a.k_starts, s, a.total_k, a.total_k, &k0, &nk);
    for (int64_t r = (int64_t)blockIdx.x * kWarps + threadIdx.x / 32; r < nq * a.heads;
         r += (int64_t)gridDim.x * kWarps) {
        const int64_t h = r % a.heads, i = r / a.heads;
        const int64_t keys = a.causal ? min(nk, max((int64_t)0, nk - nq + i + 1)) : nk;
        attend_row<T>(static_cast<const T*>(a.Q) + (q0 + i) * a.tsQ + h * a.hsQ, (int)a.Dn, (int)a.P, (int)a.Dv,
                      keys, scale_log2, static_cast<T*>(a.O) + (q0 + i) * a.tsO + h * a.hsO,
                      Spans{a.sq, a.sk, a.sr, a.sv, a.so},
                      [&](int64_t n, const T** kn, const T** kr, const T** v) {
                          *kn = static_cast<const T*>(a.Kn) + (k0 + n) * a.tsK + h * a.hsK;
                          *kr = static_cast<const T*>(a.Kr) + (k0 + n) * a.tsR;
                          *v = static_cast<const T*>(a.V) + (k0 + n) * a.tsV + h * a.hsV;
                          return true;
                      });
    }
}

}  // namespace

cudaError_t launch_latent_rows_paged(const LatentPaged& a, cudaStream_t stream) {
    const int64_t rows = a.n_seqs * a.q_len * a.heads;
    const unsigned grid = (unsigned)std::min<int64_t>((rows + kWarps - 1) / kWarps, 1 << 20);
    const float scale = a.alpha * 1.4426950408889634f;
    if (a.type == SBGEMM_TYPE_BF16) rows_paged_kernel<__nv_bfloat16><<<grid, kWarps * 32, 0, stream>>>(a, scale);
    else rows_paged_kernel<__half><<<grid, kWarps * 32, 0, stream>>>(a, scale);
    return cudaGetLastError();
}

cudaError_t launch_latent_rows_shared(const LatentShared& g, cudaStream_t stream) {
    const int64_t rows = g.paged.n_seqs * g.paged.q_len * g.paged.heads;
    const unsigned grid = (unsigned)std::min<int64_t>((rows + kWarps - 1) / kWarps, 1 << 20);
    const float scale = g.paged.alpha * 1.4426950408889634f;
    if (g.paged.type == SBGEMM_TYPE_BF16) rows_shared_kernel<__nv_bfloat16><<<grid, kWarps * 32, 0, stream>>>(g, scale);
    else rows_shared_kernel<__half><<<grid, kWarps * 32, 0, stream>>>(g, scale);
    return cudaGetLastError();
}

cudaError_t launch_latent_rows_packed(const LatentPacked& a, cudaStream_t stream) {
    const int64_t rows = std::min(a.max_q, a.total_q) * a.heads;
    const dim3 grid((unsigned)std::min<int64_t>((rows + kWarps - 1) / kWarps, 1 << 16), (unsigned)a.n_seqs);
    const float scale = a.alpha * 1.4426950408889634f;
    if (a.type == SBGEMM_TYPE_BF16) rows_packed_kernel<__nv_bfloat16><<<grid, kWarps * 32, 0, stream>>>(a, scale);
    else rows_packed_kernel<__half><<<grid, kWarps * 32, 0, stream>>>(a, scale);
    return cudaGetLastError();
}

unsigned int* status_word_latent_rows() { return word_address(&g_status); }

}  // namespace sbg
