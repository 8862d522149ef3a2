// Latent attention over a paged cache for groups of sequences with a shared
// prefix (sbgemm_latent_attention_shared).
//
// plan_kernel turns the groups into two numbers for each sequence: where the
// keys below `prefix` are found (the table row of the group's first sequence),
// and that prefix.  Starts are taken as a running maximum of their values
// clamped to [0, n_seqs], so that every kernel sees the same, sound groups
// whatever stands in device memory; what was clamped is reported here.
#include <algorithm>

#include "debug_check.cuh"
#include "serving.h"

namespace sbg {
namespace {

__device__ unsigned int g_status = 0;
constexpr int kPlanThreads = 1024;

__device__ __forceinline__ int clamped(int v, int lo, int hi) {
    const int c = min(max(v, lo), hi);
    if (c != v) record_status(&g_status, kPagedInput);
    return c;
}

__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const __grid_constant__ LatentShared g) {
    __shared__ int tops[kPlanThreads / 32];
    __shared__ int so_far;
    const LatentPaged& a = g.paged;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, n_seqs = (int)a.n_seqs;
    auto length = [&](int s) { return a.seq_lens ? clamped(a.seq_lens[s], 0, (int)a.N) : (int)a.N; };
    auto put = [&](int s, int first, int prefix) {
        if (dbg_in_bytes(g.first + s, 4, g.sw, &g_status)) g.first[s] = first;
        if (dbg_in_bytes(g.prefix + s, 4, g.sw, &g_status)) g.prefix[s] = prefix;
    };
    for (int s = tid; s < n_seqs; s += kPlanThreads) {
        length(s);                                       // reports every length
        put(s, s, 0);
    }
    if (tid == 0) so_far = 0;
    __syncthreads();
    for (int64_t g0 = 0; g0 < g.n_groups; g0 += kPlanThreads) {
        // This thread's group, from the running maximum up to its start to that
        // up to the next one's.
        const int64_t i = g0 + tid;
        const bool mine = i < g.n_groups;
        const int at = mine ? clamped(g.group_starts[i], 0, n_seqs) : 0;
        const int next = mine ? clamped(g.group_starts[i + 1], 0, n_seqs) : 0;
        int top = at;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(~0u, top, o);
            if (lane >= o) top = max(top, x);
        }
        if (lane == 31) tops[warp] = top;
        __syncthreads();
        int lo = max(so_far, top);
        for (int w = 0; w < warp; ++w) lo = max(lo, tops[w]);
        const int hi = max(lo, next);
        if (mine && (lo != at || hi != next)) record_status(&g_status, kPagedInput);
        __syncthreads();
        if (tid == kPlanThreads - 1) so_far = lo;
        if (mine && lo < hi) {
            const int prefix = clamped(g.prefix_lens[i], 0, min((int)a.N, length(lo)));
            for (int s = lo; s < hi; ++s) put(s, lo, prefix);
        } else if (mine && g.prefix_lens[i] < 0) {
            record_status(&g_status, kPagedInput);
        }
        __syncthreads();
    }
}

size_t round256(size_t n) { return (n + 255) / 256 * 256; }

}  // namespace

size_t latent_shared_workspace_bytes(int sms, int64_t n_seqs, int64_t n_groups, int64_t q_len, int64_t heads, int64_t R) {
    (void)sms; (void)n_groups; (void)q_len; (void)heads; (void)R;
    return 2 * round256((size_t)n_seqs * 4);
}

cudaError_t launch_latent_shared(const LatentPaged& a, const int32_t* group_starts, const int32_t* prefix_lens,
                                 int64_t n_groups, int sms, cudaStream_t stream) {
    (void)sms;
    char* ws = static_cast<char*>(a.workspace);
    const size_t each = round256((size_t)a.n_seqs * 4);
    LatentShared g{a, group_starts, prefix_lens, n_groups, reinterpret_cast<int32_t*>(ws),
                   reinterpret_cast<int32_t*>(ws + each), ws + 2 * each, a.workspace_bytes - 2 * each,
                   ByteSpan{(uintptr_t)ws, (uintptr_t)ws + a.workspace_bytes}};
    plan_kernel<<<1, kPlanThreads, 0, stream>>>(g);
    if (const cudaError_t e = cudaGetLastError()) return e;
    return launch_latent_rows_shared(g, stream);
}

unsigned int* status_word_latent_shared() { return word_address(&g_status); }

}  // namespace sbg
