// The status words that kernels record codes in (bounded waits that gave up,
// inputs that were skipped), one a kernel file: read and cleared by one launch
// and one copy, whatever their number (a copy out and one in for each of 14
// words took 239 us on an idle GPU, this takes 22).
#include <mutex>

#include "internal.h"

namespace sbg {
namespace {

constexpr int kWords = 20;
struct Words { unsigned int* at[kWords]; };
__device__ unsigned int g_first;             // of the last launch

// One warp, a word a lane.  An exchange, so that no code recorded meanwhile by
// another stream's kernel is lost between a read and a store of 0.
__global__ void take_kernel(const Words w) {
    const unsigned int code = threadIdx.x < kWords ? atomicExch(w.at[threadIdx.x], 0u) : 0u;
    const unsigned int set = __ballot_sync(~0u, code != 0);
    const unsigned int first = __shfl_sync(~0u, code, set ? __ffs(set) - 1 : 0);
    if (threadIdx.x == 0) g_first = first;
}

}  // namespace

bool take_status_words(cudaStream_t stream, unsigned int* code) {
    static std::mutex one_at_a_time;         // g_first is every caller's
    const std::lock_guard<std::mutex> lock(one_at_a_time);
    const Words w{{status_word_tma_ffma_256x128(), status_word_tma_ffma_128x256(), status_word_tma_ffma_512x64(),
                   status_word_tf32(), status_word_selftest(), status_word_attention_tc(), status_word_gather(),
                   status_word_attention(), status_word_attention_decode(), status_word_half_gather(), status_word_half_tc(),
                   status_word_latent_decode(), status_word_latent_prompt(), status_word_latent_rows(),
                   status_word_pages(), status_word_latent_shared(), status_word_fp8_gather(), status_word_fp8_tc(),
                   status_word_fp8_quantize(), status_word_norm_rope()}};
    for (const unsigned int* at : w.at)
        if (!at) return false;
    take_kernel<<<1, 32, 0, stream>>>(w);
    return cudaGetLastError() == cudaSuccess &&
           cudaMemcpyFromSymbolAsync(code, g_first, sizeof(*code), 0, cudaMemcpyDeviceToHost, stream) == cudaSuccess &&
           cudaStreamSynchronize(stream) == cudaSuccess;
}

}  // namespace sbg
