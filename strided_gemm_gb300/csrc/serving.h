// Internal declarations of the 16-bit serving operators: the strided product,
// latent attention (paged and packed) and the page operations.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "internal.h"

namespace sbg {

// The 16-bit strided product (include/sbgemm.h, sbgemm_half); strides in elements.
struct HalfProblem {
    int type;                        // SBGEMM_TYPE_*
    const void* A; int64_t rsA, csA, bsA;
    const void* B; int64_t rsB, csB, bsB;
    void* C;       int64_t rsC, csC, bsC;
    int64_t M, N, K, batch;
    float alpha;
    int accumulate;
    ByteSpan sa, sb, sc;             // debug builds: what A, B and C occupy
};
// Any layout, on the CUDA cores (half_gather.cu).
cudaError_t launch_half_gather(const HalfProblem& p, cudaStream_t stream);
// On the tensor cores (half_tc.cu); false if the layout has no tensor maps.
bool launch_half_tc(const HalfProblem& p, int sms, cudaStream_t stream, cudaError_t* err);

// Latent attention over a paged cache (sbgemm_latent_attention_paged).
struct LatentPaged {
    int type;
    const void* Q; int64_t hsQ, tsQ, bsQ;
    const void* cache; int64_t rsC, psC, num_blocks, block_size;
    const int32_t* table; int64_t max_blocks;
    const int32_t* seq_lens;         // nullptr: N everywhere
    void* O; int64_t hsO, tsO, bsO;
    int64_t q_len, heads, N, R, P, n_seqs;
    float alpha;
    int causal;
    void* workspace; size_t workspace_bytes;
    ByteSpan sq, sc, so;             // debug builds: what Q, the cache and O occupy
};
// Latent attention over packed sequences (sbgemm_latent_attention).
struct LatentPacked {
    int type;
    const void* Q; int64_t hsQ, tsQ, total_q;
    const void* Kn; int64_t hsK, tsK;
    const void* Kr; int64_t tsR;
    const void* V; int64_t hsV, tsV, total_k;
    const int32_t* q_starts; const int32_t* k_starts;
    int64_t n_seqs, max_q;
    void* O; int64_t hsO, tsO;
    int64_t heads, Dn, P, Dv;
    float alpha;
    int causal;
    ByteSpan sq, sk, sr, sv, so;     // debug builds: what Q, K_nope, K_rope, V and O occupy
};
// On the tensor cores, over a paged cache (latent_decode.cu); false for sizes
// and alignments it does not take.
bool launch_latent_decode(const LatentPaged& a, int sms, cudaStream_t stream, cudaError_t* err);
size_t latent_decode_workspace_bytes(int sms);
// On the tensor cores, over packed sequences (latent_prompt.cu); false likewise.
bool launch_latent_prompt(const LatentPacked& a, cudaStream_t stream, cudaError_t* err);
// One warp a query row, any sizes and alignments (latent_rows.cu).
constexpr int64_t kLatentMaxQK = 640, kLatentMaxV = 512;
cudaError_t launch_latent_rows_paged(const LatentPaged& a, cudaStream_t stream);
cudaError_t launch_latent_rows_packed(const LatentPacked& a, cudaStream_t stream);

// Page operations (pages.cu).
struct PageCaches {
    int n;
    int64_t row_bytes[SBGEMM_MAX_CACHES];
    char* base[SBGEMM_MAX_CACHES];
};
struct PagePool {
    int64_t num_blocks, block_size;
    int32_t* refs;
    int32_t* table; int64_t n_seqs, max_blocks;
    int32_t* lens;
};
struct PageRows {                    // rows to append, per cache
    const char* base[SBGEMM_MAX_CACHES];
    int64_t stride[SBGEMM_MAX_CACHES];
};
size_t pages_workspace_bytes(int64_t num_blocks, int64_t n_seqs, int64_t n);
cudaError_t launch_pages_copy(const PageCaches& c, const PagePool& p, const int32_t* pairs, int64_t n, void* ws,
                              int sms, cudaStream_t stream);
cudaError_t launch_pages_fork(const PageCaches& c, const PagePool& p, const int32_t* parents,
                              const int32_t* children, int64_t n, void* ws, int sms, cudaStream_t stream);
cudaError_t launch_pages_append(const PageCaches& c, const PagePool& p, const int32_t* seqs, const int32_t* starts,
                                int64_t n, const PageRows& rows, int64_t total, void* ws, int sms,
                                cudaStream_t stream);
cudaError_t launch_pages_free(const PagePool& p, const int32_t* seqs, int64_t n, cudaStream_t stream);
cudaError_t launch_pages_compact(const PageCaches& c, const PagePool& p, int32_t* moved, void* ws, int sms,
                                 cudaStream_t stream);

}  // namespace sbg
