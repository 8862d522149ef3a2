// C-ABI boundary of the 16-bit serving operators: argument validation and
// dispatch.  As for the fp32 product, every size a kernel depends on is checked
// before a launch (the StaleyNET "GPU Implementation" page, section "Safety"),
// so that no access leaves what the caller described; what stands in device
// memory (block tables, lengths, page requests) is checked by the kernels.
#include <cuda_runtime.h>

#include <algorithm>
#include <array>
#include <initializer_list>

#include "api_checks.h"
#include "sbgemm.h"
#include "serving.h"

namespace sbg {
namespace {

bool known_type(int type) { return type == SBGEMM_TYPE_BF16 || type == SBGEMM_TYPE_FP16; }

// ---- the pool ------------------------------------------------------------------

// Checks a pool and lays it out for the kernels; `books` asks for the
// bookkeeping arrays.  *spans receives what the caches and arrays occupy.
struct PoolView {
    PageCaches caches;
    PagePool pool;
    std::array<Bytes, SBGEMM_MAX_CACHES + 3> spans;
    size_t n_spans;
};

int read_pool(const sbgemm_page_pool* in, bool books, PoolView* v) {
    if (!in) return SBGEMM_ERR_NULL_POINTER;
    if (in->n_caches < 0 || in->n_caches > SBGEMM_MAX_CACHES) return SBGEMM_ERR_INVALID_VALUE;
    if (in->num_blocks <= 0 || in->num_blocks >= kInt / 2 || in->block_size <= 0 || in->block_size > kInt)
        return SBGEMM_ERR_INVALID_VALUE;
    if (in->n_caches > 0 && (!in->caches || !in->page_bytes)) return SBGEMM_ERR_NULL_POINTER;
    v->n_spans = 0;
    v->caches.n = (int)in->n_caches;
    for (int64_t i = 0; i < in->n_caches; ++i) {
        const int64_t pb = in->page_bytes[i];
        if (!in->caches[i]) return SBGEMM_ERR_NULL_POINTER;
        if (pb <= 0 || pb % in->block_size != 0 || pb / in->block_size % 16 != 0 || !aligned(in->caches[i], 16))
            return SBGEMM_ERR_INVALID_VALUE;
        if ((i128)pb * in->num_blocks >= (i128)1 << 60) return SBGEMM_ERR_INVALID_VALUE;
        v->caches.base[i] = static_cast<char*>(in->caches[i]);
        v->caches.row_bytes[i] = pb / in->block_size;
        const Bytes s = block(in->caches[i], pb * in->num_blocks);
        for (size_t j = 0; j < v->n_spans; ++j)
            if (meet(s, v->spans[j])) return SBGEMM_ERR_OUTPUT_OVERLAP;
        v->spans[v->n_spans++] = s;
    }
    v->pool = PagePool{in->num_blocks, in->block_size, nullptr, nullptr, 0, 0, nullptr};
    if (books) {
        if (in->n_seqs <= 0 || in->n_seqs >= kInt / 2 || in->max_blocks <= 0 || in->max_blocks >= kInt ||
            (i128)in->n_seqs * in->max_blocks >= (i128)1 << 40)
            return SBGEMM_ERR_INVALID_VALUE;
        if (!in->ref_counts || !in->block_table || !in->seq_lens) return SBGEMM_ERR_NULL_POINTER;
        if (!aligned(in->ref_counts, 4) || !aligned(in->block_table, 4) || !aligned(in->seq_lens, 4))
            return SBGEMM_ERR_INVALID_VALUE;
        v->pool.refs = in->ref_counts;
        v->pool.table = in->block_table;
        v->pool.n_seqs = in->n_seqs;
        v->pool.max_blocks = in->max_blocks;
        v->pool.lens = in->seq_lens;
        const Bytes arrays[3] = {block(in->ref_counts, in->num_blocks * 4),
                                 block(in->block_table, in->n_seqs * in->max_blocks * 4),
                                 block(in->seq_lens, in->n_seqs * 4)};
        for (const Bytes& s : arrays) {
            for (size_t j = 0; j < v->n_spans; ++j)
                if (meet(s, v->spans[j])) return SBGEMM_ERR_OUTPUT_OVERLAP;
            v->spans[v->n_spans++] = s;
        }
    }
    return SBGEMM_OK;
}

// Inputs that no pool array may meet, the workspace (`need` bytes of it) that
// may meet nothing, and all of them in device memory.
int check_pool_memory(const PoolView& v, std::initializer_list<Bytes> inputs, const sbgemm_options* opt,
                      size_t need, void** ws) {
    size_t bytes = 0;
    const int st = read_options(opt, ws, &bytes);
    if (st) return st;
    if (need && (!*ws || bytes < need)) return SBGEMM_ERR_INVALID_VALUE;
    const Bytes w = block(*ws, need ? (int64_t)need : 0);
    for (size_t j = 0; j < v.n_spans; ++j) {
        for (const Bytes& in : inputs)
            if (meet(in, v.spans[j])) return SBGEMM_ERR_OUTPUT_OVERLAP;
        if (need && meet(w, v.spans[j])) return SBGEMM_ERR_OUTPUT_OVERLAP;
    }
    if (need)
        for (const Bytes& in : inputs)
            if (meet(in, w)) return SBGEMM_ERR_OUTPUT_OVERLAP;
    for (size_t j = 0; j < v.n_spans; ++j)
        if (const int m = in_device_memory({v.spans[j]})) return m;
    if (const int m = in_device_memory(inputs)) return m;
    if (need)
        if (const int m = in_device_memory({w})) return m;
    return SBGEMM_OK;
}

// The arguments that sbgemm_latent_attention_paged and _shared have in common:
// checked, and laid out in *a, with the operands' bytes (Q, cache, O, table,
// lengths) in *spans.  *empty: there is nothing to do.
int check_latent_paged(
    int type, const void* Q, int64_t hsQ, int64_t tsQ, int64_t bsQ,
    const void* cache, int64_t rsC, int64_t psC, int64_t num_blocks, int64_t block_size,
    const int32_t* block_table, int64_t max_blocks, const int32_t* seq_lens,
    void* O, int64_t hsO, int64_t tsO, int64_t bsO,
    int64_t q_len, int64_t heads, int64_t N, int64_t R, int64_t P, int64_t n_seqs,
    float alpha, int causal, const sbgemm_options* opt, LatentPaged* a, std::array<Bytes, 5>* spans, bool* empty) {
    *empty = false;
    void* ws = nullptr;
    size_t ws_bytes = 0;
    if (const int st = read_options(opt, &ws, &ws_bytes)) return st;
    if (!known_type(type)) return SBGEMM_ERR_INVALID_VALUE;
    if (q_len < 0 || heads < 0 || N < 0 || R < 0 || P < 0 || n_seqs < 0) return SBGEMM_ERR_INVALID_VALUE;
    if (causal != 0 && causal != 1) return SBGEMM_ERR_INVALID_VALUE;
    if (q_len == 0 || heads == 0 || n_seqs == 0 || R == 0) {
        *empty = true;
        return SBGEMM_OK;
    }
    if (num_blocks <= 0 || num_blocks >= kInt || block_size <= 0 || max_blocks <= 0)
        return SBGEMM_ERR_INVALID_VALUE;
    if ((i128)max_blocks * block_size < (i128)N) return SBGEMM_ERR_INVALID_VALUE;
    if (R > kLatentMaxV || R + P > kLatentMaxQK) return SBGEMM_ERR_UNSUPPORTED;
    // (A block of keys beyond the last one still has an int for its index.)
    if (q_len >= kInt || heads >= kInt || N > kInt - 64 || n_seqs >= kInt || block_size >= kInt ||
        (i128)q_len * heads >= kInt || (i128)q_len * heads * n_seqs >= kInt)
        return SBGEMM_ERR_UNSUPPORTED;
    if (!Q || !cache || !block_table || !O) return SBGEMM_ERR_NULL_POINTER;
    if (!aligned(Q, 2) || !aligned(cache, 2) || !aligned(O, 2) || !aligned(block_table, 4) ||
        (seq_lens && !aligned(seq_lens, 4)))
        return SBGEMM_ERR_INVALID_VALUE;
    Bytes sq{}, sc{}, so{}, st{};
    if (!span_of(Q, 2, {{bsQ, n_seqs}, {tsQ, q_len}, {hsQ, heads}, {1, R + P}}, &sq) ||
        !span_of(cache, 2, {{psC, num_blocks}, {rsC, block_size}, {1, R + P}}, &sc) ||
        !span_of(O, 2, {{bsO, n_seqs}, {tsO, q_len}, {hsO, heads}, {1, R}}, &so) ||
        !span_of(block_table, 4, {{max_blocks, n_seqs}, {1, max_blocks}}, &st))
        return SBGEMM_ERR_INVALID_VALUE;
    const Bytes sl = seq_lens ? block(seq_lens, n_seqs * 4) : st;
    if (!injective(std::array<Axis, 4>{{{bsO, n_seqs}, {tsO, q_len}, {hsO, heads}, {1, R}}}))
        return SBGEMM_ERR_OUTPUT_OVERLAP;
    for (const Bytes& s : {sq, sc, st, sl})
        if (meet(so, s)) return SBGEMM_ERR_OUTPUT_OVERLAP;
    *a = LatentPaged{type, Q, hsQ, tsQ, bsQ, cache, rsC, psC, num_blocks, block_size, block_table, max_blocks,
                     seq_lens, O, hsO, tsO, bsO, q_len, heads, N, R, P, n_seqs, alpha, causal, ws, ws_bytes,
                     span_for_kernel(sq), span_for_kernel(sc), span_for_kernel(so)};
    *spans = {sq, sc, so, st, sl};
    return SBGEMM_OK;
}

}  // namespace

}  // namespace sbg

using namespace sbg;

extern "C" {

int sbgemm_half(int type, const void* A, int64_t rsA, int64_t csA, int64_t bsA,
                const void* B, int64_t rsB, int64_t csB, int64_t bsB,
                void* C, int64_t rsC, int64_t csC, int64_t bsC,
                int64_t M, int64_t N, int64_t K, int64_t batch,
                float alpha, int accumulate, void* stream) {
    if (!known_type(type)) return SBGEMM_ERR_INVALID_VALUE;
    if (M < 0 || N < 0 || K < 0 || batch < 0) return SBGEMM_ERR_INVALID_VALUE;
    if (M == 0 || N == 0 || batch == 0) return SBGEMM_OK;
    if (!C || (K > 0 && (!A || !B))) return SBGEMM_ERR_NULL_POINTER;
    if (!aligned(C, 2) || (K > 0 && (!aligned(A, 2) || !aligned(B, 2)))) return SBGEMM_ERR_INVALID_VALUE;
    Bytes sa{}, sb{}, sc{};
    if (!span_of(C, 2, {{bsC, batch}, {rsC, M}, {csC, N}}, &sc)) return SBGEMM_ERR_INVALID_VALUE;
    if (K > 0 && (!span_of(A, 2, {{bsA, batch}, {rsA, M}, {csA, K}}, &sa) ||
                  !span_of(B, 2, {{bsB, batch}, {rsB, K}, {csB, N}}, &sb)))
        return SBGEMM_ERR_INVALID_VALUE;
    if (!injective(std::array<Axis, 3>{{{bsC, batch}, {rsC, M}, {csC, N}}})) return SBGEMM_ERR_OUTPUT_OVERLAP;
    if (K > 0 && (meet(sc, sa) || meet(sc, sb))) return SBGEMM_ERR_OUTPUT_OVERLAP;
    if (K == 0 && accumulate) return SBGEMM_OK;
    const int64_t tiles = ((M + 63) / 64) * ((N + 63) / 64);
    if (M >= kInt || N >= kInt || K >= kInt || tiles >= kInt) return SBGEMM_ERR_UNSUPPORTED;
    const int sms = current_sms();
    if (!sms) return SBGEMM_ERR_CUDA;
    const int m = K > 0 ? in_device_memory({sa, sb, sc}) : in_device_memory({sc});
    if (m) return m;
    const HalfProblem p{type, A, rsA, csA, bsA, B, rsB, csB, bsB, C, rsC, csC, bsC,
                        M, N, K, batch, alpha, accumulate, span_for_kernel(sa), span_for_kernel(sb), span_for_kernel(sc)};
    cudaError_t e = cudaSuccess;
    if (launch_half_tc(p, sms, static_cast<cudaStream_t>(stream), &e)) return finish(e);
    return finish(launch_half_gather(p, static_cast<cudaStream_t>(stream)));
}

int sbgemm_latent_attention_paged(
    int type, const void* Q, int64_t hsQ, int64_t tsQ, int64_t bsQ,
    const void* cache, int64_t rsC, int64_t psC, int64_t num_blocks, int64_t block_size,
    const int32_t* block_table, int64_t max_blocks, const int32_t* seq_lens,
    void* O, int64_t hsO, int64_t tsO, int64_t bsO,
    int64_t q_len, int64_t heads, int64_t N, int64_t R, int64_t P, int64_t n_seqs,
    float alpha, int causal, void* stream, const sbgemm_options* opt) {
    LatentPaged a{};
    std::array<Bytes, 5> spans;
    bool empty = false;
    if (const int st = check_latent_paged(type, Q, hsQ, tsQ, bsQ, cache, rsC, psC, num_blocks, block_size, block_table,
                                          max_blocks, seq_lens, O, hsO, tsO, bsO, q_len, heads, N, R, P, n_seqs, alpha,
                                          causal, opt, &a, &spans, &empty))
        return st;
    if (empty) return SBGEMM_OK;
    const int sms = current_sms();
    if (!sms) return SBGEMM_ERR_CUDA;
    if (const int m = in_device_memory({spans[0], spans[1], spans[2], spans[3], spans[4]})) return m;
    if (a.workspace) {
        const Bytes w = block(a.workspace, (int64_t)std::min<size_t>(a.workspace_bytes, (size_t)1 << 60));
        for (const Bytes& s : spans)
            if (meet(w, s)) return SBGEMM_ERR_OUTPUT_OVERLAP;
        if (a.workspace_bytes == 0) a.workspace = nullptr;
        else if (const int m = in_device_memory({w})) return m;
    }
    cudaError_t e = cudaSuccess;
    if (launch_latent_decode(a, sms, static_cast<cudaStream_t>(stream), &e)) return finish(e);
    return finish(launch_latent_rows_paged(a, static_cast<cudaStream_t>(stream)));
}

int sbgemm_latent_attention_shared(
    int type, const void* Q, int64_t hsQ, int64_t tsQ, int64_t bsQ,
    const void* cache, int64_t rsC, int64_t psC, int64_t num_blocks, int64_t block_size,
    const int32_t* block_table, int64_t max_blocks, const int32_t* seq_lens,
    const int32_t* group_starts, const int32_t* prefix_lens, int64_t n_groups,
    void* O, int64_t hsO, int64_t tsO, int64_t bsO,
    int64_t q_len, int64_t heads, int64_t N, int64_t R, int64_t P, int64_t n_seqs,
    float alpha, int causal, void* stream, const sbgemm_options* opt) {
    LatentPaged a{};
    std::array<Bytes, 5> spans;
    bool empty = false;
    if (n_groups < 0) return SBGEMM_ERR_INVALID_VALUE;
    if (const int st = check_latent_paged(type, Q, hsQ, tsQ, bsQ, cache, rsC, psC, num_blocks, block_size, block_table,
                                          max_blocks, seq_lens, O, hsO, tsO, bsO, q_len, heads, N, R, P, n_seqs, alpha,
                                          causal, opt, &a, &spans, &empty))
        return st;
    if (empty) return SBGEMM_OK;
    if (n_groups >= kInt / 2) return SBGEMM_ERR_UNSUPPORTED;
    if (n_groups > 0 && (!group_starts || !prefix_lens)) return SBGEMM_ERR_NULL_POINTER;
    if (!aligned(group_starts, 4) || !aligned(prefix_lens, 4)) return SBGEMM_ERR_INVALID_VALUE;
    // (Without groups nothing of theirs is read.)
    const Bytes s0 = n_groups ? block(group_starts, (n_groups + 1) * 4) : spans[3];
    const Bytes s1 = n_groups ? block(prefix_lens, n_groups * 4) : spans[3];
    if (meet(spans[2], s0) || meet(spans[2], s1)) return SBGEMM_ERR_OUTPUT_OVERLAP;
    const int sms = current_sms();
    if (!sms) return SBGEMM_ERR_CUDA;
    const size_t need = latent_shared_workspace_bytes(sms, n_seqs, n_groups, q_len, heads, R);
    if (!a.workspace || a.workspace_bytes < need) return SBGEMM_ERR_INVALID_VALUE;
    a.workspace_bytes = need;
    const Bytes w = block(a.workspace, (int64_t)need);
    for (const Bytes& s : {spans[0], spans[1], spans[2], spans[3], spans[4], s0, s1})
        if (meet(w, s)) return SBGEMM_ERR_OUTPUT_OVERLAP;
    if (const int m = in_device_memory({spans[0], spans[1], spans[2], spans[3], spans[4], s0, s1, w})) return m;
    return finish(launch_latent_shared(a, group_starts, prefix_lens, n_groups, sms, static_cast<cudaStream_t>(stream)));
}

int sbgemm_latent_shared_workspace_bytes(int device, int64_t n_seqs, int64_t n_groups, int64_t q_len, int64_t heads,
                                         int64_t R, size_t* bytes) {
    if (!bytes) return SBGEMM_ERR_NULL_POINTER;
    if (n_seqs < 0 || n_groups < 0 || q_len < 0 || heads < 0 || R < 0) return SBGEMM_ERR_INVALID_VALUE;
    if (n_seqs >= kInt || n_groups >= kInt / 2 || q_len >= kInt || heads >= kInt || R > kLatentMaxV ||
        (i128)q_len * heads >= kInt || (i128)q_len * heads * n_seqs >= kInt)
        return SBGEMM_ERR_UNSUPPORTED;
    const DeviceProps* d = device_props(device);
    if (!d) {
        cudaGetLastError();
        return SBGEMM_ERR_CUDA;
    }
    *bytes = latent_shared_workspace_bytes(d->sm_count, n_seqs, n_groups, q_len, heads, R);
    return SBGEMM_OK;
}

int sbgemm_latent_workspace_bytes(int device, size_t* bytes) {
    if (!bytes) return SBGEMM_ERR_NULL_POINTER;
    const DeviceProps* d = device_props(device);
    if (!d) {
        cudaGetLastError();
        return SBGEMM_ERR_CUDA;
    }
    *bytes = latent_decode_workspace_bytes(d->sm_count);
    return SBGEMM_OK;
}

int sbgemm_latent_attention(
    int type, const void* Q, int64_t hsQ, int64_t tsQ, int64_t total_q,
    const void* K_nope, int64_t hsK, int64_t tsK, const void* K_rope, int64_t tsR,
    const void* V, int64_t hsV, int64_t tsV, int64_t total_k,
    const int32_t* q_starts, const int32_t* k_starts, int64_t n_seqs, int64_t max_q,
    void* O, int64_t hsO, int64_t tsO,
    int64_t heads, int64_t Dn, int64_t P, int64_t Dv, float alpha, int causal, void* stream) {
    if (!known_type(type)) return SBGEMM_ERR_INVALID_VALUE;
    if (total_q < 0 || total_k < 0 || n_seqs < 0 || max_q < 0 || heads < 0 || Dn < 0 || P < 0 || Dv < 0)
        return SBGEMM_ERR_INVALID_VALUE;
    if (causal != 0 && causal != 1) return SBGEMM_ERR_INVALID_VALUE;
    if (total_q == 0 || n_seqs == 0 || max_q == 0 || heads == 0 || Dv == 0) return SBGEMM_OK;
    if (Dn + P == 0) return SBGEMM_ERR_INVALID_VALUE;
    if (Dn + P > kLatentMaxQK || Dv > kLatentMaxV) return SBGEMM_ERR_UNSUPPORTED;
    if (total_q >= kInt || total_k >= kInt || max_q >= kInt || n_seqs > 65535 || heads > 65535 ||
        (i128)total_q * heads >= (i128)1 << 40)
        return SBGEMM_ERR_UNSUPPORTED;
    const bool keys = total_k > 0;
    if (!Q || !O || !q_starts || !k_starts || (keys && ((Dn > 0 && !K_nope) || (P > 0 && !K_rope) || !V)))
        return SBGEMM_ERR_NULL_POINTER;
    if (!aligned(Q, 2) || !aligned(O, 2) || !aligned(K_nope, 2) || !aligned(K_rope, 2) || !aligned(V, 2) ||
        !aligned(q_starts, 4) || !aligned(k_starts, 4))
        return SBGEMM_ERR_INVALID_VALUE;
    Bytes sq{}, sk{}, sr{}, sv{}, so{};
    if (!span_of(Q, 2, {{tsQ, total_q}, {hsQ, heads}, {1, Dn + P}}, &sq) ||
        !span_of(O, 2, {{tsO, total_q}, {hsO, heads}, {1, Dv}}, &so))
        return SBGEMM_ERR_INVALID_VALUE;
    sk = sr = sv = sq;                       // operands that are not read: nothing of their own
    if (keys && ((Dn > 0 && !span_of(K_nope, 2, {{tsK, total_k}, {hsK, heads}, {1, Dn}}, &sk)) ||
                 (P > 0 && !span_of(K_rope, 2, {{tsR, total_k}, {1, P}}, &sr)) ||
                 !span_of(V, 2, {{tsV, total_k}, {hsV, heads}, {1, Dv}}, &sv)))
        return SBGEMM_ERR_INVALID_VALUE;
    if (!injective(std::array<Axis, 3>{{{tsO, total_q}, {hsO, heads}, {1, Dv}}})) return SBGEMM_ERR_OUTPUT_OVERLAP;
    const Bytes s0 = block(q_starts, (n_seqs + 1) * 4), s1 = block(k_starts, (n_seqs + 1) * 4);
    for (const Bytes& s : {sq, sk, sr, sv, s0, s1})
        if (meet(so, s)) return SBGEMM_ERR_OUTPUT_OVERLAP;
    if (!current_sms()) return SBGEMM_ERR_CUDA;
    if (const int m = in_device_memory({sq, sk, sr, sv, so, s0, s1})) return m;
    const LatentPacked a{type, Q, hsQ, tsQ, total_q, K_nope, hsK, tsK, K_rope, tsR, V, hsV, tsV, total_k,
                         q_starts, k_starts, n_seqs, max_q, O, hsO, tsO, heads, Dn, P, Dv, alpha, causal,
                         span_for_kernel(sq), span_for_kernel(sk), span_for_kernel(sr), span_for_kernel(sv),
                         span_for_kernel(so)};
    cudaError_t e = cudaSuccess;
    if (launch_latent_prompt(a, static_cast<cudaStream_t>(stream), &e)) return finish(e);
    return finish(launch_latent_rows_packed(a, static_cast<cudaStream_t>(stream)));
}

int sbgemm_pages_workspace_bytes(int64_t num_blocks, int64_t n_seqs, int64_t n, size_t* bytes) {
    if (!bytes) return SBGEMM_ERR_NULL_POINTER;
    if (num_blocks < 0 || n_seqs < 0 || n < 0 || num_blocks >= kInt || n_seqs >= kInt || n >= kInt)
        return SBGEMM_ERR_INVALID_VALUE;
    *bytes = pages_workspace_bytes(num_blocks, n_seqs, n);
    return SBGEMM_OK;
}

int sbgemm_pages_copy(const sbgemm_page_pool* pool, const int32_t* pairs, int64_t n, void* stream,
                      const sbgemm_options* opt) {
    if (n < 0 || n >= kInt / 2) return SBGEMM_ERR_INVALID_VALUE;
    PoolView v;
    if (const int st = read_pool(pool, false, &v)) return st;
    if (n == 0 || v.caches.n == 0) return SBGEMM_OK;
    if (!pairs) return SBGEMM_ERR_NULL_POINTER;
    if (!aligned(pairs, 4)) return SBGEMM_ERR_INVALID_VALUE;
    const int sms = current_sms();
    if (!sms) return SBGEMM_ERR_CUDA;
    void* ws = nullptr;
    const size_t need = pages_workspace_bytes(v.pool.num_blocks, 0, 0);
    if (const int st = check_pool_memory(v, {block(pairs, n * 8)}, opt, need, &ws)) return st;
    return finish(launch_pages_copy(v.caches, v.pool, pairs, n, ws, sms, static_cast<cudaStream_t>(stream)));
}

int sbgemm_pages_fork(const sbgemm_page_pool* pool, const int32_t* parents, const int32_t* children, int64_t n,
                      void* stream, const sbgemm_options* opt) {
    if (n < 0 || n >= kInt / 2) return SBGEMM_ERR_INVALID_VALUE;
    PoolView v;
    if (const int st = read_pool(pool, true, &v)) return st;
    if (n == 0) return SBGEMM_OK;
    if (!parents || !children) return SBGEMM_ERR_NULL_POINTER;
    if (!aligned(parents, 4) || !aligned(children, 4)) return SBGEMM_ERR_INVALID_VALUE;
    const int sms = current_sms();
    if (!sms) return SBGEMM_ERR_CUDA;
    void* ws = nullptr;
    const size_t need = pages_workspace_bytes(v.pool.num_blocks, v.pool.n_seqs, n);
    if (const int st = check_pool_memory(v, {block(parents, n * 4), block(children, n * 4)}, opt, need, &ws))
        return st;
    return finish(launch_pages_fork(v.caches, v.pool, parents, children, n, ws, sms,
                                    static_cast<cudaStream_t>(stream)));
}

int sbgemm_pages_append(const sbgemm_page_pool* pool, const int32_t* seqs, const int32_t* starts, int64_t n,
                        const void* const* rows, const int64_t* row_stride, int64_t total, void* stream,
                        const sbgemm_options* opt) {
    if (n < 0 || n >= kInt / 2 || total < 0 || total >= kInt) return SBGEMM_ERR_INVALID_VALUE;
    PoolView v;
    if (const int st = read_pool(pool, true, &v)) return st;
    if (n == 0) return SBGEMM_OK;
    if (!seqs || !starts) return SBGEMM_ERR_NULL_POINTER;
    if (!aligned(seqs, 4) || !aligned(starts, 4)) return SBGEMM_ERR_INVALID_VALUE;
    const int sms = current_sms();
    if (!sms) return SBGEMM_ERR_CUDA;
    PageRows r{};
    void* ws = nullptr;
    const size_t need = pages_workspace_bytes(v.pool.num_blocks, v.pool.n_seqs, n);
    const int st = check_pool_memory(v, {block(seqs, n * 4), block(starts, (n + 1) * 4)}, opt, need, &ws);
    if (st) return st;
    if (v.caches.n > 0 && total > 0 && (!rows || !row_stride)) return SBGEMM_ERR_NULL_POINTER;
    for (int i = 0; i < v.caches.n && total > 0; ++i) {
        if (!rows[i]) return SBGEMM_ERR_NULL_POINTER;
        if (!aligned(rows[i], 16) || row_stride[i] % 16 != 0) return SBGEMM_ERR_INVALID_VALUE;
        Bytes s{};
        if (!span_of(rows[i], 1, {{row_stride[i], total}, {1, v.caches.row_bytes[i]}}, &s))
            return SBGEMM_ERR_INVALID_VALUE;
        for (size_t j = 0; j < v.n_spans; ++j)
            if (meet(s, v.spans[j])) return SBGEMM_ERR_OUTPUT_OVERLAP;
        if (meet(s, block(ws, (int64_t)need))) return SBGEMM_ERR_OUTPUT_OVERLAP;
        if (const int m = in_device_memory({s})) return m;
        r.base[i] = static_cast<const char*>(rows[i]);
        r.stride[i] = row_stride[i];
    }
    return finish(launch_pages_append(v.caches, v.pool, seqs, starts, n, r, total, ws, sms,
                                      static_cast<cudaStream_t>(stream)));
}

int sbgemm_pages_free(const sbgemm_page_pool* pool, const int32_t* seqs, int64_t n, void* stream) {
    if (n < 0 || n >= kInt) return SBGEMM_ERR_INVALID_VALUE;
    PoolView v;
    if (const int st = read_pool(pool, true, &v)) return st;
    if (n == 0) return SBGEMM_OK;
    if (!seqs) return SBGEMM_ERR_NULL_POINTER;
    if (!aligned(seqs, 4)) return SBGEMM_ERR_INVALID_VALUE;
    if (!current_sms()) return SBGEMM_ERR_CUDA;
    void* ws = nullptr;
    if (const int st = check_pool_memory(v, {block(seqs, n * 4)}, nullptr, 0, &ws)) return st;
    return finish(launch_pages_free(v.pool, seqs, n, static_cast<cudaStream_t>(stream)));
}

int sbgemm_pages_compact(const sbgemm_page_pool* pool, int32_t* moved, void* stream, const sbgemm_options* opt) {
    PoolView v;
    if (const int st = read_pool(pool, true, &v)) return st;
    if (moved && !aligned(moved, 4)) return SBGEMM_ERR_INVALID_VALUE;
    const int sms = current_sms();
    if (!sms) return SBGEMM_ERR_CUDA;
    void* ws = nullptr;
    const size_t need = pages_workspace_bytes(v.pool.num_blocks, v.pool.n_seqs, 0);
    const int st = moved ? check_pool_memory(v, {block(moved, 4)}, opt, need, &ws)
                         : check_pool_memory(v, {}, opt, need, &ws);
    if (st) return st;
    return finish(launch_pages_compact(v.caches, v.pool, moved, ws, sms, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
