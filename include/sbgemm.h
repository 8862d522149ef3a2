/*
 * sbgemm: strided batched fp32 matrix product on one GB300 (sm_103a).
 *
 *     C[b] <- alpha * A[b] * B[b]            (accumulate == 0)
 *     C[b] <- alpha * A[b] * B[b] + C[b]     (accumulate != 0)
 *
 * for b = 0 .. batch-1, where A[b] is M x K, B[b] is K x N and C[b] is M x N.
 *
 * Source of the operation: StaleyNET, "GPU Implementation", section "The matrix
 * product" -- one kernel computes, for a batch of matrix pairs, alpha times A
 * times B with the previous C optionally added; every input is described by the
 * memory distance between neighbouring rows and between neighbouring columns,
 * so a transposed input is the same memory with the two distances exchanged,
 * and the batch covers all heads and sequences of attention in one launch.  The
 * argument list generalises the row-major cuBLAS call of "rvllm CUDA path"
 * (section "Matmuls go to cuBLAS": lda/ldb/ldc and a strided batch) and the
 * {batches, rows, inner, columns} sizes of the kael.cpp "CUDA backend" page.
 *
 * Layout.  Every operand is a base pointer plus three strides counted in fp32
 * ELEMENTS (not bytes), signed 64-bit:
 *     A[b][m][k] = A[b*bsA + m*rsA + k*csA]
 *     B[b][k][n] = B[b*bsB + k*rsB + n*csB]
 *     C[b][m][n] = C[b*bsC + m*rsC + n*csC]
 * A transposed read is the stored matrix with rs and cs exchanged (a row-major
 * W[N][K] read as B = W^T has rsB = 1, csB = K).  Strides of A and B may be
 * zero (broadcast: one matrix shared by every batch entry, or one row shared
 * by every row) or negative.  C's strides must map distinct (b, m, n) to
 * distinct elements.
 *
 * Numerics.  sbgemm and sbgemm_ex with math = SBGEMM_MATH_FP32 compute every
 * product and sum in fp32 with fused multiply-adds, each output's terms added
 * in increasing k, and the result formed as fmaf(alpha, sum, C_old).  Integer
 * inputs whose partial sums stay below 2^24 give exact results.
 * SBGEMM_MATH_TF32 (opt-in, sbgemm_ex only) rounds A and B to tf32 on the
 * tensor cores and accumulates in fp32.
 *
 * Ownership and synchronisation.  All pointers are device memory owned by the
 * caller (cudaMalloc, cudaMallocAsync, managed memory, or any allocator that
 * hands out such memory).  The library allocates nothing per call; it keeps
 * only immutable per-device properties, initialised once.  Calls are enqueued
 * on `stream` (a cudaStream_t; NULL = the legacy default stream) and return
 * without synchronising; errors raised inside a kernel surface at the
 * caller's next synchronisation.  The functions are thread-safe.
 *
 * Edge cases.  M, N or batch equal to 0: nothing is done (SBGEMM_OK, pointers
 * may be NULL).  K == 0: C <- alpha*0 (overwrite) or C is left as it was
 * (accumulate).  Without accumulation C is never read, so stale NaNs in C do
 * not leak into the result.
 *
 * Errors are returned as sbgemm_status codes; nothing is launched on error.
 */
#ifndef SBGEMM_H
#define SBGEMM_H

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define SBGEMM_API __attribute__((visibility("default")))
#else
#define SBGEMM_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    SBGEMM_OK = 0,
    SBGEMM_ERR_INVALID_VALUE = 1,   /* negative size, misaligned pointer, stride
                                       span overflowing int64, bad option value */
    SBGEMM_ERR_NULL_POINTER = 2,    /* a needed operand pointer is NULL */
    SBGEMM_ERR_OUTPUT_OVERLAP = 3,  /* C's strides map two outputs to one element,
                                       or C's address span meets A's or B's */
    SBGEMM_ERR_UNSUPPORTED = 4,     /* a forced path cannot serve this layout */
    SBGEMM_ERR_CUDA = 5,            /* CUDA runtime/driver error (launch, attribute,
                                       tensor-map encoding, no device) */
    SBGEMM_ERR_DEVICE_TIMEOUT = 6,  /* a bounded in-kernel wait expired; see
                                       sbgemm_device_status */
    SBGEMM_ERR_NOT_DEVICE_MEMORY = 7, /* an operand is not device-accessible memory,
                                       or its span leaves its allocation */
    SBGEMM_ERR_DEVICE_CHECK = 8     /* a kernel's own check found an input it
                                       could not use (a paged block id or
                                       sequence length out of range; a page
                                       request that is not valid or finds no
                                       free page; a debug build's out-of-span
                                       address) and skipped it; see
                                       sbgemm_device_status */
} sbgemm_status;

/* Arithmetic of sbgemm_options.math. */
enum {
    SBGEMM_MATH_FP32 = 0,  /* fp32 FFMA on the CUDA cores (default, strict) */
    SBGEMM_MATH_TF32 = 1   /* tf32 inputs, fp32 accumulation, on the tensor cores */
};

/* Kernel paths; sbgemm_options.force_path and sbgemm_plan_info.path. */
enum {
    SBGEMM_PATH_NONE = -1,        /* nothing to launch (empty problem, or
                                     K == 0 with accumulate) */
    SBGEMM_PATH_AUTO = 0,         /* let the planner choose */
    SBGEMM_PATH_GATHER_FFMA = 1,  /* any strides: coalesced strided gather into
                                     shared memory, FFMA register micro-tiles */
    SBGEMM_PATH_TMA_FFMA = 2,     /* unit-stride operands: TMA + mbarrier ring,
                                     FFMA register micro-tiles */
    SBGEMM_PATH_TMA_TF32 = 3      /* unit-stride operands (an MN-major one is
                                     transposed in shared memory): TMA +
                                     tcgen05.mma kind::tf32 with the
                                     accumulator in TMEM */
};

/* Operand layout classes reported by sbgemm_plan. */
enum {
    SBGEMM_LAYOUT_K_MAJOR = 0,   /* unit stride along K (A: csA == 1, B: rsB == 1);
                                    for C: unit stride along N (csC == 1) */
    SBGEMM_LAYOUT_MN_MAJOR = 1,  /* unit stride along M (A) or N (B);
                                    for C: unit stride along M (rsC == 1) */
    SBGEMM_LAYOUT_GENERAL = 2    /* no unit stride */
};

/* How the planner may split a tile's K range across CTAs when a workspace is
 * given; sbgemm_options.k_split.  The split follows the work-list scheme of
 * persistent CTAs, and its partial sums are added in a fixed order, so every
 * choice is deterministic from run to run (the pages' "Chapter 09 CUDA
 * backend", section "Reductions", for device sums; "GPU Implementation",
 * section "Making the embedding gradient repeatable", for gradients). */
enum {
    SBGEMM_KSPLIT_ANY = 0,    /* default: chained stream-K over the last waves,
                                 or, with fewer tiles than SMs and long K
                                 (e.g. the weight gradient Gt*X), independent K
                                 pieces summed in a fixed order; the latter
                                 rounds differently from the unsplit product.
                                 Small products on the gather path are cut
                                 into K pieces the same way, and products of
                                 at most 16384 outputs with K > 128 split K
                                 across the 32 lanes of a warp (one output per
                                 warp, a fixed shuffle tree). */
    SBGEMM_KSPLIT_EXACT = 1,  /* only splits whose result is bit-identical to
                                 the unsplit schedule (chained stream-K) */
    SBGEMM_KSPLIT_NONE = 2    /* never split K */
};

/* sbgemm_plan_info.stream_k. */
enum {
    SBGEMM_STREAM_K_NONE = 0,     /* every tile computed whole by one CTA */
    SBGEMM_STREAM_K_CHAINED = 1,  /* last waves split; a tail continues its
                                     head's k-ordered accumulation, so results
                                     do not change */
    SBGEMM_STREAM_K_PIECES = 2    /* all tiles split into independent K pieces
                                     over the SMs, the tail adding the earlier
                                     pieces' partial sums latest first (on the
                                     gather path the tile's last CTA adds all
                                     pieces in piece order) */
};

typedef struct {
    int math;          /* SBGEMM_MATH_* */
    int force_path;    /* SBGEMM_PATH_AUTO or a specific path */
    void* workspace;   /* optional device scratch owned by the caller, 256-byte
                          aligned, at least sbgemm_workspace_bytes() long; NULL
                          = none.  With it the planner may split the last waves
                          of tiles along K across all SMs (stream-K).  The
                          library writes it on `stream` during the call; calls
                          that may run concurrently need separate workspaces. */
    size_t workspace_bytes;
    int k_split;       /* SBGEMM_KSPLIT_*; 0 = any */
    int reserved[1];   /* must be zero */
} sbgemm_options;

typedef struct {
    int path;                 /* SBGEMM_PATH_* chosen (NONE: no launch) */
    int a_layout, b_layout, c_layout;   /* SBGEMM_LAYOUT_* */
    int a_broadcast, b_broadcast;       /* batch stride 0 with batch > 1 */
    int a_tma, b_tma;         /* operand can be fetched by a TMA tensor map */
    int tile_m, tile_n, tile_k;
    int ctas_per_sm;          /* resident CTAs per SM the plan assumes */
    int64_t ctas;             /* CTAs launched (0 when path == NONE) */
    int64_t tiles;            /* output tiles over all batch entries */
    int stream_k;             /* SBGEMM_STREAM_K_*: how tiles are split along K
                                 (needs a workspace) */
    int k_slices;             /* K slices (tile_k deep) per tile */
    int64_t dp_tiles;         /* tiles computed whole, data-parallel */
    int reserved[4];
} sbgemm_plan_info;

/* Activation of the fused epilogue; sbgemm_epilogue.activation.  The pages
 * name ReLU, GeluTanh and GeluExact ("Chapter 09 CUDA backend", section
 * "Elementwise"), the sigmoid ("PyTorch demystified 3") and SiLU ("rvllm
 * CUDA path", the FFN's silu(gate)). */
enum {
    SBGEMM_ACT_NONE = 0,
    SBGEMM_ACT_RELU = 1,       /* max(z, 0) */
    SBGEMM_ACT_SIGMOID = 2,    /* 1 / (1 + e^-z) */
    SBGEMM_ACT_SILU = 3,       /* z / (1 + e^-z) */
    SBGEMM_ACT_GELU_TANH = 4,  /* z/2 (1 + tanh(sqrt(2/pi) (z + 0.044715 z^3))) */
    SBGEMM_ACT_GELU_ERF = 5    /* z/2 (1 + erf(z / sqrt(2))) */
};

/* Fused epilogue of sbgemm_fused:
 *     C[b,m,n] <- act(alpha * (A*B)[b,m,n] + (accumulate ? C_old[b,m,n] : 0) + D[b,m,n])
 * with D[b,m,n] = D[b*bsD + m*rsD + n*csD] (strides in fp32 elements; zero
 * strides broadcast, so a bias per output column is rsD = 0, csD = 1, bsD = 0,
 * and a bias per batch entry and column is bsD = N).  The fusion of
 * "PyTorch demystified 3", section "Summary": the feed-forward layer's bias is
 * added inside the matmul kernel, saving a pass over C and a launch.
 * Rounding: alpha*acc (+ C_old) as sbgemm forms it, one fp32 add of D, then
 * the activation in fp32 through the CUDA math library. */
typedef struct {
    const float* D;            /* NULL = no addend; device memory, 4-byte aligned,
                                  its span must not meet C's */
    int64_t rsD, csD, bsD;
    int activation;            /* SBGEMM_ACT_* */
    int reserved[3];           /* must be zero */
} sbgemm_epilogue;

/* Strict fp32 product on the CUDA cores; the planner picks the kernel.
 * Arguments as described above; stream is a cudaStream_t (NULL = default). */
SBGEMM_API int sbgemm(const float* A, int64_t rsA, int64_t csA, int64_t bsA,
           const float* B, int64_t rsB, int64_t csB, int64_t bsB,
           float* C, int64_t rsC, int64_t csC, int64_t bsC,
           int64_t M, int64_t N, int64_t K, int64_t batch,
           float alpha, int accumulate, void* stream);

/* As sbgemm, with the arithmetic and the kernel path chosen by `opt` (NULL =
 * defaults).  math = SBGEMM_MATH_TF32 opts in to the tensor cores; when the
 * operands cannot be fetched by TMA (each needs a unit stride along K or
 * along its M / N index), the planner falls back to strict fp32 unless the
 * TF32 path was forced (then SBGEMM_ERR_UNSUPPORTED). */
SBGEMM_API int sbgemm_ex(const float* A, int64_t rsA, int64_t csA, int64_t bsA,
              const float* B, int64_t rsB, int64_t csB, int64_t bsB,
              float* C, int64_t rsC, int64_t csC, int64_t bsC,
              int64_t M, int64_t N, int64_t K, int64_t batch,
              float alpha, int accumulate, void* stream,
              const sbgemm_options* opt);

/* As sbgemm_ex, with a fused epilogue (NULL = none: same as sbgemm_ex).  All
 * paths and schedules apply it once per output, after the last K slice.  With
 * an epilogue, K == 0 with accumulate writes act(C_old + D) instead of
 * leaving C unchanged.  Errors as sbgemm_ex, plus SBGEMM_ERR_INVALID_VALUE for
 * an unknown activation, non-zero reserved fields, a misaligned D or a D span
 * overflowing int64; SBGEMM_ERR_OUTPUT_OVERLAP when D's span meets C's (or the
 * workspace); SBGEMM_ERR_NOT_DEVICE_MEMORY when D is not inside one device
 * allocation. */
SBGEMM_API int sbgemm_fused(const float* A, int64_t rsA, int64_t csA, int64_t bsA,
                 const float* B, int64_t rsB, int64_t csB, int64_t bsB,
                 float* C, int64_t rsC, int64_t csC, int64_t bsC,
                 int64_t M, int64_t N, int64_t K, int64_t batch,
                 float alpha, int accumulate, const sbgemm_epilogue* epi,
                 void* stream, const sbgemm_options* opt);

/* Fused attention over a batch of (sequence, head) problems, every operand
 * laid out by strides in fp32 elements like the product's:
 *     O[b,m,e] = sum_n softmax_n(alpha * sum_d Q[b,m,d] K[b,n,d]) V[b,n,e]
 * with Q[b,m,d] = Q[b*bsQ + m*rsQ + d*csQ], K[b,n,d], V[b,n,e] and O[b,m,e]
 * alike.  The pages compute attention as three steps (scores, softmax,
 * probs @ V) with the scores in global memory between them and name a fused
 * kernel as the fix ("rvllm CUDA path", section "What's basic about it");
 * here the scores and probabilities stay on chip.  Grouped-query heads are
 * rows of one batch entry stacked against one K and V ("rvllm CUDA path",
 * section "Matmuls go to cuBLAS").
 *   causal: 0, or 1 to mask keys n > position(m) = (m mod q_len) + N - q_len
 *           (q_len: query rows per head, 0 < q_len <= N; ignored when 0).
 *   D, Dv:  head dimensions; this build supports D = Dv = 32, 64, 96 or 128.
 * fp32 arithmetic: scores by FFMA, the softmax with exp2 of alpha*log2(e)
 * scaled scores, P V by FFMA.  Up to 8 query rows per batch entry (4 when D
 * is 96 or 128), a decode step, run a kernel that splits each entry's keys
 * across CTAs when sbgemm_attention_ex gives it a workspace (one CTA per
 * entry without one).  Asynchronous on `stream`; allocates nothing.
 * Errors: SBGEMM_ERR_INVALID_VALUE (negative size, N == 0 with rows to
 * compute, a bad causal flag or q_len, misaligned pointer, span overflow),
 * SBGEMM_ERR_NULL_POINTER, SBGEMM_ERR_OUTPUT_OVERLAP (O not injective or
 * meeting Q, K or V), SBGEMM_ERR_UNSUPPORTED (another head dimension, M over
 * 65535 x 128 rows), SBGEMM_ERR_NOT_DEVICE_MEMORY, SBGEMM_ERR_CUDA.  M, batch
 * or Dv zero: nothing to do. */
SBGEMM_API int sbgemm_attention(const float* Q, int64_t rsQ, int64_t csQ, int64_t bsQ,
                     const float* K, int64_t rsK, int64_t csK, int64_t bsK,
                     const float* V, int64_t rsV, int64_t csV, int64_t bsV,
                     float* O, int64_t rsO, int64_t csO, int64_t bsO,
                     int64_t M, int64_t N, int64_t D, int64_t Dv, int64_t batch,
                     float alpha, int causal, int64_t q_len, void* stream);

/* sbgemm_attention with options.  opt->math = SBGEMM_MATH_TF32 opts in to the
 * tensor-core kernel: S = Q K^T and P V by tcgen05 MMAs (tf32 inputs, fp32
 * accumulation), the softmax in fp32 as above.  It takes Q, K and V with unit
 * stride along the head dimension (csQ = csK = csV = 1), 16-byte aligned bases
 * and row / batch strides (a zero batch stride broadcasts); other layouts run
 * the fp32 kernel, unless opt->force_path = SBGEMM_PATH_TMA_TF32, which then
 * returns SBGEMM_ERR_UNSUPPORTED.  Problems of a few rows per entry (see
 * sbgemm_attention) run the fp32 decode kernel in either math unless the
 * tensor-core kernel is forced.  opt->workspace (caller-owned device memory
 * of opt->workspace_bytes, meeting no operand) lets the decode kernel split
 * the keys of an entry into chunks, each writing (2 + Dv) floats per row,
 * that a second launch merges in chunk order; sbgemm_workspace_bytes is
 * plenty.  k_split is ignored; force_path must be AUTO or TMA_TF32 (TMA_TF32
 * with math = TF32).  NULL opt is sbgemm_attention.  Errors as
 * sbgemm_attention, plus those of the options and of the workspace
 * (SBGEMM_ERR_NOT_DEVICE_MEMORY, SBGEMM_ERR_OUTPUT_OVERLAP). */
SBGEMM_API int sbgemm_attention_ex(const float* Q, int64_t rsQ, int64_t csQ, int64_t bsQ,
                        const float* K, int64_t rsK, int64_t csK, int64_t bsK,
                        const float* V, int64_t rsV, int64_t csV, int64_t bsV,
                        float* O, int64_t rsO, int64_t csO, int64_t bsO,
                        int64_t M, int64_t N, int64_t D, int64_t Dv, int64_t batch,
                        float alpha, int causal, int64_t q_len, void* stream,
                        const sbgemm_options* opt);

/* Fused attention reading K and V straight out of a paged cache through a
 * block table ("rvllm CUDA path", section "The kernels": the cache is one
 * buffer [num_blocks][block_size][n_kv_heads][head_dim], and context position
 * pos of a sequence lives in block block_table[seq * max_blocks + pos /
 * block_size] at offset pos % block_size; section "What's basic about it":
 * reading the blocks directly instead of gathering the whole context into a
 * contiguous buffer every decode step).
 *   K_cache, V_cache: [num_blocks][block_size][n_kv_heads][D] and [..][Dv]
 *           fp32, contiguous, 16-byte aligned.
 *   block_table: int32 [n_seqs][max_blocks] on the device; entries past a
 *           sequence's last block are never read.
 *   seq_lens: int32 [n_seqs] on the device, each sequence's context length
 *           (1..N, and >= q_len when causal), or NULL for N everywhere.
 *   N:      the longest context, at most max_blocks * block_size.
 *   Q, O:   strided like sbgemm_attention's, batch entry b = seq * n_kv_heads
 *           + head, M rows each (grouped-query heads stacked as rows);
 *           causal positions use the entry's own length:
 *           position(m) = (m mod q_len) + len - q_len.
 * O[b] is sbgemm_attention of Q[b] against the keys and values of positions
 * 0..len-1 of (seq, head).  D = Dv = 32, 64, 96 or 128; fp32 arithmetic as
 * sbgemm_attention (opt->math is not read); few-row problems use the decode
 * kernel and opt->workspace as sbgemm_attention_ex, others the row-block
 * kernel.  The host checks sizes, spans and overlaps as sbgemm_attention
 * (the caches, the table and seq_lens as operands O must not meet); the
 * table's and seq_lens' contents are device data and are checked by the
 * kernels: a block id outside [0, num_blocks) reads as a zero key and value,
 * a length out of range is clamped, and either makes the next
 * sbgemm_device_status return SBGEMM_ERR_DEVICE_CHECK (code 10); no access
 * leaves the caches.  opt->force_path must be AUTO.  Asynchronous on
 * `stream`; allocates nothing. */
SBGEMM_API int sbgemm_attention_paged(const float* Q, int64_t rsQ, int64_t csQ, int64_t bsQ,
                                      const float* K_cache, const float* V_cache,
                                      int64_t num_blocks, int64_t block_size, int64_t n_kv_heads,
                                      const int32_t* block_table, int64_t max_blocks,
                                      const int32_t* seq_lens,
                                      float* O, int64_t rsO, int64_t csO, int64_t bsO,
                                      int64_t M, int64_t N, int64_t D, int64_t Dv, int64_t n_seqs,
                                      float alpha, int causal, int64_t q_len, void* stream,
                                      const sbgemm_options* opt);

/* ---- 16-bit serving operators ------------------------------------------------
 * Operands below are arrays of 16-bit floats; strides count ELEMENTS (signed
 * 64-bit) as above.  Products are exact, sums and softmax statistics are fp32,
 * and each output is rounded once, to nearest even.  On the tensor cores
 * attention rounds its softmax weights to `type` too, for their product with
 * the values: relative to a reference within a factor of 2^8 of the row's
 * largest weight (fp16 below 2^-14 of the reference: to a multiple of 2^-24).
 * The paged form divides by the sum of the rounded weights, the packed form by
 * that of the weights before. */
enum {
    SBGEMM_TYPE_BF16 = 1,
    SBGEMM_TYPE_FP16 = 2
};

/* The strided batched product of sbgemm on 16-bit operands:
 *     C[b] <- alpha * A[b] * B[b] (+ C[b]),  A, B and C of `type`.
 * Arguments, edge cases and errors as sbgemm (pointers 2-byte aligned;
 * SBGEMM_ERR_INVALID_VALUE also for an unknown type).  Operands that a tensor
 * map can describe (a unit stride, 16-byte aligned base and other strides) run
 * on the tensor cores; every other layout runs a CUDA-core kernel with the
 * same sums in another order. */
SBGEMM_API int sbgemm_half(int type, const void* A, int64_t rsA, int64_t csA, int64_t bsA,
                           const void* B, int64_t rsB, int64_t csB, int64_t bsB,
                           void* C, int64_t rsC, int64_t csC, int64_t bsC,
                           int64_t M, int64_t N, int64_t K, int64_t batch,
                           float alpha, int accumulate, void* stream);

/* Latent attention, absorbed form, over a paged cache.  The cache keeps one
 * row a token for all heads, [c (R) | k_rope (P)]; a head's key is W_uk c with
 * k_rope beside it and its value W_uv c.  With W_uk absorbed into the query
 * (q_lat = W_uk^T q_nope, see sbgemm_half) the scores and the average need c
 * alone, and W_uv is applied to the average afterwards:
 *     O[s,t,h,:] = sum_n p_n c_n,  p = softmax_n(alpha * Q[s,t,h,:] . row_n)
 * over the keys n < len(s) and, when causal, n <= len(s) - q_len + t: the
 * q_len query tokens are a sequence's last ones (1 in a decode step, more with
 * drafted tokens).  A query with no key gives zeros.
 *   Q[s,t,h,:]   Q + s*bsQ + t*tsQ + h*hsQ, R + P contiguous elements
 *   O[s,t,h,:]   alike, R contiguous elements
 *   cache        page j, row i at cache + j*psC + i*rsC, R + P contiguous
 *   block_table  int32 [n_seqs][max_blocks]; seq_lens int32 [n_seqs] (0..N) or
 *                NULL for N everywhere; N <= max_blocks * block_size
 * Rows of the cache past a sequence's end are not read.  A block id outside
 * [0, num_blocks) reads as zero rows and a length outside [0, N] is clamped;
 * either makes the next sbgemm_device_status return SBGEMM_ERR_DEVICE_CHECK
 * (code 10).  NaN or infinity in a row that some queries of a sequence
 * mask and others do not may reach all of its queries.
 * R = 128, 256, 384 or 512 with P <= 64 a multiple of 8 and 16-byte aligned
 * bases and strides run on the tensor cores; other sizes up to R <= 512, R + P
 * <= 640 and other alignments run a slower kernel.  opt->workspace
 * (sbgemm_latent_workspace_bytes) lets the keys of a sequence be split over
 * the whole GPU (calls that may run at the same time need workspaces of their
 * own); without it one CTA reads all keys of a sequence for each 64 query rows.
 * The results depend on the split, and so on the lengths of all sequences,
 * in their rounding only, and repeat from run to run.  Of `opt` only the
 * workspace is read; force_path must be AUTO.  Errors as
 * sbgemm_attention_paged.  Asynchronous; allocates nothing. */
SBGEMM_API int sbgemm_latent_attention_paged(
    int type, const void* Q, int64_t hsQ, int64_t tsQ, int64_t bsQ,
    const void* cache, int64_t rsC, int64_t psC, int64_t num_blocks, int64_t block_size,
    const int32_t* block_table, int64_t max_blocks, const int32_t* seq_lens,
    void* O, int64_t hsO, int64_t tsO, int64_t bsO,
    int64_t q_len, int64_t heads, int64_t N, int64_t R, int64_t P, int64_t n_seqs,
    float alpha, int causal, void* stream, const sbgemm_options* opt);

/* Workspace with which sbgemm_latent_attention_paged splits keys freely. */
SBGEMM_API int sbgemm_latent_workspace_bytes(int device, size_t* bytes);

/* Latent attention, expanded form: every head's keys and values made from the
 * latents beforehand (one sbgemm_half of the latents with W_uk and W_uv), the
 * rope part of the keys shared by all heads.  Sequences are packed one behind
 * the other: sequence s has the queries q_starts[s] .. q_starts[s+1]-1 and the
 * keys k_starts[s] .. k_starts[s+1]-1 (int32 [n_seqs + 1] on the device).
 *     O[i,h,:] = sum_n p_n V[n,h,:],
 *     p = softmax_n(alpha * (Q[i,h,:Dn] . K_nope[n,h,:] + Q[i,h,Dn:] . K_rope[n,:]))
 * over the sequence's keys and, when causal, its first key_count - query_count
 * + (i - q_start) + 1 of them.  A query with no key gives zeros; rows of O
 * that belong to no sequence are left as they were.
 *   Q[i,h,:] = Q + i*tsQ + h*hsQ (Dn + P contiguous); K_nope[n,h,:] (Dn),
 *   V[n,h,:] (Dv) and O[i,h,:] (Dv) alike; K_rope[n,:] = K_rope + n*tsR (P;
 *   may be NULL when P == 0, K_nope when Dn == 0)
 *   total_q, total_k: rows of Q / O and of the keys; max_q: the most queries
 *   of a sequence
 * Starts that decrease, leave [0, total] or hold more than max_q queries are
 * clamped and reported as code 10 (sbgemm_device_status).  NaN or infinity in
 * V of a key that some queries of a 128-query block mask and others do not may
 * reach all of the block's queries.  Dn and Dv <= 128, P <= 64, all multiples
 * of 8, with 16-byte aligned bases and strides run on the tensor cores; other
 * sizes up to Dn + P <= 640 and Dv <= 512 a slower kernel.  Errors as
 * sbgemm_attention_paged.  Asynchronous; allocates nothing. */
SBGEMM_API int sbgemm_latent_attention(
    int type, const void* Q, int64_t hsQ, int64_t tsQ, int64_t total_q,
    const void* K_nope, int64_t hsK, int64_t tsK, const void* K_rope, int64_t tsR,
    const void* V, int64_t hsV, int64_t tsV, int64_t total_k,
    const int32_t* q_starts, const int32_t* k_starts, int64_t n_seqs, int64_t max_q,
    void* O, int64_t hsO, int64_t tsO,
    int64_t heads, int64_t Dn, int64_t P, int64_t Dv, float alpha, int causal, void* stream);

/* A pool of pages and the sequences that hold them, all in device memory.
 * Page j of cache i is the page_bytes[i] bytes from caches[i] + j *
 * page_bytes[i], block_size equal rows, so the caches of sbgemm_attention_paged
 * and sbgemm_latent_attention_paged alike (one cache a layer, or one for K and
 * one for V).  Sequence s holds the pages block_table[s][0 .. ceil(seq_lens[s]
 * / block_size) - 1]; ref_counts[j] counts the holders of page j, 0 = free.
 * The operations below run on `stream` as kernels, with no copy to the host
 * and no synchronisation, give the same result every time, and take the free
 * page with the lowest index first.  Requests they cannot serve are left out
 * whole and make the next sbgemm_device_status return
 * SBGEMM_ERR_DEVICE_CHECK: code 11 for one that is not valid, 12 when no page
 * was left.  Two operations on one pool need the same stream (or events). */
enum { SBGEMM_MAX_CACHES = 64 };
typedef struct {
    void* const* caches;         /* host array of n_caches device pointers,
                                    16-byte aligned */
    const int64_t* page_bytes;   /* host array; positive; page_bytes / block_size
                                    a whole multiple of 16 */
    int64_t n_caches;            /* 0 .. SBGEMM_MAX_CACHES */
    int64_t num_blocks, block_size;
    int32_t* ref_counts;         /* [num_blocks] */
    int32_t* block_table;        /* [n_seqs][max_blocks] */
    int64_t n_seqs, max_blocks;
    int32_t* seq_lens;           /* [n_seqs] */
} sbgemm_page_pool;

/* Bytes of workspace (opt->workspace) for any operation on such a pool with up
 * to n requests (pairs, forks or sequences). */
SBGEMM_API int sbgemm_pages_workspace_bytes(int64_t num_blocks, int64_t n_seqs, int64_t n, size_t* bytes);

/* Copies page pairs[k][0] to page pairs[k][1] in every cache, k < n (int32
 * [n][2]).  The bookkeeping is not touched and may be NULL.  A pair is not
 * valid if an id is out of range, if an earlier pair has the same destination,
 * or if its source is the destination of another pair. */
SBGEMM_API int sbgemm_pages_copy(const sbgemm_page_pool* pool, const int32_t* pairs, int64_t n,
                                 void* stream, const sbgemm_options* opt);

/* Forks: sequence children[k] becomes a copy of sequence parents[k] as it was
 * before the call.  Full pages are shared (their counts raised); the rows of a
 * last page that is not full are copied into a fresh page, so that parent and
 * child can both be appended to.  Not valid: an index out of range, a child
 * that holds tokens, is also a parent, or is an earlier request's child, a
 * parent whose length or last page is out of range.  (A shared page's id that
 * is out of range is carried over as it is, and reported.)  Requests are
 * granted in order while fresh pages last; those from the first one on that
 * the pool cannot serve are refused. */
SBGEMM_API int sbgemm_pages_fork(const sbgemm_page_pool* pool, const int32_t* parents, const int32_t* children,
                                 int64_t n, void* stream, const sbgemm_options* opt);

/* Appends rows: sequence seqs[k] grows by the tokens starts[k] ..
 * starts[k+1]-1 (int32 [n + 1]) of `rows`, which holds `total` tokens for each
 * cache: token j's row in cache i is at rows[i] + j * row_stride[i] bytes (host
 * arrays of n_caches; 16-byte aligned, strides multiples of 16).  Fresh pages
 * are taken as needed.  Not valid: an index out of range, a sequence that an
 * earlier request has, more tokens than max_blocks pages hold, a last page
 * that is not full and not the sequence's alone; starts that decrease or leave
 * [0, total] make every request not valid.  Granted in order while pages
 * last, as in sbgemm_pages_fork. */
SBGEMM_API int sbgemm_pages_append(const sbgemm_page_pool* pool, const int32_t* seqs, const int32_t* starts,
                                   int64_t n, const void* const* rows, const int64_t* row_stride, int64_t total,
                                   void* stream, const sbgemm_options* opt);

/* Frees sequences: the counts of their pages fall by one and their lengths
 * become 0 (their table rows stay as they were).  A sequence given twice is
 * freed once.  Not valid: an index out of range; a page out of range or not in
 * use is left out.  The caches may be NULL (n_caches == 0). */
SBGEMM_API int sbgemm_pages_free(const sbgemm_page_pool* pool, const int32_t* seqs, int64_t n, void* stream);

/* Compacts the pool: with U pages in use, the k-th page in use at an index >=
 * U moves to the k-th free index < U, in every cache, with its count and every
 * sequence's table entry; afterwards the pages 0 .. U-1 are in use.  *moved
 * (device, may be NULL) receives the number of pages moved. */
SBGEMM_API int sbgemm_pages_compact(const sbgemm_page_pool* pool, int32_t* moved, void* stream,
                                    const sbgemm_options* opt);

/* Validate and plan without launching or touching device memory: reports the
 * layout classes and the kernel path, tile and CTA count that sbgemm_ex would
 * use.  Pointers are only checked for NULL and alignment (no device query). */
SBGEMM_API int sbgemm_plan(const float* A, int64_t rsA, int64_t csA, int64_t bsA,
                const float* B, int64_t rsB, int64_t csB, int64_t bsB,
                const float* C, int64_t rsC, int64_t csC, int64_t bsC,
                int64_t M, int64_t N, int64_t K, int64_t batch,
                int accumulate, const sbgemm_options* opt,
                sbgemm_plan_info* info);

/* Workspace size that lets sbgemm_ex use the stream-K schedule on `device`
 * (one fp32 tile of partial sums per SM plus one flag word per SM); the
 * gather path's K pieces of small products fit in it too.  Returns
 * SBGEMM_OK and writes *bytes, or SBGEMM_ERR_CUDA if the device cannot be
 * queried. */
SBGEMM_API int sbgemm_workspace_bytes(int device, size_t* bytes);

/* Size in bytes of sbgemm_noalloc's scratch array (20 MiB + 4 KiB). */
#define SBGEMM_NOALLOC_SCRATCH_BYTES ((size_t)20 * 1024 * 1024 + 4096)

/* The fp32 product for callers that cannot allocate device memory.
 * The paper has no counterpart: it exists because the stream-K schedule (and
 * the K pieces of small products) needs scratch that sbgemm_ex takes from its
 * caller, and some callers cannot make any (code running under CUDA graph
 * capture, plugins given only their input and output buffers, loops that
 * must not pay cudaMalloc's synchronisation, runtimes whose allocator owns
 * all device memory).
 *
 * Arguments, layout and errors are those of sbgemm.  The call is sbgemm_ex
 * with math = FP32, the automatic path, k_split = SBGEMM_KSPLIT_ANY and the
 * library's scratch as the workspace, so its results are bit-identical to
 * sbgemm_ex given those options and a workspace of
 * SBGEMM_NOALLOC_SCRATCH_BYTES.  Against sbgemm (no workspace) they can
 * differ in rounding, within the fp32 bound, for the products the planner
 * cuts into independent K pieces (few output tiles with a long K, or small
 * products on the gather path): those pieces are summed in a fixed order
 * rather than in one k-ordered chain.
 *
 * The scratch is a file-scope device array of SBGEMM_NOALLOC_SCRATCH_BYTES
 * inside the library (room for the schedule on devices of up to 160 SMs),
 * created when the library's module is loaded and held on every GPU that
 * loads the library until the process exits.  Nothing is allocated per call:
 * no cudaMalloc, cudaFree or allocating library routine runs.  The first call
 * on a device looks up the array's device address (cudaGetSymbolAddress)
 * with that device current; make that first call before any stream capture
 * (a first call on a capturing stream returns SBGEMM_ERR_CUDA without
 * touching the stream, and a failed lookup is retried by the next call).
 * Every call shares the one array, which keeps the last call's contents; the
 * schedule clears its flags and counters on `stream` before each launch.
 * Calls that overlap on the GPU (different streams, or different host
 * threads) race on the scratch and must be serialised by the caller.
 * Returns SBGEMM_ERR_UNSUPPORTED if the current device would need more
 * scratch than the array holds (more than 160 SMs). */
SBGEMM_API int sbgemm_noalloc(const float* A, int64_t rsA, int64_t csA, int64_t bsA,
                              const float* B, int64_t rsB, int64_t csB, int64_t bsB,
                              float* C, int64_t rsC, int64_t csC, int64_t bsC,
                              int64_t M, int64_t N, int64_t K, int64_t batch,
                              float alpha, int accumulate, void* stream);

/* Reads and clears the device-side status words that kernels set when a
 * bounded in-kernel wait gives up or a device-side check skips an input
 * (after synchronising `stream`; the first code recorded is kept).  Returns
 * SBGEMM_OK, SBGEMM_ERR_DEVICE_TIMEOUT (codes 1-8) or SBGEMM_ERR_DEVICE_CHECK
 * (codes 9-12); *where_out (may be NULL) receives the code (0 if none): 1 a
 * loaded stage, 2 a released stage, 3 copies in flight at exit, 4 the MMAs of
 * a tile, 5 a free accumulator, 6 a stream-K partial sum, 7 / 8 the
 * self-test's mbarrier / flag, 9 an address outside its operand's span (debug
 * builds only; the access was skipped), 10 a paged-attention block id or
 * sequence length (or a packed sequence's start) out of range, 11 a page
 * request that is not valid, 12 one that found no free page. */
SBGEMM_API int sbgemm_device_status(void* stream, int* where_out);

/* Failure-detection self-test (a diagnostic of the library, not part of the
 * product).  Launches one CTA on `stream` that waits, with the bounded-wait
 * helpers every kernel uses and a limit of `limit_us` microseconds (1 ..
 * 2,000,000), on a condition nothing satisfies: an mbarrier phase that never
 * completes (SBGEMM_SELFTEST_MBARRIER) or a global flag no code sets
 * (SBGEMM_SELFTEST_FLAG).  The wait gives up, records its code, and the kernel
 * returns; the context stays usable and the next sbgemm_device_status call
 * returns SBGEMM_ERR_DEVICE_TIMEOUT with that code.  Returns SBGEMM_OK once
 * launched, SBGEMM_ERR_INVALID_VALUE for an unknown test or limit. */
enum { SBGEMM_SELFTEST_MBARRIER = 1, SBGEMM_SELFTEST_FLAG = 2 };
SBGEMM_API int sbgemm_selftest(int what, int64_t limit_us, void* stream);

/* Static, human-readable name of a status code. */
SBGEMM_API const char* sbgemm_status_string(int status);

/* Library version as MAJOR*10000 + MINOR*100 + PATCH. */
SBGEMM_API int sbgemm_version(void);

#ifdef __cplusplus
}
#endif

#endif /* SBGEMM_H */
