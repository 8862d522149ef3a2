// Internal declarations of the operators around a layer's products: 8-bit
// products and quantisation, norms and rotations.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "internal.h"

namespace sbg {

// ---- products of 8-bit floats (include/sbgemm.h, sbgemm_fp8) --------------------
// An operand of `rows` rows (M of A, N of B); strides in elements.
struct Fp8Operand {
    int type;                        // SBGEMM_TYPE_E4M3 or _E5M2
    int group;                       // rows a scale covers: 1 or 128
    const uint8_t* data; int64_t rs, ks, bs;
    const float* scale; int64_t rsS, ksS, bsS;
    int64_t rows;
    ByteSpan sd, ss;                 // debug builds: what the data and the scales occupy
};
struct Fp8Problem {
    Fp8Operand a, b;
    int type_c;
    void* C; int64_t rsC, csC, bsC;
    int64_t K, batch;
    float alpha;
    int accumulate;
    ByteSpan sc;                     // debug builds: what C occupies
};
constexpr int kScaleBlock = 128;     // elements of K a scale covers
// Any layout, on the CUDA cores (fp8_gather.cu).
cudaError_t launch_fp8_gather(const Fp8Problem& p, cudaStream_t stream);
// On the tensor cores (fp8_tc.cu); false if the layout has no tensor maps.
bool launch_fp8_tc(const Fp8Problem& p, int sms, cudaStream_t stream, cudaError_t* err);

// Quantisation (fp8_quantize.cu): X [batch][M][K] into an operand of M rows.
struct QuantizeProblem {
    int type_x;
    const void* X; int64_t rsX, csX, bsX;
    int type_y, group;
    uint8_t* Y; int64_t rsY, ksY, bsY;
    float* S; int64_t rsS, ksS, bsS;
    int64_t M, K, batch;
    ByteSpan sx, sy, ss;
};
cudaError_t launch_quantize(const QuantizeProblem& p, cudaStream_t stream);

// ---- norms and rotations (norm_rope.cu) ------------------------------------------
struct RopePart {
    const void* x; int64_t tsX, hsX;
    const void* dy; int64_t tsD, hsD;    // backward only
    void* y; int64_t tsY, hsY;           // y, or dx
    int heads, D, norm, start;
    const void* weight;
    float* dweight;
    ByteSpan sx, sd, sy, sw, sdw;
};
struct RopeProblem {
    int type;
    RopePart part[SBGEMM_MAX_ROPE_PARTS];
    int n_parts;
    const int32_t* positions;
    int64_t tokens;
    const uint64_t* steps;
    int dims;
    float magnitude;
    int interleaved;
    float eps;
    int accumulate;                      // backward: dweight is added to
    float* workspace;                    // backward: partial sums of the dweights
};
cudaError_t launch_norm_rope(const RopeProblem& p, int sms, cudaStream_t stream);
cudaError_t launch_norm_rope_backward(const RopeProblem& p, int sms, cudaStream_t stream);
size_t norm_rope_workspace_bytes(int sms, int64_t norm_total);
constexpr int64_t kRopeMaxD = 4096;

}  // namespace sbg
