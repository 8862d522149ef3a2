// C-ABI boundary of the operators around a layer's products (8-bit products and
// their quantisation, norms and rotations): argument validation and dispatch.
// As for the other products, every size a kernel depends on is checked before a
// launch, so that no access leaves what the caller described.
#include <cuda_runtime.h>

#include <array>

#include "api_checks.h"
#include "layers.h"
#include "sbgemm.h"

namespace sbg {
namespace {

int64_t float_bytes(int type) {
    return type == SBGEMM_TYPE_BF16 || type == SBGEMM_TYPE_FP16 ? 2 : type == SBGEMM_TYPE_FP32 ? 4 : 0;
}

// One 8-bit matrix of rows x K over the batch: its data's and scales' bytes.
int read_fp8(const sbgemm_fp8_matrix* m, int64_t rows, int64_t K, int64_t batch, Fp8Operand* out, Bytes* data,
             Bytes* scales) {
    if (m->type != SBGEMM_TYPE_E4M3 && m->type != SBGEMM_TYPE_E5M2) return SBGEMM_ERR_INVALID_VALUE;
    if (m->group != 1 && m->group != 128) return SBGEMM_ERR_INVALID_VALUE;
    *out = Fp8Operand{m->type, m->group, static_cast<const uint8_t*>(m->data), m->row_stride, m->k_stride,
                      m->batch_stride, m->scale, m->scale_row_stride, m->scale_k_stride, m->scale_batch_stride,
                      rows, {}, {}};
    if (K == 0) return SBGEMM_OK;
    if (!m->data || !m->scale) return SBGEMM_ERR_NULL_POINTER;
    if (!aligned(m->scale, 4)) return SBGEMM_ERR_INVALID_VALUE;
    const int64_t groups = (rows + m->group - 1) / m->group, blocks = (K + kScaleBlock - 1) / kScaleBlock;
    if (!span_of(m->data, 1, {{m->batch_stride, batch}, {m->row_stride, rows}, {m->k_stride, K}}, data) ||
        !span_of(m->scale, 4,
                 {{m->scale_batch_stride, batch}, {m->scale_row_stride, groups}, {m->scale_k_stride, blocks}}, scales))
        return SBGEMM_ERR_INVALID_VALUE;
    out->sd = span_for_kernel(*data);
    out->ss = span_for_kernel(*scales);
    return SBGEMM_OK;
}

// An array [tokens][heads][D] with unit stride along D.
struct Rows { const void* base; int64_t ts, hs, tokens, heads, D, esize; Bytes span; };

bool rows_span(Rows* r) {
    return span_of(r->base, r->esize, {{r->ts, r->tokens}, {r->hs, r->heads}, {1, r->D}}, &r->span);
}

// v modulo a positive pitch.
i128 modulo(i128 v, i128 pitch) {
    const i128 r = v % pitch;
    return r < 0 ? r + pitch : r;
}

// Whether two arrays share an element, or may: packed arrays have spans that meet,
// but parts of a token that do not (one projection's queries and keys side by side)
// or, token by token, parts of a head's place that do not (queries, keys and values
// head by head).
bool rows_meet(const Rows& a, const Rows& b) {
    if (!meet(a.span, b.span)) return false;
    if (a.esize != b.esize || a.hs < 0 || b.hs < 0) return true;
    i128 off = (i128)reinterpret_cast<uintptr_t>(b.base) - (i128)reinterpret_cast<uintptr_t>(a.base);
    if (a.tokens > 1) {
        const i128 pitch = (i128)a.ts * a.esize;
        if (a.ts != b.ts || pitch <= 0) return true;
        const i128 wa = ((i128)a.hs * (a.heads - 1) + a.D) * a.esize, wb = ((i128)b.hs * (b.heads - 1) + b.D) * b.esize;
        off = modulo(off, pitch);
        if (off >= wa && off + wb <= pitch) return false;
        // A part of a token of each in every pitch from a's start on, or from b's: then
        // no others can meet.
        if (wa > pitch || off + wb > pitch) {
            if (wb > pitch || pitch - off + wa > pitch) return true;
            off -= pitch;
        }
    }
    // Heads in step (a single one is in step with any).
    if (a.heads > 1 && b.heads > 1 && a.hs != b.hs) return true;
    const i128 step = (i128)(a.heads > 1 ? a.hs : b.hs) * a.esize;
    if (step <= 0) return true;
    off = modulo(off, step);
    return !(off >= a.D * a.esize && off + b.D * b.esize <= step);
}

bool same_rows(const Rows& a, const Rows& b) {
    return a.base == b.base && (a.ts == b.ts || a.tokens <= 1) && (a.hs == b.hs || a.heads <= 1);
}

template <size_t most> struct SpanList {
    Bytes at[most];
    size_t n = 0;
    void add(const Bytes& s) { at[n++] = s; }
};

// What both directions check; in: x (or dy and x) of each part, out: y or dx.
struct RopeArrays {
    Rows in[SBGEMM_MAX_ROPE_PARTS][2];
    int n_in[SBGEMM_MAX_ROPE_PARTS];
    Rows out[SBGEMM_MAX_ROPE_PARTS];
};

int check_rope_common(int type, const void* parts, int64_t n_parts, const int32_t* positions, int64_t tokens,
                      const uint64_t* steps, int64_t dims, int interleaved) {
    if (!float_bytes(type)) return SBGEMM_ERR_INVALID_VALUE;
    if (n_parts < 0 || n_parts > SBGEMM_MAX_ROPE_PARTS || tokens < 0 || dims < 0 || dims % 2 != 0)
        return SBGEMM_ERR_INVALID_VALUE;
    if (interleaved != 0 && interleaved != 1) return SBGEMM_ERR_INVALID_VALUE;
    if (n_parts > 0 && !parts) return SBGEMM_ERR_NULL_POINTER;
    if (n_parts == 0 || tokens == 0) return SBGEMM_OK;
    if (tokens >= kInt || dims > kRopeMaxD) return SBGEMM_ERR_UNSUPPORTED;
    if (dims > 0 && (!positions || !steps)) return SBGEMM_ERR_NULL_POINTER;
    if (dims > 0 && (!aligned(positions, 4) || !aligned(steps, 8))) return SBGEMM_ERR_INVALID_VALUE;
    return SBGEMM_OK;
}

int check_rope_sizes(int64_t heads, int64_t D, int64_t norm, int64_t start, int64_t dims, int64_t tokens) {
    if (heads < 0 || D < 0 || norm < 0 || start < 0 || norm > D || start > D || dims > D - start)
        return SBGEMM_ERR_INVALID_VALUE;
    if (D > kRopeMaxD || heads >= kInt || (i128)heads * tokens >= (i128)1 << 40) return SBGEMM_ERR_UNSUPPORTED;
    return SBGEMM_OK;
}

// Outputs have distinct elements and meet neither each other nor an input,
// except that an output may be an input of its own part; `extra`: arrays that
// no output may meet.
int check_rope_overlaps(const RopeArrays& a, const RopeProblem& p, const Bytes* extra, size_t n_extra) {
    for (int i = 0; i < p.n_parts; ++i) {
        const Rows& o = a.out[i];
        if (!injective(std::array<Axis, 3>{{{o.ts, o.tokens}, {o.hs, o.heads}, {1, o.D}}}))
            return SBGEMM_ERR_OUTPUT_OVERLAP;
        for (int j = 0; j < p.n_parts; ++j) {
            if (j > i && rows_meet(o, a.out[j])) return SBGEMM_ERR_OUTPUT_OVERLAP;
            for (int k = 0; k < a.n_in[j]; ++k)
                if (!(i == j && same_rows(o, a.in[j][k])) && rows_meet(o, a.in[j][k])) return SBGEMM_ERR_OUTPUT_OVERLAP;
        }
        for (size_t k = 0; k < n_extra; ++k)
            if (meet(o.span, extra[k])) return SBGEMM_ERR_OUTPUT_OVERLAP;
    }
    return SBGEMM_OK;
}

}  // namespace
}  // namespace sbg

using namespace sbg;

extern "C" {

int sbgemm_fp8(const sbgemm_fp8_matrix* A, const sbgemm_fp8_matrix* B, int type_c, void* C, int64_t rsC, int64_t csC,
               int64_t bsC, int64_t M, int64_t N, int64_t K, int64_t batch, float alpha, int accumulate,
               void* stream) {
    const int64_t esize = float_bytes(type_c);
    if (!esize) return SBGEMM_ERR_INVALID_VALUE;
    if (!A || !B) return SBGEMM_ERR_NULL_POINTER;
    if (M < 0 || N < 0 || K < 0 || batch < 0) return SBGEMM_ERR_INVALID_VALUE;
    if (M == 0 || N == 0 || batch == 0) return SBGEMM_OK;
    if (!C) return SBGEMM_ERR_NULL_POINTER;
    if (!aligned(C, esize)) return SBGEMM_ERR_INVALID_VALUE;
    Fp8Problem p{};
    Bytes da{}, db{}, sa{}, sb{}, sc{};
    if (const int st = read_fp8(A, M, K, batch, &p.a, &da, &sa)) return st;
    if (const int st = read_fp8(B, N, K, batch, &p.b, &db, &sb)) return st;
    if (!span_of(C, esize, {{bsC, batch}, {rsC, M}, {csC, N}}, &sc)) return SBGEMM_ERR_INVALID_VALUE;
    if (!injective(std::array<Axis, 3>{{{bsC, batch}, {rsC, M}, {csC, N}}})) return SBGEMM_ERR_OUTPUT_OVERLAP;
    if (K > 0)
        for (const Bytes& s : {da, db, sa, sb})
            if (meet(sc, s)) return SBGEMM_ERR_OUTPUT_OVERLAP;
    if (K == 0 && accumulate) return SBGEMM_OK;
    const int64_t tiles = ((M + 63) / 64) * ((N + 63) / 64);
    if (M >= kInt || N >= kInt || K >= kInt || batch >= kInt || tiles >= kInt) return SBGEMM_ERR_UNSUPPORTED;
    const int sms = current_sms();
    if (!sms) return SBGEMM_ERR_CUDA;
    if (const int m = K > 0 ? in_device_memory({da, db, sa, sb, sc}) : in_device_memory({sc})) return m;
    p.type_c = type_c;
    p.C = C; p.rsC = rsC; p.csC = csC; p.bsC = bsC;
    p.K = K; p.batch = batch;
    p.alpha = alpha;
    p.accumulate = accumulate;
    p.sc = span_for_kernel(sc);
    cudaError_t e = cudaSuccess;
    if (launch_fp8_tc(p, sms, static_cast<cudaStream_t>(stream), &e)) return finish(e);
    return finish(launch_fp8_gather(p, static_cast<cudaStream_t>(stream)));
}

int sbgemm_quantize_fp8(int type_x, const void* X, int64_t rsX, int64_t csX, int64_t bsX,
                        const sbgemm_fp8_matrix* Y, int64_t M, int64_t K, int64_t batch, void* stream) {
    const int64_t esize = float_bytes(type_x);
    if (!esize) return SBGEMM_ERR_INVALID_VALUE;
    if (!Y) return SBGEMM_ERR_NULL_POINTER;
    if (M < 0 || K < 0 || batch < 0) return SBGEMM_ERR_INVALID_VALUE;
    Fp8Operand y{};
    Bytes sx{}, sd{}, ss{};
    if (M == 0 || K == 0 || batch == 0) return SBGEMM_OK;
    if (const int st = read_fp8(Y, M, K, batch, &y, &sd, &ss)) return st;
    if (!X) return SBGEMM_ERR_NULL_POINTER;
    if (!aligned(X, esize)) return SBGEMM_ERR_INVALID_VALUE;
    if (!span_of(X, esize, {{bsX, batch}, {rsX, M}, {csX, K}}, &sx)) return SBGEMM_ERR_INVALID_VALUE;
    const int64_t groups = (M + y.group - 1) / y.group, blocks = (K + kScaleBlock - 1) / kScaleBlock;
    if (!injective(std::array<Axis, 3>{{{y.bs, batch}, {y.rs, M}, {y.ks, K}}}) ||
        !injective(std::array<Axis, 3>{{{y.bsS, batch}, {y.rsS, groups}, {y.ksS, blocks}}}))
        return SBGEMM_ERR_OUTPUT_OVERLAP;
    if (meet(sd, sx) || meet(ss, sx) || meet(sd, ss)) return SBGEMM_ERR_OUTPUT_OVERLAP;
    if (M >= kInt || K >= kInt || batch >= kInt || (i128)M * blocks * batch >= (i128)1 << 40)
        return SBGEMM_ERR_UNSUPPORTED;
    if (!current_sms()) return SBGEMM_ERR_CUDA;
    if (const int m = in_device_memory({sx, sd, ss})) return m;
    const QuantizeProblem p{type_x, X, rsX, csX, bsX, y.type, y.group, static_cast<uint8_t*>(Y->data), y.rs, y.ks,
                            y.bs, Y->scale, y.rsS, y.ksS, y.bsS, M, K, batch, span_for_kernel(sx), y.sd, y.ss};
    return finish(launch_quantize(p, static_cast<cudaStream_t>(stream)));
}

int sbgemm_norm_rope(int type, const sbgemm_rope_part* parts, int64_t n_parts, const int32_t* positions,
                     int64_t tokens, const uint64_t* steps, int64_t dims, float magnitude, int interleaved, float eps,
                     void* stream) {
    if (const int st = check_rope_common(type, parts, n_parts, positions, tokens, steps, dims, interleaved)) return st;
    if (n_parts == 0 || tokens == 0) return SBGEMM_OK;
    const int64_t esize = float_bytes(type);
    RopeProblem p{};
    RopeArrays a{};
    Bytes extra[2 + SBGEMM_MAX_ROPE_PARTS];
    size_t n_extra = 0;
    if (dims > 0) {
        extra[n_extra++] = block(positions, tokens * 4);
        extra[n_extra++] = block(steps, dims / 2 * 8);
    }
    for (int64_t i = 0; i < n_parts; ++i) {
        const sbgemm_rope_part& s = parts[i];
        if (const int st = check_rope_sizes(s.heads, s.D, s.norm, s.start, dims, tokens)) return st;
        if (s.heads == 0 || s.D == 0) continue;
        if (!s.x || !s.y) return SBGEMM_ERR_NULL_POINTER;
        if (!aligned(s.x, esize) || !aligned(s.y, esize) || !aligned(s.weight, esize)) return SBGEMM_ERR_INVALID_VALUE;
        const int n = p.n_parts;
        a.in[n][0] = Rows{s.x, s.x_token, s.x_head, tokens, s.heads, s.D, esize, {}};
        a.out[n] = Rows{s.y, s.y_token, s.y_head, tokens, s.heads, s.D, esize, {}};
        a.n_in[n] = 1;
        if (!rows_span(&a.in[n][0]) || !rows_span(&a.out[n])) return SBGEMM_ERR_INVALID_VALUE;
        RopePart& o = p.part[n];
        o.x = s.x; o.tsX = s.x_token; o.hsX = s.x_head;
        o.y = s.y; o.tsY = s.y_token; o.hsY = s.y_head;
        o.heads = (int)s.heads; o.D = (int)s.D; o.norm = (int)s.norm; o.start = (int)s.start;
        o.sx = span_for_kernel(a.in[n][0].span);
        o.sy = span_for_kernel(a.out[n].span);
        if (s.weight && s.norm > 0) {
            o.weight = s.weight;
            extra[n_extra] = block(s.weight, s.norm * esize);
            o.sw = span_for_kernel(extra[n_extra++]);
        }
        ++p.n_parts;
    }
    if (p.n_parts == 0) return SBGEMM_OK;
    if (const int st = check_rope_overlaps(a, p, extra, n_extra)) return st;
    const int sms = current_sms();
    if (!sms) return SBGEMM_ERR_CUDA;
    SpanList<2 * SBGEMM_MAX_ROPE_PARTS + 2 + SBGEMM_MAX_ROPE_PARTS> used;
    for (int i = 0; i < p.n_parts; ++i) {
        used.add(a.in[i][0].span);
        used.add(a.out[i].span);
    }
    for (size_t k = 0; k < n_extra; ++k) used.add(extra[k]);
    if (const int m = in_device_memory(used.at, used.n)) return m;
    p.type = type;
    p.positions = dims > 0 ? positions : nullptr;
    p.tokens = tokens;
    p.steps = steps;
    p.dims = (int)dims;
    p.magnitude = magnitude;
    p.interleaved = interleaved;
    p.eps = eps;
    return finish(launch_norm_rope(p, sms, static_cast<cudaStream_t>(stream)));
}

int sbgemm_norm_rope_backward(int type, const sbgemm_rope_grad* parts, int64_t n_parts, const int32_t* positions,
                              int64_t tokens, const uint64_t* steps, int64_t dims, float magnitude, int interleaved,
                              float eps, int accumulate, void* stream, const sbgemm_options* opt) {
    void* ws = nullptr;
    size_t ws_bytes = 0;
    if (const int st = read_options(opt, &ws, &ws_bytes)) return st;
    if (const int st = check_rope_common(type, parts, n_parts, positions, tokens, steps, dims, interleaved)) return st;
    if (n_parts == 0) return SBGEMM_OK;
    const int64_t esize = float_bytes(type);
    RopeProblem p{};
    RopeArrays a{};
    Bytes extra[3 + 2 * SBGEMM_MAX_ROPE_PARTS];
    size_t n_extra = 0;
    if (dims > 0 && tokens > 0) {
        extra[n_extra++] = block(positions, tokens * 4);
        extra[n_extra++] = block(steps, dims / 2 * 8);
    }
    Bytes weights[SBGEMM_MAX_ROPE_PARTS] = {}, zeros[SBGEMM_MAX_ROPE_PARTS] = {};
    int n_zeros = 0;
    int64_t total = 0;
    bool wanted = false;
    for (int64_t i = 0; i < n_parts; ++i) {
        const sbgemm_rope_grad& s = parts[i];
        if (const int st = check_rope_sizes(s.heads, s.D, s.norm, s.start, dims, tokens)) return st;
        if (s.D == 0) continue;
        const bool grad = s.dweight && s.norm > 0;
        if (tokens == 0 || s.heads == 0) {
            // No rows: a dweight that is not added to is zero.
            if (grad && !accumulate) {
                if (!aligned(s.dweight, 4)) return SBGEMM_ERR_INVALID_VALUE;
                zeros[n_zeros++] = block(s.dweight, s.norm * 4);
            }
            continue;
        }
        if (!s.dy || !s.dx || (s.norm > 0 && !s.x)) return SBGEMM_ERR_NULL_POINTER;
        if (!aligned(s.dy, esize) || !aligned(s.dx, esize) || (s.norm > 0 && !aligned(s.x, esize)) ||
            !aligned(s.weight, esize) || !aligned(s.dweight, 4))
            return SBGEMM_ERR_INVALID_VALUE;
        const int n = p.n_parts;
        a.in[n][0] = Rows{s.dy, s.dy_token, s.dy_head, tokens, s.heads, s.D, esize, {}};
        a.in[n][1] = Rows{s.x, s.x_token, s.x_head, tokens, s.heads, s.norm, esize, {}};
        a.out[n] = Rows{s.dx, s.dx_token, s.dx_head, tokens, s.heads, s.D, esize, {}};
        a.n_in[n] = s.norm > 0 ? 2 : 1;
        if (!rows_span(&a.in[n][0]) || (s.norm > 0 && !rows_span(&a.in[n][1])) || !rows_span(&a.out[n]))
            return SBGEMM_ERR_INVALID_VALUE;
        RopePart& o = p.part[n];
        o.dy = s.dy; o.tsD = s.dy_token; o.hsD = s.dy_head;
        o.y = s.dx; o.tsY = s.dx_token; o.hsY = s.dx_head;
        o.heads = (int)s.heads; o.D = (int)s.D; o.norm = (int)s.norm; o.start = (int)s.start;
        o.sd = span_for_kernel(a.in[n][0].span);
        o.sy = span_for_kernel(a.out[n].span);
        if (s.norm > 0) {
            o.x = s.x; o.tsX = s.x_token; o.hsX = s.x_head;
            o.sx = span_for_kernel(a.in[n][1].span);
            if (s.weight) {
                o.weight = s.weight;
                extra[n_extra] = block(s.weight, s.norm * esize);
                o.sw = span_for_kernel(extra[n_extra++]);
            }
        }
        if (grad) {
            o.dweight = s.dweight;
            weights[n] = block(s.dweight, s.norm * 4);
            o.sdw = span_for_kernel(weights[n]);
            wanted = true;
        }
        total += s.norm;
        ++p.n_parts;
    }
    if (p.n_parts == 0 && n_zeros == 0) return SBGEMM_OK;
    if (const int st = check_rope_overlaps(a, p, extra, n_extra)) return st;
    // (A part has no rows because the others have none either, or has no heads: its
    // gradient, which is zeroed first, meets nothing of theirs.)
    for (int i = 0; i < n_zeros; ++i) {
        for (int j = 0; j < p.n_parts; ++j) {
            if (meet(zeros[i], a.out[j].span) || meet(zeros[i], weights[j])) return SBGEMM_ERR_OUTPUT_OVERLAP;
            for (int k = 0; k < a.n_in[j]; ++k)
                if (meet(zeros[i], a.in[j][k].span)) return SBGEMM_ERR_OUTPUT_OVERLAP;
        }
        for (size_t k = 0; p.n_parts > 0 && k < n_extra; ++k)
            if (meet(zeros[i], extra[k])) return SBGEMM_ERR_OUTPUT_OVERLAP;
    }
    const int sms = current_sms();
    if (!sms) return SBGEMM_ERR_CUDA;
    for (int i = 0; i < n_zeros; ++i)
        if (const int m = in_device_memory({zeros[i]})) return m;
    Bytes w{};
    if (wanted) {
        const size_t need = norm_rope_workspace_bytes(sms, total);
        if (!ws || ws_bytes < need) return SBGEMM_ERR_INVALID_VALUE;
        w = block(ws, (int64_t)need);
    }
    for (int i = 0; i < p.n_parts; ++i) {
        // A weight's gradient and the workspace meet nothing else.
        for (int j = 0; j < p.n_parts; ++j) {
            if (!p.part[i].dweight) break;
            if (j > i && p.part[j].dweight && meet(weights[i], weights[j])) return SBGEMM_ERR_OUTPUT_OVERLAP;
            if (meet(weights[i], a.out[j].span) || meet(weights[i], w)) return SBGEMM_ERR_OUTPUT_OVERLAP;
            for (int k = 0; k < a.n_in[j]; ++k)
                if (meet(weights[i], a.in[j][k].span)) return SBGEMM_ERR_OUTPUT_OVERLAP;
            for (size_t k = 0; k < n_extra; ++k)
                if (meet(weights[i], extra[k])) return SBGEMM_ERR_OUTPUT_OVERLAP;
        }
        if (wanted && meet(w, a.out[i].span)) return SBGEMM_ERR_OUTPUT_OVERLAP;
        for (int k = 0; wanted && k < a.n_in[i]; ++k)
            if (meet(w, a.in[i][k].span)) return SBGEMM_ERR_OUTPUT_OVERLAP;
    }
    for (size_t k = 0; wanted && k < n_extra; ++k)
        if (meet(w, extra[k])) return SBGEMM_ERR_OUTPUT_OVERLAP;
    for (int i = 0; wanted && i < n_zeros; ++i)
        if (meet(w, zeros[i])) return SBGEMM_ERR_OUTPUT_OVERLAP;
    SpanList<4 * SBGEMM_MAX_ROPE_PARTS + 3 + 2 * SBGEMM_MAX_ROPE_PARTS + 1> used;
    for (int i = 0; i < p.n_parts; ++i) {
        used.add(a.in[i][0].span);
        used.add(a.out[i].span);
        if (a.n_in[i] > 1) used.add(a.in[i][1].span);
        if (p.part[i].dweight) used.add(weights[i]);
    }
    for (size_t k = 0; k < n_extra; ++k) used.add(extra[k]);
    if (wanted) used.add(w);
    if (const int m = in_device_memory(used.at, used.n)) return m;
    p.type = type;
    p.positions = dims > 0 ? positions : nullptr;
    p.tokens = tokens;
    p.steps = steps;
    p.dims = (int)dims;
    p.magnitude = magnitude;
    p.interleaved = interleaved;
    p.eps = eps;
    p.accumulate = accumulate;
    p.workspace = wanted ? static_cast<float*>(ws) : nullptr;
    for (int i = 0; i < n_zeros; ++i) {
        const cudaError_t e = cudaMemsetAsync(reinterpret_cast<void*>((uintptr_t)zeros[i].lo), 0,
                                              (size_t)(zeros[i].hi - zeros[i].lo), static_cast<cudaStream_t>(stream));
        if (e != cudaSuccess) return finish(e);
    }
    if (p.n_parts == 0) return SBGEMM_OK;
    return finish(launch_norm_rope_backward(p, sms, static_cast<cudaStream_t>(stream)));
}

int sbgemm_norm_rope_workspace_bytes(int device, int64_t norm_total, size_t* bytes) {
    if (!bytes) return SBGEMM_ERR_NULL_POINTER;
    if (norm_total < 0 || norm_total > SBGEMM_MAX_ROPE_PARTS * kRopeMaxD) return SBGEMM_ERR_INVALID_VALUE;
    const DeviceProps* d = device_props(device);
    if (!d) {
        cudaGetLastError();
        return SBGEMM_ERR_CUDA;
    }
    *bytes = norm_rope_workspace_bytes(d->sm_count, norm_total);
    return SBGEMM_OK;
}

}  // extern "C"
