// Latent attention over packed sequences on the tensor cores (expanded form,
// see sbgemm_latent_attention): O = softmax(alpha Q K^T) V with K_h = [k_nope_h
// | k_rope], the rope part one for all heads.
//
// One CTA per 256 queries of a sequence and head: two tiles of 128 rows (the
// MMA's M) that share every block of 128 keys.  Per block j and tile t:
//   S_t = Q_t K_j^T    SS MMAs, 64-wide pieces of the head dimension, into TMEM
//   P_t = exp2(alpha log2(e) S_t - ref)   one thread a row: one pass over the
//         scores for their maximum, one for the weights, which are rounded to
//         the operands' type (summed before) and written over the scores
//   O_t += P_t V_j     TS MMAs, A = P_t from TMEM, B = V_j read MN-major from
//         the rows as TMA lands them
// A row's reference maximum rises only when a score exceeds it by 2^8; then
// the row's own thread scales its sums and its row of O_t.  The tensor pipe
// takes P V_0, S_0 of the next block, P V_1, S_1 of the next block in turn, so
// that each tile's softmax runs under the other's MMAs, and the scores of a
// tile coming in say that its P V before them is done.
//
// Shared memory holds Q (96 KB at 192 dimensions) and a ring of eight 16 KB
// pieces, 128 keys x 64 dimensions each, of K_0, V_0, K_1, V_1, ...: a piece
// is released as soon as both tiles have read it, which lets five pieces of a
// block be followed by three of the next.  Two whole stages would not fit.
//
// Roles (12 warps, all waits bounded): warp 0 TMA, warp 1 MMAs, warps 4-7 and
// 8-11 the rows of the two tiles.  In the last block they also zero the rows of
// V past the sequence's end, which belong to the next sequence (0 times its
// infinities would not be 0).
//
// Bound: the tensor pipe, 128 x 128 x (192 + 128) products a tile and block in
// 20 MMAs of 66 cycles; the exponentials come next (16 a cycle and SM).
#include <algorithm>
#include <atomic>

#include "serving.h"
#include "tc16.cuh"

namespace sbg {
namespace {

constexpr int BM = 128, BN = 128, kTiles = 2;
constexpr int kSlots = 8;
constexpr int kPiece = 128 * 128;            // 128 rows of 64 elements
constexpr int kQPieces = 3;                  // 64-wide pieces of a query row at most
constexpr int kThreads = 12 * 32;
constexpr uint32_t kColS = 0, kColO = kTiles * BN;
constexpr float kRaise = 8.0f;
__device__ unsigned int g_wait_status = 0;

struct Params {
    const int32_t* q_starts; const int32_t* k_starts;
    int total_q, total_k, max_q;
    void* O; int64_t hsO, tsO;
    int heads, q_blocks;
    int n_pieces, v_pieces, rope;            // pieces of K's nope part and of V; rope: one more piece
    int n_steps, r_steps;                    // MMA K steps of the last nope piece and of the rope piece
    int Dn, Dv;
    float scale_log2;
    int causal;
    uint32_t idesc_s, idesc_v, idesc_v_half; // P V of all columns at once; of 64 of them
    int v_tail;                              // columns of V's last piece
    uint32_t idesc_v_tail;
    int o_vec;                               // O rows take 16-byte stores
};

struct Smem {
    alignas(1024) uint8_t q[kTiles][kQPieces][kPiece];
    alignas(1024) uint8_t ring[kSlots][kPiece];
    uint64_t q_full, full[kSlots], empty[kSlots];
    uint64_t s_full[kTiles], p_full[kTiles], o_done[kTiles], v_clean, done;
    uint32_t tmem_base;
};
constexpr size_t kSmemBytes = sizeof(Smem) + 1024;
static_assert(kSmemBytes <= 232448, "shared memory per CTA");

// starts[s], starts[s + 1] as a range inside [0, total] of at most `most` rows.
__device__ __forceinline__ bool packed_range(const int32_t* starts, int s, int total, int most, int* lo, int* n) {
    const int a = starts[s], b = starts[s + 1];
    const int x = min(max(a, 0), total), y = min(max(b, x), total);
    *lo = x;
    *n = min(y - x, most);
    return a == x && b == y && *n == y - x;
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 1)
prompt_kernel(const __grid_constant__ CUtensorMap tqn, const __grid_constant__ CUtensorMap tqr,
              const __grid_constant__ CUtensorMap tkn, const __grid_constant__ CUtensorMap tkr,
              const __grid_constant__ CUtensorMap tv, const __grid_constant__ Params p) {
    extern __shared__ uint8_t raw[];
    Smem& sh = *reinterpret_cast<Smem*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
    const int warp = uniform_warp(), lane = threadIdx.x & 31;
    // Query blocks of one head side by side (they share its keys), the ones
    // with the most keys first.
    const int qb = p.q_blocks - 1 - (int)(blockIdx.x % p.q_blocks);
    const int head = blockIdx.x / p.q_blocks, seq = blockIdx.y;
    int q0, nq, k0, nk;
    const bool good = packed_range(p.q_starts, seq, p.total_q, p.max_q, &q0, &nq) &
                      packed_range(p.k_starts, seq, p.total_k, p.total_k, &k0, &nk);
    if (!good && threadIdx.x == 0) record_status(&g_wait_status, kPagedInput);
    const int m0 = qb * (kTiles * BM);
    if (m0 >= nq) return;
    int nb[kTiles], blocks = 0;
#pragma unroll
    for (int t = 0; t < kTiles; ++t) {
        const int first = m0 + t * BM, last = min(first + BM, nq) - 1;
        int keys = first < nq ? nk : 0;
        if (p.causal) keys = min(keys, max(0, last + nk - nq + 1));
        nb[t] = (keys + BN - 1) / BN;
        blocks = max(blocks, nb[t]);
    }
    const int k_pieces = p.n_pieces + p.rope, per_block = k_pieces + p.v_pieces;

    if (threadIdx.x == 0) {
        mbar_init(&sh.q_full, 1);
        for (int s = 0; s < kSlots; ++s) {
            mbar_init(&sh.full[s], 1);
            mbar_init(&sh.empty[s], 1);
        }
        for (int t = 0; t < kTiles; ++t) {
            mbar_init(&sh.s_full[t], 1);
            mbar_init(&sh.p_full[t], 4);
            mbar_init(&sh.o_done[t], 1);
        }
        mbar_init(&sh.v_clean, 4);
        mbar_init(&sh.done, 1);
        fence_mbar_init();
        prefetch_tensormap(&tqn);
        prefetch_tensormap(&tkn);
        prefetch_tensormap(&tv);
    }
    if (warp == 1) {
        tmem_alloc(&sh.tmem_base, kTmemAll);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    constexpr uint32_t tmem = kTmemBase;
    // V's rows from here on are another sequence's, in the last block.
    const int v_rows = nk - (blocks - 1) * BN;
    const bool clean = blocks > 0 && v_rows < BN;

    if (warp == 0) {
        // ---- TMA ----------------------------------------------------------------
        if (lane == 0 && blocks > 0) {
            int tiles = 0;
            for (int t = 0; t < kTiles; ++t) tiles += nb[t] > 0;
            mbar_arrive_expect_tx(&sh.q_full, (uint32_t)(tiles * k_pieces * kPiece));
            for (int t = 0; t < kTiles; ++t) {
                if (nb[t] == 0) continue;
                for (int c = 0; c < p.n_pieces; ++c)
                    tma_load_3d(sh.q[t][c], &tqn, &sh.q_full, 64 * c, head, q0 + m0 + t * BM);
                if (p.rope) tma_load_3d(sh.q[t][p.n_pieces], &tqr, &sh.q_full, 0, head, q0 + m0 + t * BM);
            }
            int i = 0;
            const int total = blocks * per_block;
            for (int j = 0; i < total; ++j) {
                const int n0 = k0 + j * BN;
                bool ok = true;
                for (int c = 0; c < per_block; ++c, ++i) {
                    const int s = i % kSlots;
                    if (i >= kSlots && !mbar_wait(&sh.empty[s], (uint32_t)((i / kSlots - 1) & 1))) {
                        record_status(&g_wait_status, kWaitEmpty);
                        ok = false;
                        break;
                    }
                    mbar_arrive_expect_tx(&sh.full[s], kPiece);
                    if (c < p.n_pieces) tma_load_3d(sh.ring[s], &tkn, &sh.full[s], 64 * c, head, n0);
                    else if (c < k_pieces) tma_load_3d(sh.ring[s], &tkr, &sh.full[s], 0, 0, n0);
                    else tma_load_3d(sh.ring[s], &tv, &sh.full[s], 64 * (c - k_pieces), head, n0);
                }
                if (!ok) break;
            }
            // Copies still landing keep the CTA's shared memory.
            for (int q = i > kSlots ? i - kSlots : 0; q < i; ++q)
                if (!mbar_wait(&sh.full[q % kSlots], (uint32_t)((q / kSlots) & 1))) {
                    record_status(&g_wait_status, kWaitDrain);
                    break;
                }
            if (!mbar_wait(&sh.q_full, 0)) record_status(&g_wait_status, kWaitDrain);
        }
    } else if (warp == 1) {
        // ---- MMAs -----------------------------------------------------------------
        if (elect_one()) {
            bool ok = true;
            const uint32_t q_lo = smem_u32(sh.q), ring_lo = smem_u32(sh.ring);
            auto wait_piece = [&](int i) {
                if (ok && !mbar_wait(&sh.full[i % kSlots], (uint32_t)((i / kSlots) & 1))) {
                    record_status(&g_wait_status, kWaitFull);
                    ok = false;
                }
            };
            // S_t of block j.
            auto scores = [&](int t, int j) {
                if (j >= nb[t]) return;
                const int first = j * per_block;
                for (int c = 0; c < k_pieces; ++c) {
                    wait_piece(first + c);
                    if (!ok) return;
                    tc_fence_after();
                    const uint64_t da = desc16(q_lo + (t * kQPieces + c) * kPiece);
                    const uint64_t db = desc16(ring_lo + (first + c) % kSlots * kPiece);
                    const int steps = c < p.n_pieces - 1 ? 4 : c == p.n_pieces - 1 ? p.n_steps : p.r_steps;
                    if (steps == 4) {
#pragma unroll
                        for (int x = 0; x < 4; ++x)
                            mma16_ss(tmem + kColS + t * BN, da + x * kStepK, db + x * kStepK, p.idesc_s,
                                     (c | x) ? 1u : 0u);
                    } else {
                        for (int x = 0; x < steps; ++x)
                            mma16_ss(tmem + kColS + t * BN, da + x * kStepK, db + x * kStepK, p.idesc_s,
                                     (c | x) ? 1u : 0u);
                    }
                }
                mma_commit(&sh.s_full[t]);
            };
            auto release = [&](int first, int n) {
                for (int c = 0; c < n; ++c) mma_commit(&sh.empty[(first + c) % kSlots]);
            };
            if (blocks > 0) {
                if (!mbar_wait(&sh.q_full, 0)) {
                    record_status(&g_wait_status, kWaitFull);
                    ok = false;
                }
                if (ok) scores(0, 0);
                if (ok) scores(1, 0);
                if (ok) release(0, k_pieces);
            }
            for (int j = 0; j < blocks && ok; ++j) {
                const int first = j * per_block + k_pieces;      // V_j's pieces
                for (int c = 0; c < p.v_pieces; ++c) wait_piece(first + c);
                if (ok && clean && j == blocks - 1 && !mbar_wait(&sh.v_clean, 0)) {
                    record_status(&g_wait_status, kWaitFull);
                    ok = false;
                }
                for (int t = 0; t < kTiles && ok; ++t) {
                    if (j < nb[t]) {
                        if (!mbar_wait(&sh.p_full[t], (uint32_t)(j & 1))) {
                            record_status(&g_wait_status, kWaitMma);
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        const uint32_t d = tmem + kColO + t * BN, a = tmem + kColS + t * BN;
                        const int s = first % kSlots;
                        if (p.v_pieces == 1 || s + 1 < kSlots) {
                            // V's pieces lie side by side: all columns at once.
                            const uint64_t db = desc16(ring_lo + s * kPiece, kPiece);
#pragma unroll
                            for (int x = 0; x < BN / 16; ++x)
                                mma16_ts(d, a + 8 * x, db + x * kStepMN, p.idesc_v, (j | x) ? 1u : 0u);
                        } else {
                            const uint64_t d0 = desc16(ring_lo + s * kPiece), d1 = desc16(ring_lo);
#pragma unroll
                            for (int x = 0; x < BN / 16; ++x)
                                mma16_ts(d, a + 8 * x, d0 + x * kStepMN, p.idesc_v_half, (j | x) ? 1u : 0u);
#pragma unroll
                            for (int x = 0; x < BN / 16; ++x)
                                mma16_ts(d + 64, a + 8 * x, d1 + x * kStepMN, p.idesc_v_tail, (j | x) ? 1u : 0u);
                        }
                        if (j == nb[t] - 1) mma_commit(&sh.o_done[t]);
                    }
                    if (t == kTiles - 1) release(first, p.v_pieces);
                    if (j + 1 < blocks) {
                        scores(t, j + 1);
                        if (t == kTiles - 1 && ok) release((j + 1) * per_block, k_pieces);
                    }
                }
            }
            // Nothing may still be writing TMEM when it is freed.
            mma_commit(&sh.done);
            if (!mbar_wait(&sh.done, 0)) record_status(&g_wait_status, kWaitMma);
        }
    } else if (warp >= 4) {
        // ---- softmax and output, one row a thread ------------------------------------
        const int t = (warp - 4) >> 2, quarter = warp & 3;
        const int row = quarter * 32 + lane, m = m0 + t * BM + row;      // in the sequence
        const int n_blocks = t == 0 ? nb[0] : nb[1];
        const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
        const uint32_t s_at = tmem + lanes + kColS + t * BN, o_at = tmem + lanes + kColO + t * BN;
        const int last = p.causal ? min(nk - 1, m + nk - nq) : nk - 1;   // last key the row sees
        // Blocks below this one hide nothing from any of the tile's rows.
        const int open = (p.causal ? min(nk, max(0, m0 + t * BM + nk - nq + 1)) : nk) / BN;
        const float scale = p.scale_log2;
        float ref = -INFINITY, sum = 0.0f;
        bool ok = true;
        for (int j = 0; j < n_blocks; ++j) {
            if (!mbar_wait(&sh.s_full[t], (uint32_t)(j & 1))) {
                record_status(&g_wait_status, kWaitMma);
                ok = false;
                break;
            }
            tc_fence_after();
            const bool edge = j >= open;
            const int see = last - j * BN;               // columns up to this one count
            float top = -INFINITY;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float v[64];
                tmem_ld64(s_at + 64 * h, v);
                if (scale < 0.0f) {                      // the largest weight has the least score
#pragma unroll
                    for (int x = 0; x < 64; ++x) v[x] = -v[x];
                }
                if (edge) {
#pragma unroll
                    for (int x = 0; x < 64; ++x)
                        if (64 * h + x > see) v[x] = -INFINITY;
                }
                // Two chains of three-input maxima.
                float a = top, b = -INFINITY;
#pragma unroll
                for (int x = 0; x < 64; x += 4) {
                    asm("max.f32 %0, %0, %1, %2;" : "+f"(a) : "f"(v[x]), "f"(v[x + 1]));
                    asm("max.f32 %0, %0, %1, %2;" : "+f"(b) : "f"(v[x + 2]), "f"(v[x + 3]));
                }
                top = fmaxf(a, b);
            }
            top *= fabsf(scale);
            const bool rise = top > ref + kRaise;
            if (__any_sync(~0u, rise)) {
                const float f = rise ? exp2f(ref - top) : 1.0f;      // 0 at the first rise
                if (rise) ref = top;
                sum *= f;
                if (j > 0) {
#pragma unroll 1
                    for (int c = 0; c < p.Dv; c += 32) {
                        float o[32];
                        uint32_t bits[32];
                        tmem_ld32(o_at + c, o);
#pragma unroll
                        for (int x = 0; x < 32; ++x) bits[x] = __float_as_uint(o[x] * f);
                        tmem_st_bits<32>(o_at + c, bits);
                    }
                }
            }
            const float shift = ref == -INFINITY ? 0.0f : ref;       // no key yet: every weight is 0
            float part[2] = {0.0f, 0.0f};
#pragma unroll
            for (int h = 0; h < 4; ++h) {
                float v[32];
                uint32_t w[16];
                tmem_ld32(s_at + 32 * h, v);
#pragma unroll
                for (int x = 0; x < 32; ++x) {
                    v[x] = fmaf(v[x], scale, -shift);
                    if (edge && 32 * h + x > see) v[x] = -INFINITY;
                    v[x] = ex2_approx(v[x]);
                    part[x & 1] += v[x];
                }
#pragma unroll
                for (int x = 0; x < 16; ++x) w[x] = pack2<T>(v[2 * x], v[2 * x + 1]);
                // Columns 16 h .. of the row's scores, all read by now.
                tmem_st_bits<16>(s_at + 16 * h, w);
            }
            sum += part[0] + part[1];
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.p_full[t]);
            if (clean && j == blocks - 1 && t == (nb[1] == blocks ? 1 : 0)) {
                // These pieces are the ring's last: their phase is the slots' current one.
                for (int c = 0; c < p.v_pieces; ++c) {
                    const int i = j * per_block + k_pieces + c;
                    if (!mbar_wait(&sh.full[i % kSlots], (uint32_t)((i / kSlots) & 1))) {
                        record_status(&g_wait_status, kWaitFull);
                        ok = false;
                        break;
                    }
                    // Whole rows: the swizzle stays inside a row's 128 bytes.
                    uint4* rows = reinterpret_cast<uint4*>(sh.ring[i % kSlots]);
                    for (int x = v_rows * 8 + row; x < BN * 8; x += BM) rows[x] = make_uint4(0, 0, 0, 0);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.v_clean);
            }
        }
        if (ok && n_blocks > 0 && !mbar_wait(&sh.o_done[t], 0)) {
            record_status(&g_wait_status, kWaitMma);
            ok = false;
        }
        ok = __all_sync(~0u, ok);
        if (ok) {
            tc_fence_after();
            const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
            T* out = static_cast<T*>(p.O) + (int64_t)(q0 + m) * p.tsO + (int64_t)head * p.hsO;
#pragma unroll 1
            for (int c = 0; c < p.Dv; c += 32) {
                float o[32];
                if (n_blocks > 0) tmem_ld32(o_at + c, o);
                if (m >= nq) continue;
#pragma unroll
                for (int x = 0; x < 32; ++x) o[x] = sum == 0.0f ? 0.0f : o[x] * inv;
                if (p.o_vec && c + 32 <= p.Dv) {
#pragma unroll
                    for (int x = 0; x < 32; x += 8)
                        *reinterpret_cast<uint4*>(out + c + x) =
                            make_uint4(pack2<T>(o[x], o[x + 1]), pack2<T>(o[x + 2], o[x + 3]),
                                       pack2<T>(o[x + 4], o[x + 5]), pack2<T>(o[x + 6], o[x + 7]));
                } else {
#pragma unroll
                    for (int x = 0; x < 32; ++x)
                        if (c + x < p.Dv) out[c + x] = from_float<T>(o[x]);
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(kTmemBase, kTmemAll);
    }
}

// [rows][heads][inner] as a tensor map with boxes of 128 rows of one head.
bool make_map(CUtensorMap* map, const void* base, int64_t inner, int64_t heads, int64_t hs, int64_t rows, int64_t ts) {
    const int64_t row = (inner + 7) / 8 * 8;
    const uint64_t dims[3] = {(uint64_t)inner, (uint64_t)heads, (uint64_t)rows};
    const uint64_t strides[2] = {(uint64_t)(heads > 1 ? hs : row) * 2, (uint64_t)(rows > 1 ? ts : row) * 2};
    const uint32_t box[3] = {64, 1, 128};
    return encode_tmap_16(map, base, 3, dims, strides, box);
}

bool mappable(const void* base, int64_t heads, int64_t hs, int64_t rows, int64_t ts) {
    auto ok = [](int64_t s) { return s > 0 && s % 8 == 0 && s < ((int64_t)1 << 39); };
    return reinterpret_cast<uintptr_t>(base) % 16 == 0 && (heads == 1 || ok(hs)) && (rows == 1 || ok(ts));
}

template <typename T>
cudaError_t launch(const CUtensorMap* m, const Params& p, int64_t n_seqs, cudaStream_t stream) {
    static std::atomic<uint64_t> attr_done{0};
    int dev = 0;
    cudaGetDevice(&dev);
    const uint64_t bit = 1ull << (dev & 63);
    if (!(attr_done.load() & bit)) {
        const cudaError_t e = cudaFuncSetAttribute(prompt_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   (int)kSmemBytes);
        if (e != cudaSuccess) return e;
        attr_done.fetch_or(bit);
    }
    const dim3 grid((unsigned)(p.q_blocks * p.heads), (unsigned)n_seqs);
    prompt_kernel<T><<<grid, kThreads, kSmemBytes, stream>>>(m[0], m[1], m[2], m[3], m[4], p);
    return cudaGetLastError();
}

}  // namespace

bool launch_latent_prompt(const LatentPacked& a, cudaStream_t stream, cudaError_t* err) {
    if (a.Dn % 8 != 0 || a.P % 8 != 0 || a.Dv % 8 != 0 || a.Dn > 128 || a.P > 64 || a.Dv > 128) return false;
    if (a.total_k == 0 || !mappable(a.Q, a.heads, a.hsQ, a.total_q, a.tsQ) ||
        (a.Dn > 0 && !mappable(a.Kn, a.heads, a.hsK, a.total_k, a.tsK)) ||
        (a.P > 0 && !mappable(a.Kr, 1, 0, a.total_k, a.tsR)) || !mappable(a.V, a.heads, a.hsV, a.total_k, a.tsV))
        return false;
    const int64_t q_blocks = (std::min(a.max_q, a.total_q) + kTiles * BM - 1) / (kTiles * BM);
    if (q_blocks * a.heads > INT32_MAX) return false;
    // The parts a problem lacks get another operand's map, which no load uses.
    CUtensorMap m[5];
    const char* q = static_cast<const char*>(a.Q);
    bool ok = make_map(&m[4], a.V, a.Dv, a.heads, a.hsV, a.total_k, a.tsV);
    m[0] = m[1] = m[2] = m[3] = m[4];
    if (a.Dn > 0)
        ok = ok && make_map(&m[0], q, a.Dn, a.heads, a.hsQ, a.total_q, a.tsQ) &&
             make_map(&m[2], a.Kn, a.Dn, a.heads, a.hsK, a.total_k, a.tsK);
    if (a.P > 0)
        ok = ok && make_map(&m[1], q + 2 * a.Dn, a.P, a.heads, a.hsQ, a.total_q, a.tsQ) &&
             make_map(&m[3], a.Kr, a.P, 1, 0, a.total_k, a.tsR);
    if (!ok) {
        *err = cudaErrorInvalidValue;
        return true;
    }
    Params p{};
    p.q_starts = a.q_starts; p.k_starts = a.k_starts;
    p.total_q = (int)a.total_q; p.total_k = (int)a.total_k; p.max_q = (int)a.max_q;
    p.O = a.O; p.hsO = a.hsO; p.tsO = a.tsO;
    p.heads = (int)a.heads; p.q_blocks = (int)q_blocks;
    p.n_pieces = (int)((a.Dn + 63) / 64);
    p.rope = a.P > 0;
    p.v_pieces = (int)((a.Dv + 63) / 64);
    p.n_steps = a.Dn > 0 ? (int)((a.Dn - (p.n_pieces - 1) * 64 + 15) / 16) : 0;
    p.r_steps = (int)((a.P + 15) / 16);
    p.Dn = (int)a.Dn; p.Dv = (int)a.Dv;
    p.scale_log2 = a.alpha * 1.4426950408889634f;
    p.causal = a.causal;
    const bool bf = a.type == SBGEMM_TYPE_BF16;
    p.idesc_s = idesc16(bf, BN, false, false);
    p.idesc_v = idesc16(bf, (int)((a.Dv + 15) / 16 * 16), false, true);
    p.idesc_v_half = idesc16(bf, 64, false, true);
    p.v_tail = (int)(a.Dv > 64 ? a.Dv - 64 : 0);
    p.idesc_v_tail = idesc16(bf, std::max(16, (p.v_tail + 15) / 16 * 16), false, true);
    p.o_vec = reinterpret_cast<uintptr_t>(a.O) % 16 == 0 && a.tsO % 8 == 0 && (a.heads == 1 || a.hsO % 8 == 0);
    *err = bf ? launch<__nv_bfloat16>(m, p, a.n_seqs, stream) : launch<__half>(m, p, a.n_seqs, stream);
    return true;
}

unsigned int read_and_clear_status_latent_prompt(cudaStream_t stream) {
    return read_and_clear_word(reinterpret_cast<const void*>(&g_wait_status), stream);
}

}  // namespace sbg
