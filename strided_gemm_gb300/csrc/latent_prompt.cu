// Latent attention over packed sequences on the tensor cores (expanded form,
// see sbgemm_latent_attention): O = softmax(alpha Q K^T) V with K_h = [k_nope_h
// | k_rope], the rope part one for all heads.
//
// One CTA per 256 queries of a sequence and head: two tiles of 128 rows (the
// MMA's M) that share every block of 128 keys.  Per block j and tile t:
//   S_t = Q_t K_j^T    SS MMAs, 64-wide pieces of the head dimension, into TMEM
//   P_t = exp2(alpha log2(e) S_t - ref)   one thread a row, one pass over the
//         scores: the weights, rounded to the operands' type (summed before;
//         summing them as rounded took the loop over the registers, 444 us
//         for the 416 below, and the outputs were no nearer), and the scores'
//         maximum; then the weights go over the scores
//   O_t += P_t V_j     TS MMAs, A = P_t from TMEM, B = V_j read MN-major from
//         the rows as TMA lands them
// A row's reference maximum rises only when a score exceeds it by 2^8; then
// the row's own thread scales its sums and its row of O_t and weighs the block
// again (a pass for the maximum before the weights cost 350 cycles a block: 439
// us where this takes 416).  The tensor pipe takes P V_0, S_0 of the next
// block, P V_1, S_1 of the next block in turn, so that each tile's softmax runs
// under the other's MMAs, and the scores of a tile coming in say that its P V
// before them is done.
//
// Shared memory holds Q (96 KB at 192 dimensions) and a ring of eight 16 KB
// pieces, 128 keys x 64 dimensions each, of K_0, V_0, K_1, V_1, ...: a block's
// K is free once both tiles have its scores, its V once both P V are done,
// which lets five pieces of a block be followed by three of the next.  Two
// whole stages would not fit.  A commit that follows another one without MMAs
// between them holds the issue up for about 360 cycles (a barrier for each
// piece: 549 us, 515 without, for the prompts below), so
// every commit serves all that wait for it: the scores of the last tile tell
// its softmax, which tells the TMA warp (a commit to barriers of even and odd
// blocks for both cost registers: 426 us for 416, 14.3 for 12.5).
//
// Roles (12 warps, all waits bounded): warp 0 TMA, warp 1 MMAs, warps 4-7 and
// 8-11 the rows of the two tiles.  In the last block they also zero the rows of
// V past the sequence's end, which belong to the next sequence (0 times its
// infinities would not be 0).
//
// Measured on a GB300, bf16, 128 + 64 and 128 dimensions: three sequences of
// 2048 to 4096 queries after 1000 keys, 32 heads, causal, 416 us (1.20
// PFLOP/s); 2 heads x 16384, not causal, 1.38 PFLOP/s; 333 queries, 16 heads
// 13 us.  Bound: a block takes a tile's softmax (1.5 k cycles), its P V and next
// scores (20 MMAs of 66 cycles) and two notifications, 3.6 k cycles in a chain,
// against 2.6 k of the tensor pipe for both tiles.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <type_traits>

#include "debug_check.cuh"
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
    int Dv;
    // |alpha| log2 e, but never 0, so that a hidden score's infinity stays one: for
    // an alpha of 0 the least float, under which the largest score is below 2^-20.
    float scale;
    int negative;                            // alpha < 0
    float unit;                              // 1; NaN for an alpha that is: of rows that have a key
    int causal;
    uint32_t idesc_s, idesc_v, idesc_v_half; // P V of all columns at once; of 64 of them
    uint32_t idesc_v_tail;                   // and of V's last piece
    int o_vec;                               // O rows take 16-byte stores
    ByteSpan so;                             // debug builds: what O occupies
};

struct Smem {
    alignas(1024) uint8_t q[kTiles][kQPieces][kPiece];
    alignas(1024) uint8_t ring[kSlots][kPiece];
    // [2]: one for the even blocks, one for the odd ones.  Nothing is asked of
    // block b + 2 before block b is through, so a wait for block b never finds its
    // barrier a round further (where the parity says "not yet" for ever).
    uint64_t q_full, k_full[2], v_full[2], v_empty[2], k_empty[2];
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

// Whole: three pieces of K and two of V, every one of 64 columns (128 + 64
// dimensions of keys, 128 of values), known to the compiler.
template <typename T, bool kWhole>
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
    // Blocks of each tile.
    auto blocks_of = [&](int t) {
        const int first = m0 + t * BM, last = min(first + BM, nq) - 1;
        int keys = first < nq ? nk : 0;
        if (p.causal) keys = min(keys, max(0, last + nk - nq + 1));
        return (keys + BN - 1) / BN;
    };
    const int nb0 = blocks_of(0), nb1 = blocks_of(1), blocks = max(nb0, nb1);
    const int last_tile = nb1 > 0 ? 1 : 0;       // it has every block that any tile has
    const int k_pieces = kWhole ? 3 : p.n_pieces + p.rope, v_pieces = kWhole ? 2 : p.v_pieces;
    const int per_block = k_pieces + v_pieces;

    if (threadIdx.x == 0) {
        mbar_init(&sh.q_full, 1);
        for (int s = 0; s < 2; ++s) {
            mbar_init(&sh.k_full[s], 1);
            mbar_init(&sh.v_full[s], 1);
            mbar_init(&sh.v_empty[s], 1);
            mbar_init(&sh.k_empty[s], 1);
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
            mbar_arrive_expect_tx(&sh.q_full, (uint32_t)(((nb0 > 0) + (nb1 > 0)) * k_pieces * kPiece));
#pragma unroll
            for (int t = 0; t < kTiles; ++t) {
                if ((t == 0 ? nb0 : nb1) == 0) continue;
                for (int c = 0; c < k_pieces - p.rope; ++c)
                    tma_load_3d(sh.q[t][c], &tqn, &sh.q_full, 64 * c, head, q0 + m0 + t * BM);
                if (p.rope) tma_load_3d(sh.q[t][p.n_pieces], &tqr, &sh.q_full, 0, head, q0 + m0 + t * BM);
            }
            // The piece that was in a slot before: of a K, free with the last
            // tile's scores of its block, or of a V, free with its P V.
            int k_free = 0, v_free = 0;              // blocks known to be free
            int old = -kSlots, old_block = 0, old_piece = 0;
            bool ok = true;
            auto need_k = [&](int b) {               // blocks come here in order, none left out
                if (ok && b >= k_free) {
                    ok = bar_wait(&sh.k_empty[b & 1], (uint32_t)((b >> 1) & 1));
                    k_free = b + 1;
                }
            };
            auto need_v = [&](int b) {
                if (ok && b >= v_free) {
                    ok = bar_wait(&sh.v_empty[b & 1], (uint32_t)((b >> 1) & 1));
                    v_free = b + 1;
                }
            };
            auto next_slot = [&](int i) {
                if (old >= 0) {
                    if (old_piece < k_pieces) need_k(old_block);
                    else need_v(old_block);
                    if (++old_piece == per_block) {
                        old_piece = 0;
                        ++old_block;
                    }
                }
                ++old;
                return sh.ring[i & (kSlots - 1)];
            };
            int i = 0, j = 0;
            for (; j < blocks && ok; ++j) {
                const int n0 = k0 + j * BN;
                uint64_t* kb = &sh.k_full[j & 1];
                uint64_t* vb = &sh.v_full[j & 1];
                for (int c = 0; c < per_block; ++c, ++i) {
                    // The last block on this one's barriers is through.
                    if (j >= 2 && c == 0) need_k(j - 2);
                    if (j >= 2 && c == k_pieces) need_v(j - 2);
                    uint8_t* dst = next_slot(i);
                    if (!ok) {
                        record_status(&g_wait_status, kWaitEmpty);
                        break;
                    }
                    if (c == 0) mbar_arrive_expect_tx(kb, (uint32_t)(k_pieces * kPiece));
                    if (c == k_pieces) mbar_arrive_expect_tx(vb, (uint32_t)(v_pieces * kPiece));
                    if (c < k_pieces - p.rope) tma_load_3d(dst, &tkn, kb, 64 * c, head, n0);
                    else if (c < k_pieces) tma_load_3d(dst, &tkr, kb, 0, 0, n0);
                    else tma_load_3d(dst, &tv, vb, 64 * (c - k_pieces), head, n0);
                }
            }
            // Copies still landing keep the CTA's shared memory (of the blocks
            // before the last two the MMAs have seen every one).
            for (int q = max(0, j - 2); ok && q < j; ++q)
                if (!bar_wait(&sh.k_full[q & 1], (uint32_t)((q >> 1) & 1)) ||
                    !bar_wait(&sh.v_full[q & 1], (uint32_t)((q >> 1) & 1))) {
                    record_status(&g_wait_status, kWaitDrain);
                    break;
                }
            if (!bar_wait(&sh.q_full, 0)) record_status(&g_wait_status, kWaitDrain);
        }
    } else if (warp == 1) {
        // ---- MMAs -----------------------------------------------------------------
        // One thread's chain of waits and issues: every instruction between two
        // MMAs is latency (a wait that is over costs some 250 cycles with its
        // address arithmetic), so there is one barrier a block for K and for V,
        // and slots follow by additions.
        if (elect_one()) {
            bool ok = true;
            const uint32_t q_lo = smem_u32(sh.q), ring_lo = smem_u32(sh.ring);
            auto fail = [&](unsigned int code) {
                record_status(&g_wait_status, code);
                ok = false;
            };
            // S_t of block j, whose K begins at slot `s`.
            auto scores = [&](auto tile, int j, uint32_t s) {
                constexpr int t = decltype(tile)::value;
                if (j >= (t == 0 ? nb0 : nb1)) return;
                if ((t == 0 || j >= nb0) && !bar_wait(&sh.k_full[j & 1], (uint32_t)((j >> 1) & 1)))
                    return fail(kWaitFull);
                tc_fence_after();
                if constexpr (kWhole) {
#pragma unroll
                    for (int c = 0; c < 3; ++c) {
                        const uint64_t da = desc16(q_lo + (t * kQPieces + c) * kPiece);
                        const uint64_t db = desc16(ring_lo + ((s + c) & (kSlots - 1)) * kPiece);
#pragma unroll
                        for (int x = 0; x < 4; ++x)
                            mma16_ss(tmem + kColS + t * BN, da + x * kStepK, db + x * kStepK, p.idesc_s,
                                     (c | x) ? 1u : 0u);
                    }
                } else {
                    for (int c = 0; c < k_pieces; ++c) {
                        const uint64_t da = desc16(q_lo + (t * kQPieces + c) * kPiece);
                        const uint64_t db = desc16(ring_lo + ((s + c) & (kSlots - 1)) * kPiece);
                        const int steps = c < p.n_pieces - 1 ? 4 : c == p.n_pieces - 1 ? p.n_steps : p.r_steps;
                        for (int x = 0; x < steps; ++x)
                            mma16_ss(tmem + kColS + t * BN, da + x * kStepK, db + x * kStepK, p.idesc_s,
                                     (c | x) ? 1u : 0u);
                    }
                }
                mma_commit(&sh.s_full[t]);
            };
            // O_t += P_t V of block j, whose V begins at slot `s`.
            auto values = [&](auto tile, int j, uint32_t s) {
                constexpr int t = decltype(tile)::value;
                const int n = t == 0 ? nb0 : nb1;
                if (j >= n) return;
                if (!bar_wait(&sh.p_full[t], (uint32_t)(j & 1))) return fail(kWaitMma);
                tc_fence_after();
                constexpr uint32_t d = tmem + kColO + t * BN, a = tmem + kColS + t * BN;
                if (v_pieces == 1 || s + 1 < kSlots) {
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
                if (j == n - 1) mma_commit(&sh.o_done[t]);
                else if (t == last_tile) mma_commit(&sh.v_empty[j & 1]);
            };
            constexpr std::integral_constant<int, 0> t0{};
            constexpr std::integral_constant<int, 1> t1{};
            if (blocks > 0) {
                if (!bar_wait(&sh.q_full, 0)) fail(kWaitFull);
                if (ok) scores(t0, 0, 0);
                if (ok) scores(t1, 0, 0);
            }
            uint32_t ks = 0;                         // slot of K_j's first piece
            for (int j = 0; j < blocks && ok; ++j) {
                const uint32_t vs = (ks + k_pieces) & (kSlots - 1);
                ks = (ks + per_block) & (kSlots - 1);
                if (!bar_wait(&sh.v_full[j & 1], (uint32_t)((j >> 1) & 1)) ||
                    (clean && j == blocks - 1 && !bar_wait(&sh.v_clean, 0))) {
                    fail(kWaitFull);
                    break;
                }
                values(t0, j, vs);
                if (ok) scores(t0, j + 1, ks);
                if (ok) values(t1, j, vs);
                if (ok) scores(t1, j + 1, ks);
            }
            // Nothing may still be writing TMEM when it is freed.
            mma_commit(&sh.done);
            if (!bar_wait(&sh.done, 0)) record_status(&g_wait_status, kWaitMma);
        }
    } else if (warp >= 4) {
        // ---- softmax and output, one row a thread ------------------------------------
        const int t = (warp - 4) >> 2, quarter = warp & 3;
        const int row = quarter * 32 + lane, m = m0 + t * BM + row;      // in the sequence
        const int n_blocks = t == 0 ? nb0 : nb1;
        const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
        const uint32_t s_at = tmem + lanes + kColS + t * BN, o_at = tmem + lanes + kColO + t * BN;
        const int last = p.causal ? min(nk - 1, m + nk - nq) : nk - 1;   // last key the row sees
        // Blocks below this one hide nothing from any of the tile's rows.
        const int open = (p.causal ? min(nk, max(0, m0 + t * BM + nk - nq + 1)) : nk) / BN;
        const float scale = p.scale;
        const bool negative = p.negative;
        float ref = -INFINITY, sum = 0.0f;
        bool ok = true;
        for (int j = 0; j < n_blocks; ++j) {
            if (!bar_wait(&sh.s_full[t], (uint32_t)(j & 1))) {
                record_status(&g_wait_status, kWaitMma);
                ok = false;
                break;
            }
            // Both tiles have their scores: the block's K is read.
            if (warp == 4 * last_tile + 4 && lane == 0) mbar_arrive(&sh.k_empty[j & 1]);
            tc_fence_after();
            const bool edge = j >= open;
            const int see = last - j * BN;               // columns up to this one count
            const float hidden = negative ? INFINITY : -INFINITY;
            if (edge) {
                // Scores that the row does not see are hidden in TMEM first, so
                // that the pass below has no masked form of its own (which took
                // it over the registers).
#pragma unroll 1
                for (int h = 0; h < 4; ++h) {
                    if (!__any_sync(~0u, see < 32 * h + 31)) continue;
                    float v[32];
                    uint32_t bits[32];
                    tmem_ld<32>(s_at + 32 * h, v);
#pragma unroll
                    for (int x = 0; x < 32; ++x) bits[x] = __float_as_uint(32 * h + x <= see ? v[x] : hidden);
                    tmem_st_bits<32>(s_at + 32 * h, bits);
                }
                tmem_wait_st();
            }
            if (j == 0) {
                // The first reference is the block's maximum.
                float top = hidden;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float v[64];
                    tmem_ld64(s_at + 64 * h, v);
#pragma unroll
                    for (int x = 0; x < 64; ++x) top = negative ? fminf(top, v[x]) : fmaxf(top, v[x]);
                }
                ref = top == hidden ? -INFINITY : negative ? -top * scale : top * scale;
            }
            // One pass over the row's scores, 16 columns under way while 16 are
            // worked on: the weights against the reference, packed in registers,
            // their sum, and the scores' maximum.
            uint32_t w[2][32];
            float top, part;
            auto weigh = [&] {
                const float shift = ref == -INFINITY ? 0.0f : ref;   // no key yet: every weight is 0
                float t0 = -INFINITY, t1 = -INFINITY, s0 = 0.0f, s1 = 0.0f;
                uint32_t v[2][16];
                tmem_ld16_begin(s_at, v[0]);
                tmem_ld16_end(v[0]);
#pragma unroll
                for (int h = 0; h < 8; ++h) {
                    if (h < 7) tmem_ld16_begin(s_at + 16 * (h + 1), v[(h + 1) & 1]);
                    if (negative) {                  // alpha < 0: the largest weight has the least score
#pragma unroll
                        for (int x = 0; x < 16; ++x) v[h & 1][x] ^= 0x80000000u;
                    }
#pragma unroll
                    for (int x = 0; x < 16; x += 2) {
                        float a = __uint_as_float(v[h & 1][x]), b = __uint_as_float(v[h & 1][x + 1]);
                        if (x & 2) asm("max.f32 %0, %0, %1, %2;" : "+f"(t1) : "f"(a), "f"(b));
                        else asm("max.f32 %0, %0, %1, %2;" : "+f"(t0) : "f"(a), "f"(b));
                        a = ex2_approx(fmaf(a, scale, -shift));
                        b = ex2_approx(fmaf(b, scale, -shift));
                        s0 += a;
                        s1 += b;
                        w[h >> 2][8 * (h & 3) + x / 2] = pack2_here<T>(a, b);
                    }
                    if (h < 7) tmem_ld16_end(v[(h + 1) & 1]);
                }
                top = fmaxf(t0, t1);
                part = s0 + s1;
            };
            weigh();
            const bool rise = top * scale > ref + kRaise;
            if (!__any_sync(~0u, rise)) {
                // Over the scores' first columns, all read by now.
#pragma unroll
                for (int h = 0; h < 2; ++h) tmem_st_bits<32>(s_at + 32 * h, w[h]);
                sum += part;
            } else {
                // Rare: what was summed is scaled to the new references, and the
                // block weighed again (written over the scores chunk by chunk,
                // always behind what is read).
                const float f = rise ? exp2f(ref - top * scale) : 1.0f;      // 0 for a first key
                if (rise) ref = top * scale;
                sum *= f;
                if (j > 0) {
#pragma unroll 1
                    for (int c = 0; c < p.Dv; c += 32) {
                        float o[32];
                        uint32_t bits[32];
                        tmem_ld<32>(o_at + c, o);
#pragma unroll
                        for (int x = 0; x < 32; ++x) bits[x] = __float_as_uint(o[x] * f);
                        tmem_st_bits<32>(o_at + c, bits);
                    }
                }
                const float shift = ref == -INFINITY ? 0.0f : ref;
#pragma unroll 1
                for (int h = 0; h < 4; ++h) {
                    float v[32];
                    uint32_t bits[16];
                    tmem_ld<32>(s_at + 32 * h, v);
#pragma unroll
                    for (int x = 0; x < 32; ++x) {
                        v[x] = ex2_approx(fmaf(negative ? -v[x] : v[x], scale, -shift));
                        sum += v[x];
                    }
#pragma unroll
                    for (int x = 0; x < 16; ++x) bits[x] = pack2<T>(v[2 * x], v[2 * x + 1]);
                    tmem_st_bits<16>(s_at + 16 * h, bits);
                }
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.p_full[t]);
            if (clean && j == blocks - 1 && t == last_tile) {
                // V_j - 2, the last one on this barrier, was read long ago: its
                // phase is over and this one's is the current one.
                if (!bar_wait(&sh.v_full[j & 1], (uint32_t)((j >> 1) & 1))) {
                    record_status(&g_wait_status, kWaitFull);
                    ok = false;
                }
                for (int c = 0; ok && c < v_pieces; ++c) {
                    // Whole rows: the swizzle stays inside a row's 128 bytes.
                    uint4* rows = reinterpret_cast<uint4*>(sh.ring[(j * per_block + k_pieces + c) & (kSlots - 1)]);
                    for (int x = v_rows * 8 + row; x < BN * 8; x += BM) rows[x] = make_uint4(0, 0, 0, 0);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.v_clean);
            }
        }
        if (ok && n_blocks > 0 && !bar_wait(&sh.o_done[t], 0)) {
            record_status(&g_wait_status, kWaitMma);
            ok = false;
        }
        ok = __all_sync(~0u, ok);
        if (ok) {
            tc_fence_after();
            const float inv = sum == 0.0f ? 0.0f : p.unit / sum;
            T* out = static_cast<T*>(p.O) + (int64_t)(q0 + m) * p.tsO + (int64_t)head * p.hsO;
#pragma unroll 1
            for (int c = 0; c < p.Dv; c += 32) {
                float o[32];
                if (n_blocks > 0) tmem_ld32(o_at + c, o);
                if (m >= nq || !dbg_in_bytes(out + c, sizeof(T) * min(32, p.Dv - c), p.so, &g_wait_status)) continue;
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
        cudaError_t e = cudaFuncSetAttribute(prompt_kernel<T, true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)kSmemBytes);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(prompt_kernel<T, false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     (int)kSmemBytes);
        if (e != cudaSuccess) return e;
        attr_done.fetch_or(bit);
    }
    const dim3 grid((unsigned)(p.q_blocks * p.heads), (unsigned)n_seqs);
    const bool whole = p.n_pieces == 2 && p.rope && p.v_pieces == 2 && p.n_steps == 4 && p.r_steps == 4 && p.Dv == 128;
    if (whole) prompt_kernel<T, true><<<grid, kThreads, kSmemBytes, stream>>>(m[0], m[1], m[2], m[3], m[4], p);
    else prompt_kernel<T, false><<<grid, kThreads, kSmemBytes, stream>>>(m[0], m[1], m[2], m[3], m[4], p);
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
    p.Dv = (int)a.Dv;
    const float scale = std::fabs(a.alpha * 1.4426950408889634f);
    p.scale = scale > 0.0f ? scale : 1.0e-45f;
    p.negative = a.alpha < 0.0f;
    p.unit = std::isnan(a.alpha) ? a.alpha : 1.0f;
    p.causal = a.causal;
    p.so = a.so;
    const bool bf = a.type == SBGEMM_TYPE_BF16;
    p.idesc_s = idesc16(bf, BN, false, false);
    p.idesc_v = idesc16(bf, (int)((a.Dv + 15) / 16 * 16), false, true);
    p.idesc_v_half = idesc16(bf, 64, false, true);
    p.idesc_v_tail = idesc16(bf, std::max<int>(16, (int)(a.Dv - 64 + 15) / 16 * 16), false, true);
    p.o_vec = reinterpret_cast<uintptr_t>(a.O) % 16 == 0 && a.tsO % 8 == 0 && (a.heads == 1 || a.hsO % 8 == 0);
    *err = bf ? launch<__nv_bfloat16>(m, p, a.n_seqs, stream) : launch<__half>(m, p, a.n_seqs, stream);
    return true;
}

unsigned int* status_word_latent_prompt() { return word_address(&g_wait_status); }

}  // namespace sbg
