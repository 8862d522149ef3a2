// Latent attention over a paged cache on the tensor cores (absorbed form, see
// sbgemm_latent_attention_paged): every head of a sequence reads the same rows
// [c | k_rope], as keys whole and as values without their rope part.
//
// A unit of work is a block of BT keys of one sequence for NB query rows
// (token, head) of it, NB = 16, 32 or 64.  The products are computed
// transposed, keys and latents along the MMA's M and query rows along its N,
// so that a few heads waste nothing and the one copy of the rows in shared
// memory serves both:
//   S^T = K Q^T      M: 64 keys, N = NB, K = R + P,
//                    A = the rows, K-major; B = the queries
//   O^T += C^T P^T   M: 128 latents a tile, N = NB, K = BT keys,
//                    A = the same rows read MN-major; B = P^T, written by the
//                    softmax as rows of NB weights a key
// Such MMAs are bound by shared memory's 128 bytes a cycle for A and B: 24
// cycles for the scores' 64 x 16 x 16 (40 with M = 128), 40 for 128 x 16 x 16.
// O^T stays in TMEM (R / 128 tiles of NB columns) over all blocks of a
// sequence.  The softmax keeps a reference maximum a query row, raised only
// when a score exceeds it by a factor of 2^8 (then O^T, the sums and the
// reference are scaled, by all eight warps); P is rounded to the operands'
// type for the MMA and summed as rounded, in fp32, so that the weights add up to
// one.  Weights up to 2^8 of either type lose nothing by it; in fp16 one below
// 2^-14 keeps an absolute 2^-25.
//
// Work is spread as one list of blocks over the CTAs (one an SM), each CTA an
// equal run of it that may begin and end inside a sequence.  A sequence that
// lies in one CTA is written out at once; the pieces of others go to the
// workspace as (maximum, sum, unnormalised O) in fp32, and a second launch
// joins them in order.  The lists depend on the lengths alone, which the
// device knows; no result depends on timing.
//
// Roles (12 warps): a warp for each of the 2 or 3 stages loads every second
// or third block's rows, each run of rows inside a page looked up in the table
// and fetched by TMA, one lane a run (a bad page's coordinate lies outside the
// tensor map and reads as zeros).  A sequence's last, partial block, and pages
// whose runs are shorter than 8 rows, come by 16-byte cp.async with zeros past
// the end, so that nothing there can reach a result (cp.async for every block
// was bound by its issue: 6.4 us a block).  Warp 3 issues the MMAs, the scores
// of block j + 1 before P V of block j when its rows are there in time; warps
// 4-11 do the softmax, rescaling, queries and output.  Every wait is bounded.
//
// Up to 32 rows three stages of 48 keys keep two blocks' loads in flight under
// the third's MMAs: 8.7 k cycles for 144 keys, where two stages of 64 loaded and
// computed in turns, 11 k cycles for 128 (16 heads, all SMs).  64 rows' queries
// leave room for two stages of 64 only, which load and compute in turns: a block
// takes the time until its rows are in and a chain of scores, softmax and P V of
// 3.4 k cycles. So the block that a stage takes next is prefetched into L2: 128
// heads as below 171 us, 178 without. (Before it four stages of 32 keys took 443
// us for 177; each stage's load and release in two halves 181.)
//
// Measured on a GB300, bf16 or fp16, R = 512, P = 64, join included: 64
// sequences of 2048 to 8192 keys with 128 heads 171 us (399 MB: 2.3 TB/s, 539
// TFLOP/s); 32 sequences of up to 8191 keys with 16 heads 54 us (193 MB: 3.6
// TB/s, in the loop 5.5 to 5.9); one of 701 keys with 16 heads 14.5 us.
// Bound: few heads by the cache's bytes and a start of 7 us; 128 heads by the
// chain above and, at a sequence's end, the way of 64 x 512 sums to the workspace
// and back (join 12 us).
#include <algorithm>
#include <atomic>

#include "debug_check.cuh"
#include "serving.h"
#include "tc16.cuh"

namespace sbg {
namespace {

constexpr int kMmaWarp = 3, kMathWarp = 4, kMathWarps = 8, kWarps = 12;
constexpr int kThreads = kWarps * 32;
constexpr int kMaxChunks = 9;                // 64-wide pieces of a row: R <= 512 and the rope part
constexpr int kMaxTiles = 4;                 // R / 128
// Keys a block and stages of the ring, by query rows.
template <int NB> struct Shape {
    static constexpr int BT = NB == 64 ? 64 : 48;
    static constexpr int kStages = NB == 64 ? 2 : 3;
    static constexpr int kChunkBytes = BT * 128;             // a piece of a block: BT rows of 128 swizzled bytes
};
constexpr float kRaise = 8.0f;               // log2 headroom before the reference maximum rises
__device__ unsigned int g_wait_status = 0;

// A sequence that begins in a group's CTA `member` and ends in a later one: its
// first piece is that CTA's first or (second = 1) last one, the others are the
// first ones of the CTAs behind, up to `last`.
struct Join { int32_t seq, member, last, second; };

struct Params {
    const void* Q; int64_t hsQ, tsQ, bsQ;
    const void* cache; int64_t rsC, psC;
    const int32_t* table; const int32_t* seq_lens;
    void* O; int64_t hsO, tsO, bsO;
    int64_t max_blocks;
    int num_blocks, block_size;
    int run;                                 // rows a TMA box takes: the run of a block inside a page; 0: no TMA
    int q_len, heads, rows, N, R, P, n_seqs;
    int chunks, rope_steps;                  // 64-wide pieces of a row; MMA K steps of the rope piece
    int groups, per_group;                   // query-row groups; CTAs for each
    int split;                               // sequences may be split (workspace given)
    float scale_log2;
    int causal;
    uint32_t idesc_s, idesc_o;
    int o_vec;                               // rows of O take 8-byte stores
    float* parts;                            // [2 * CTAs][NB][2 + R]: maxima, sums, then O rows
    ByteSpan sq, sc, so, sw;                 // debug builds: what Q, the cache, O and the workspace occupy
};

template <int NB>
struct Ctl {
    uint64_t full[Shape<NB>::kStages], empty[Shape<NB>::kStages];
    uint64_t q_full, s_full[2], p_full, o_free, done;
    uint32_t tmem_base;
    int seq0, tile0, count;                  // this CTA's run of the list
    int scan[kWarps], rest[kWarps];
    alignas(16) float ref[NB];               // reference maxima
    alignas(16) float factor[NB];            // a rise's factors, then 1 / sum
    union alignas(16) {
        float part[4][NB];                   // maxima or sums of the four key quarters
        int64_t out[NB];                     // element offset of a row of O (-1: none)
    };
};

template <int NB>
constexpr size_t smem_bytes(int chunks) {
    using H = Shape<NB>;
    return (size_t)chunks * (NB * 128 + H::kStages * H::kChunkBytes) + H::kChunkBytes + sizeof(Ctl<NB>) + 1024;
}

// A vote and barrier of the eight math warps.
__device__ __forceinline__ bool math_any(bool v) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred a, b;\n\tsetp.ne.b32 a, %1, 0;\n\t"
        "barrier.cta.red.or.pred b, 1, 256, a;\n\tselp.u32 %0, 1, 0, b;\n\t}"
        : "=r"(r) : "r"((uint32_t)v) : "memory");
    return r != 0;
}
__device__ __forceinline__ void math_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool read) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(read ? 16 : 0) : "memory");
}

__device__ __forceinline__ int seq_len(const Params& p, int s, bool report) {
    if (!p.seq_lens) return p.N;
    const int n = p.seq_lens[s];
    if (n >= 0 && n <= p.N) return n;
    if (report) record_status(&g_wait_status, kPagedInput);
    return n < 0 ? 0 : p.N;
}
// Blocks a sequence counts for in the list: an empty one has its zeros to write.
template <int BT>
__device__ __forceinline__ int units_of(int len) { return len > 0 ? (len + BT - 1) / BT : 1; }

// A CTA's walk over its run: pieces of sequences in order.
template <int BT>
struct Walk {
    int seq, tile, left;     // the next piece begins at block `tile` of `seq`; units left
    int len, j0, j1;         // the piece: blocks j0 .. j1 - 1 of a sequence of `len` keys
    int s, units;            // its sequence and that one's units
    __device__ __forceinline__ bool next(const Params& p, bool report = false) {
        if (left <= 0 || seq >= p.n_seqs) return false;
        s = seq;
        len = seq_len(p, s, report);
        units = units_of<BT>(len);
        j0 = tile;
        const int n = min(units - tile, left);
        j1 = len > 0 ? j0 + n : j0;
        left -= n;
        tile += n;
        if (tile >= units) {
            seq += p.split ? 1 : p.per_group;
            tile = 0;
        }
        return true;
    }
};

template <typename T, int NB>
__global__ void __launch_bounds__(kThreads, 1)
decode_kernel(const __grid_constant__ CUtensorMap rows_map, const __grid_constant__ Params p) {
    constexpr int BT = Shape<NB>::BT, kStages = Shape<NB>::kStages, kChunkBytes = Shape<NB>::kChunkBytes;
    constexpr uint32_t kColO = 0, kColS = kMaxTiles * NB;
    static_assert(kColS + 2 * NB <= 512, "TMEM columns");
    extern __shared__ uint8_t raw[];
    uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
    uint8_t* sq = base;                                      // queries: [chunk][NB rows][128 bytes]
    uint8_t* skv = sq + p.chunks * (NB * 128);               // rows: [stage][chunk][BT][128]
    uint8_t* sp = skv + kStages * p.chunks * kChunkBytes;    // weights: [BT keys][128 bytes]
    Ctl<NB>& c = *reinterpret_cast<Ctl<NB>*>(sp + kChunkBytes);
    const int tid = threadIdx.x, warp = uniform_warp(), lane = tid & 31;
    const int group = blockIdx.x % p.groups, member = blockIdx.x / p.groups;
    const int tiles_o = p.R / 128;

    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&c.full[i], 1);
            mbar_init(&c.empty[i], 1);
        }
        mbar_init(&c.q_full, kMathWarps);
        for (int i = 0; i < 2; ++i) mbar_init(&c.s_full[i], 1);
        mbar_init(&c.p_full, kMathWarps);
        mbar_init(&c.o_free, kMathWarps);
        mbar_init(&c.done, 1);
        fence_mbar_init();
    }
    if (warp == kMmaWarp) {
        tmem_alloc(&c.tmem_base, kTmemAll);
        tmem_relinquish();
    }

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    // This CTA's run: units [lo, hi) of the list, lo located in a sequence.
    if (p.split) {
        // Units of this thread's sequence of the first round, and their sum over
        // the warp's lanes up to it; pools of more sequences look again below.
        const int u0 = tid < p.n_seqs ? units_of<BT>(seq_len(p, tid, false)) : 0;
        int rest = 0;
        for (int s = tid + kThreads; s < p.n_seqs; s += kThreads) rest += units_of<BT>(seq_len(p, s, false));
        auto warp_sum = [&](int v) {
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int x = __shfl_up_sync(~0u, v, o);
                if (lane >= o) v += x;
            }
            return v;
        };
        int inc = warp_sum(u0);
        const int rest_sum = p.n_seqs > kThreads ? __reduce_add_sync(~0u, rest) : 0;
        if (lane == 31) {
            c.scan[warp] = inc;
            c.rest[warp] = rest_sum;
        }
        __syncthreads();
        int total = 0;
        for (int w = 0; w < kWarps; ++w) total += c.scan[w] + c.rest[w];
        // No CTA between a sequence's first and last one is empty.
        const int members = min(p.per_group, total);
        const int lo = member < members ? (int)((int64_t)member * total / members) : 0;
        const int hi = member < members ? (int)((int64_t)(member + 1) * total / members) : 0;
        if (tid == 0) c.count = hi - lo;
        int before = 0;                      // units of the sequences of earlier rounds
        for (int s0 = 0; s0 < p.n_seqs && before <= lo; s0 += kThreads) {
            const int s = s0 + tid;
            int u = u0;
            if (s0 > 0) {
                u = s < p.n_seqs ? units_of<BT>(seq_len(p, s, false)) : 0;
                inc = warp_sum(u);
                __syncthreads();
                if (lane == 31) c.scan[warp] = inc;
                __syncthreads();
            }
            int at = before, round = 0;
            for (int w = 0; w < kWarps; ++w) {
                if (w < warp) at += c.scan[w];
                round += c.scan[w];
            }
            at += inc - u;
            if (u && lo >= at && lo < at + u) {
                c.seq0 = s;
                c.tile0 = lo - at;
            }
            before += round;
        }
        if (tid == 0 && hi == lo) c.seq0 = c.tile0 = 0;
    } else if (tid == 0) {
        c.seq0 = member;
        c.tile0 = 0;
        c.count = INT32_MAX;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    constexpr uint32_t tmem = kTmemBase;
    Walk<BT> w{c.seq0, c.tile0, c.count};

    if (warp < kStages) {
        // ---- rows of the cache into shared memory ---------------------------------
        const int st = warp;                 // this warp's stage
        const int r0 = lane >> 3, piece = lane & 7;
        const uint32_t stage = smem_u32(skv) + st * p.chunks * kChunkBytes;
        const char* cache = static_cast<const char*>(p.cache);
        const int row_pieces = (p.R + p.P) / 8;
        int i = 0;                           // blocks so far, over all pieces
        int landing = 0;                     // from 1, the stage's last block if it came by TMA
        bool ok = true;
        while (ok && w.next(p)) {
            const int32_t* table = p.table + w.s * p.max_blocks;
            // The page of a run's first row; num_blocks, outside the tensor map, for a bad one.
            auto page_of = [&](int n) {
                const int page = table[n / p.block_size];
                if (page >= 0 && page < p.num_blocks) return page;
                record_status(&g_wait_status, kPagedInput);
                return p.num_blocks;
            };
            int next = -1, next_page = 0;    // the stage's next block, already looked up
            for (int j = w.j0; j < w.j1; ++j, ++i) {
                if (i % kStages != st) continue;
                const uint32_t ph_empty = (uint32_t)((i / kStages - 1) & 1);
                if (p.run && (j + 1) * BT <= w.len) {
                    // A whole block: lane x takes run x.
                    const int runs = BT / p.run, n = j * BT + lane * p.run;
                    int page = next_page;
                    if (lane < runs && next != j) page = page_of(n);
                    if (i >= kStages && !bar_wait(&c.empty[st], ph_empty)) {
                        record_status(&g_wait_status, kWaitEmpty);
                        ok = false;
                    }
                    ok = __all_sync(~0u, ok);
                    if (!ok) break;
                    if (lane == 0) mbar_arrive_expect_tx(&c.full[st], (uint32_t)(p.chunks * kChunkBytes));
                    __syncwarp();
                    if (lane < runs) {
                        uint8_t* dst = skv + st * p.chunks * kChunkBytes + lane * p.run * 128;
                        for (int k = 0; k < p.chunks; ++k)
                            tma_load_3d(dst + k * kChunkBytes, &rows_map, &c.full[st], k * 64, n % p.block_size, page);
                    }
                    landing = i + 1;
                    // Into L2 already what this stage takes next (with three stages
                    // another two blocks are under way as it is).
                    next = j + kStages;
                    if (NB == 64 && next < w.j1 && (next + 1) * BT <= w.len) {
                        if (lane < runs) {
                            const int at = next * BT + lane * p.run;
                            next_page = page_of(at);
                            if (next_page < p.num_blocks)
                                for (int k = 0; k < p.chunks; ++k)
                                    tma_prefetch_3d(&rows_map, k * 64, at % p.block_size, next_page);
                        }
                    } else {
                        next = -1;
                    }
                    continue;
                }
                // The rows' places first: their table entries arrive while the stage drains.
                const char* src[BT / 4];
#pragma unroll
                for (int g = 0; g < BT / 4; ++g) {
                    const int n = j * BT + r0 + 4 * g;
                    src[g] = nullptr;
                    if (n < w.len) {
                        const int page = table[n / p.block_size];
                        if (page >= 0 && page < p.num_blocks)
                            src[g] = cache + 2 * (page * p.psC + (n % p.block_size) * p.rsC) + piece * 16;
                        else
                            record_status(&g_wait_status, kPagedInput);
                    }
                }
                if (i >= kStages && !bar_wait(&c.empty[st], ph_empty)) {
                    record_status(&g_wait_status, kWaitEmpty);
                    ok = false;
                }
                ok = __all_sync(~0u, ok);
                if (!ok) break;
#pragma unroll
                for (int g = 0; g < BT / 4; ++g) {
                    const int r = r0 + 4 * g;
                    const uint32_t dst = stage + r * 128 + ((piece ^ (r & 7)) << 4);
                    for (int k = 0; k < p.chunks; ++k) {
                        const bool read = src[g] != nullptr && k * 8 + piece < row_pieces &&
                                          dbg_in_bytes(src[g] + k * 128, 16, p.sc, &g_wait_status);
                        cp_async16(dst + k * kChunkBytes, read ? src[g] + k * 128 : cache, read);
                    }
                }
                asm volatile("cp.async.commit_group;\n\tcp.async.wait_group 0;" ::: "memory");
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&c.full[st]);
                landing = 0;                 // the stage's earlier blocks are through
            }
        }
        // Copies still landing keep the CTA's shared memory.
        if (landing && !bar_wait(&c.full[st], (uint32_t)(((landing - 1) / kStages) & 1)))
            record_status(&g_wait_status, kWaitDrain);
    } else if (warp == kMmaWarp) {
        // ---- MMAs ------------------------------------------------------------------
        if (elect_one()) {
            const uint32_t q_lo = smem_u32(sq), kv_lo = smem_u32(skv), p_lo = smem_u32(sp);
            const uint32_t stage_bytes = p.chunks * kChunkBytes;
            int i = 0, filled = 0;           // blocks and pieces with blocks so far
            bool ok = true;
            auto scores = [&](int b) {       // S^T of block number b
                tc_fence_after();
                const uint32_t d = tmem + kColS + (b & 1) * NB;
                uint64_t da = desc16(kv_lo + b % kStages * stage_bytes), dq = desc16(q_lo);
                for (int k = 0; k < p.R / 64; ++k) {
#pragma unroll
                    for (int x = 0; x < 4; ++x)
                        mma16_ss(d, da + x * kStepK, dq + x * kStepK, p.idesc_s, (k | x) ? 1u : 0u);
                    da += kChunkBytes >> 4;
                    dq += NB * 128 >> 4;
                }
                for (int x = 0; x < p.rope_steps; ++x)
                    mma16_ss(d, da + x * kStepK, dq + x * kStepK, p.idesc_s, 1u);
                mma_commit(&c.s_full[b & 1]);
            };
            auto timed_out = [&](unsigned int code) {
                record_status(&g_wait_status, code);
                ok = false;
            };
            while (ok && w.next(p)) {
                const int n = w.j1 - w.j0;
                if (n == 0) continue;        // an empty sequence
                if (!bar_wait(&c.q_full, (uint32_t)(filled & 1)) ||
                    !bar_wait(&c.full[i % kStages], (uint32_t)((i / kStages) & 1))) {
                    timed_out(kWaitFull);
                    break;
                }
                scores(i);
                for (int j = 0; j < n && ok; ++j, ++i) {
                    // The next block's scores as soon as its rows are there, but
                    // this block's P V does not wait for them.
                    bool ahead = j + 1 >= n;
                    const uint32_t ph_next = (uint32_t)(((i + 1) / kStages) & 1);
                    const long long t0 = clock64();
                    while (!mbar_try_wait(&c.p_full, (uint32_t)(i & 1))) {
                        if (!ahead && mbar_try_wait(&c.full[(i + 1) % kStages], ph_next)) {
                            scores(i + 1);
                            ahead = true;
                        }
                        if (clock64() - t0 > kWaitCycles) {
                            timed_out(kWaitMma);
                            break;
                        }
                    }
                    if (!ok) break;
                    if (j == 0 && filled > 0 && !bar_wait(&c.o_free, (uint32_t)((filled - 1) & 1))) {
                        timed_out(kWaitAccFree);
                        break;
                    }
                    tc_fence_after();
                    const uint32_t rows = kv_lo + i % kStages * stage_bytes;
                    for (int t = 0; t < tiles_o; ++t) {
                        const uint64_t da = desc16(rows + 2 * t * kChunkBytes, kChunkBytes), dp = desc16(p_lo);
#pragma unroll
                        for (int x = 0; x < BT / 16; ++x)
                            mma16_ss(tmem + kColO + t * NB, da + x * kStepMN, dp + x * kStepMN, p.idesc_o,
                                     (j | x) ? 1u : 0u);
                    }
                    mma_commit(&c.empty[i % kStages]);
                    if (!ahead) {
                        if (!bar_wait(&c.full[(i + 1) % kStages], ph_next)) {
                            timed_out(kWaitFull);
                            break;
                        }
                        scores(i + 1);
                    }
                }
                ++filled;
            }
            // Nothing may still be writing TMEM when it is freed.
            mma_commit(&c.done);
            if (!bar_wait(&c.done, 0)) record_status(&g_wait_status, kWaitMma);
        }
    } else if (warp >= kMathWarp) {
        // ---- queries, softmax, output ------------------------------------------------
        const int m = tid - kMathWarp * 32;                  // 0 .. 255
        const int quarter = warp & 3, half = (warp - kMathWarp) >> 2;
        const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
        // Keys lie in lanes 0-15 of each quarter (the accumulator of an M = 64
        // MMA); a warp takes half of the columns, its lower and upper lanes a
        // half of those each, for the same keys.
        constexpr int CPW = NB / 2, CPT = NB / 4;
        const int row = quarter * 16 + (lane & 15), col = half * CPW + (lane >> 4) * CPT;
        const bool mine = row < BT;
        const int row_pieces = (p.R + p.P) / 8;
        int i = 0, piece_no = 0;                             // blocks and pieces so far
        bool ok = true;
        // Queries of the walk's piece on their way into shared memory.
        auto fetch_queries = [&](const Walk<BT>& w) {
            if (w.j1 > w.j0) {
                for (int x = m; x < NB * p.chunks * 8; x += 256) {
                    const int r = x / (p.chunks * 8), k = x % (p.chunks * 8);
                    const int gr = group * NB + r, t = gr / p.heads, h = gr % p.heads;
                    bool read = gr < p.rows && k < row_pieces;
                    const T* src = static_cast<const T*>(p.Q);
                    if (read) src += w.s * p.bsQ + t * p.tsQ + h * p.hsQ + k * 8;
                    read = read && dbg_in_bytes(src, 16, p.sq, &g_wait_status);
                    cp_async16(smem_u32(sq) + (k >> 3) * (NB * 128) + r * 128 + (((k & 7) ^ (r & 7)) << 4), src, read);
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        // P V of block number b is done: its weights are read and O is settled.
        auto pv_done = [&](int b) { return bar_wait(&c.empty[b % kStages], (uint32_t)((b / kStages) & 1)); };
        bool more = w.next(p, group == 0);
        if (more) fetch_queries(w);
        while (more) {
            const Walk<BT> now = w;          // this piece; the walk looks one ahead
            const int n = now.j1 - now.j0;
            if (m < NB) c.ref[m] = -INFINITY;
            if (n > 0) {
                asm volatile("cp.async.wait_group 0;" ::: "memory");
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&c.q_full);
            }
            math_sync();

            float l[CPT];
#pragma unroll
            for (int x = 0; x < CPT; ++x) l[x] = 0.0f;
            bool failed = false;
            for (int j = 0; j < n; ++j, ++i) {
                if (!bar_wait(&c.s_full[i & 1], (uint32_t)((i >> 1) & 1))) {
                    record_status(&g_wait_status, kWaitMma);
                    ok = false;
                }
                tc_fence_after();
                float a[CPT];
                bool rise = false;
                {
                    float v[CPW];
                    tmem_ld<CPW>(tmem + lanes + kColS + (i & 1) * NB + half * CPW, v);
#pragma unroll
                    for (int x = 0; x < CPT; ++x) {
                        const float other = __shfl_xor_sync(~0u, v[CPT + x], 16);
                        a[x] = (lane < 16 ? v[x] : other) * p.scale_log2;
                    }
                }
                const int first = (now.j0 + j) * BT;
                const int safe = p.causal ? now.len - p.q_len : now.len - 1;    // keys up to here: every row's
                if (!mine) {
#pragma unroll
                    for (int x = 0; x < CPT; ++x) a[x] = -INFINITY;
                } else if (first + BT - 1 > safe) {
#pragma unroll
                    for (int x = 0; x < CPT; ++x) {
                        int limit = now.len - 1;
                        if (p.causal) {
                            const int r = group * NB + col + x;
                            if (r < p.rows) limit = safe + r / p.heads;
                        }
                        if (first + row > limit) a[x] = -INFINITY;
                    }
                }
#pragma unroll
                for (int x = 0; x < CPT; ++x) rise |= a[x] > c.ref[col + x] + kRaise;
                if (math_any(rise || !ok)) {
                    if (math_any(!ok)) {
                        failed = true;
                        break;
                    }
                    // Raise the references to the block's maxima and scale what was summed.
#pragma unroll
                    for (int x = 0; x < CPT; ++x) {
                        float v = a[x];
#pragma unroll
                        for (int o = 8; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(~0u, v, o));
                        if ((lane & 15) == 0) c.part[quarter][col + x] = v;
                    }
                    math_sync();
                    if (m < NB) {
                        const float old = c.ref[m];
                        const float top = fmaxf(old, fmaxf(fmaxf(c.part[0][m], c.part[1][m]),
                                                           fmaxf(c.part[2][m], c.part[3][m])));
                        c.factor[m] = top == -INFINITY ? 1.0f : exp2f(old - top);    // 0 at the first rise
                        c.ref[m] = top;
                    }
                    math_sync();
#pragma unroll
                    for (int x = 0; x < CPT; ++x) l[x] *= c.factor[col + x];
                    if (j > 0) {
                        if (!pv_done(i - 1)) {
                            record_status(&g_wait_status, kWaitMma);
                            ok = false;
                        }
                        tc_fence_after();
                        constexpr int W = NB < 32 ? NB : 32;
#pragma unroll 1
                        for (int t = half; t < tiles_o; t += 2)
#pragma unroll 1
                            for (int x0 = 0; x0 < NB; x0 += W) {
                                const uint32_t at = tmem + lanes + kColO + t * NB + x0;
                                float o[W];
                                uint32_t bits[W];
                                tmem_ld<W>(at, o);
#pragma unroll
                                for (int x = 0; x < W; ++x) bits[x] = __float_as_uint(o[x] * c.factor[x0 + x]);
                                tmem_st_bits<W>(at, bits);
                            }
                        tmem_wait_st();
                    }
                }
                uint32_t w2[CPT / 2];
#pragma unroll
                for (int x = 0; x < CPT; x += 2) {
                    const float r0 = c.ref[col + x], r1 = c.ref[col + x + 1];
                    // A row that has seen no key yet has no reference: its weights are 0.
                    const float p0 = ex2_approx(a[x] - (r0 == -INFINITY ? 0.0f : r0));
                    const float p1 = ex2_approx(a[x + 1] - (r1 == -INFINITY ? 0.0f : r1));
                    w2[x / 2] = pack2<T>(p0, p1);
                    const float2 rounded = unpack2<T>(w2[x / 2]);
                    l[x] += rounded.x;
                    l[x + 1] += rounded.y;
                }
                // The block before has read its weights.
                if (i > 0 && !pv_done(i - 1)) {
                    record_status(&g_wait_status, kWaitMma);
                    ok = false;
                }
                if (mine) {
                    uint8_t* to = sp + row * 128;
                    const int at = col * 2, swz = (row & 7) << 4;
                    if constexpr (CPT >= 8) {
#pragma unroll
                        for (int x = 0; x < CPT / 8; ++x)
                            *reinterpret_cast<uint4*>(to + ((at + 16 * x) ^ swz)) =
                                make_uint4(w2[4 * x], w2[4 * x + 1], w2[4 * x + 2], w2[4 * x + 3]);
                    } else {
                        *reinterpret_cast<uint2*>(to + (at ^ swz)) = make_uint2(w2[0], w2[1]);
                    }
                }
                fence_proxy_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&c.p_full);
            }
            if (failed) break;
            // Every score of the piece is done (its last weights are written):
            // the next one's queries may come in under the rest.
            more = w.next(p, group == 0);
            if (more) fetch_queries(w);

            // The piece is done: its sums, then O^T out of TMEM.
            if (n > 0 && !pv_done(i - 1)) {
                record_status(&g_wait_status, kWaitMma);
                ok = false;
            }
            tc_fence_after();
#pragma unroll
            for (int x = 0; x < CPT; ++x) {
                float v = l[x];
#pragma unroll
                for (int o = 8; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
                if ((lane & 15) == 0) c.part[quarter][col + x] = v;
            }
            if (math_any(!ok)) break;
            const bool whole = now.j0 == 0 && (now.len == 0 || now.j1 == now.units);
            // A split sequence: this CTA's first piece goes to slot 0, its last to slot 1.
            const int slot = 2 * blockIdx.x + (piece_no > 0 ? 1 : 0);
            float* part = p.parts + (int64_t)slot * NB * (2 + p.R);
            if (m < NB) {
                const float sum = c.part[0][m] + c.part[1][m] + c.part[2][m] + c.part[3][m];
                c.factor[m] = sum == 0.0f ? 0.0f : whole ? 1.0f / sum : 1.0f;
                if (!whole && dbg_in_bytes(part, 4 * NB * (2 + p.R), p.sw, &g_wait_status)) {
                    part[m] = c.ref[m];
                    part[NB + m] = sum;
                }
            }
            math_sync();
            if (m < NB) {
                const int r = group * NB + m, t = r / p.heads, h = r % p.heads;
                c.out[m] = r < p.rows ? now.s * p.bsO + t * p.tsO + h * p.hsO : -1;
            }
            math_sync();
            // (Each branch its own loop: the rows' factors and places are read as
            // vectors, and one address runs over a piece's rows.)
            constexpr int W = NB < 32 ? NB : 32;
#pragma unroll 1
            for (int t = half; t < tiles_o; t += 2)
#pragma unroll 1
                for (int x0 = 0; x0 < NB; x0 += W) {
                    float o[W];
                    if (n > 0) tmem_ld<W>(tmem + lanes + kColO + t * NB + x0, o);
                    const int e = t * 128 + quarter * 32 + lane;
#pragma unroll
                    for (int x = 0; x < W; x += 4) {
                        const float4 f = *reinterpret_cast<const float4*>(&c.factor[x0 + x]);
                        o[x] = f.x == 0.0f ? 0.0f : o[x] * f.x;                // no key: zeros
                        o[x + 1] = f.y == 0.0f ? 0.0f : o[x + 1] * f.y;
                        o[x + 2] = f.z == 0.0f ? 0.0f : o[x + 2] * f.z;
                        o[x + 3] = f.w == 0.0f ? 0.0f : o[x + 3] * f.w;
                    }
                    if (!whole) {
                        float* dst = part + 2 * NB + (int64_t)x0 * p.R + e;
#pragma unroll
                        for (int x = 0; x < W; ++x, dst += p.R)
                            if (dbg_in_bytes(dst, 4, p.sw, &g_wait_status)) *dst = o[x];
                    } else {
                        T* dst = static_cast<T*>(p.O) + e;
#pragma unroll
                        for (int x = 0; x < W; x += 2) {
                            const longlong2 at = *reinterpret_cast<const longlong2*>(&c.out[x0 + x]);
                            if (at.x >= 0 && dbg_in_bytes(dst + at.x, sizeof(T), p.so, &g_wait_status))
                                dst[at.x] = from_float<T>(o[x]);
                            if (at.y >= 0 && dbg_in_bytes(dst + at.y, sizeof(T), p.so, &g_wait_status))
                                dst[at.y] = from_float<T>(o[x + 1]);
                        }
                    }
                }
            tc_fence_before();
            __syncwarp();
            if (n > 0 && lane == 0) mbar_arrive(&c.o_free);
            math_sync();                                         // c.* is free for the next piece
            ++piece_no;
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");   // on a failure too: shared memory outlives them
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(kTmemBase, kTmemAll);
    }
}

// Joins the pieces of split sequences in order: with the largest maximum M of
// a row's pieces, O = sum 2^(m - M) O_piece / sum 2^(m - M) l_piece.  Few
// pieces: a thread takes eight columns of a row over all of them, four pieces'
// loads in flight at once; many (one long sequence): eight warps share the pieces of
// 128 columns of a row.
constexpr int kJoinThreads = 256, kFewPieces = 8, kMaxJoins = 512;
// Blocks a SM: as many as stay resident, every one making the list once. Two,
// with the registers to have all of a thread's loads in flight, take the three
// measurements above, one sequence first, to 14.5, 51.7 and 167 us; three, for
// the larger amounts of 64 rows, to 16.0, 52.0 and 165.5; eight in turns to
// 16.5, 54.6 and 168.
template <int NB> constexpr int kJoinBlocks = NB == 64 ? 3 : 2;

template <typename T>
__device__ __forceinline__ void store4(T* o, float4 v, bool vec) {
    if (vec) {
        *reinterpret_cast<uint2*>(o) = make_uint2(pack2<T>(v.x, v.y), pack2<T>(v.z, v.w));
    } else {
        o[0] = from_float<T>(v.x);
        o[1] = from_float<T>(v.y);
        o[2] = from_float<T>(v.z);
        o[3] = from_float<T>(v.w);
    }
}
__device__ __forceinline__ void add4(float4& o, float w, const float4& v) {
    o.x = fmaf(w, v.x, o.x);
    o.y = fmaf(w, v.y, o.y);
    o.z = fmaf(w, v.z, o.z);
    o.w = fmaf(w, v.w, o.w);
}
__device__ __forceinline__ float4 scale4(const float4& o, float f) {
    return make_float4(o.x * f, o.y * f, o.z * f, o.w * f);
}

template <typename T, int NB>
__global__ void __launch_bounds__(kJoinThreads, kJoinBlocks<NB>) join_kernel(const __grid_constant__ Params p) {
    // Launched while the pieces are still being made: which sequences are split
    // follows from the lengths, as in the kernel that splits them, so that every
    // block has its list, those of few pieces from the front and those of many
    // from the back, before it waits for the pieces.
    constexpr int BT = Shape<NB>::BT, kJoinWarps = kJoinThreads / 32;
    __shared__ Join list[kMaxJoins];
    __shared__ float4 sums[8][32];
    __shared__ float tops[8], ls[8];
    __shared__ int scan[kJoinWarps], found[2][kJoinWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int few = 0, many = 0;
    {
        auto units_at = [&](int s) { return s < p.n_seqs ? units_of<BT>(seq_len(p, s, false)) : 0; };
        const int u0 = units_at(threadIdx.x);
        int mine = u0;
        for (int s = threadIdx.x + kJoinThreads; s < p.n_seqs; s += kJoinThreads) mine += units_at(s);
        mine = __reduce_add_sync(~0u, mine);
        if (lane == 0) scan[warp] = mine;
        __syncthreads();
        int total = 0;
        for (int w = 0; w < kJoinWarps; ++w) total += scan[w];
        const int members = min(p.per_group, total);
        int before = 0;                      // units of the sequences of earlier rounds
        for (int s0 = 0; s0 < p.n_seqs; s0 += kJoinThreads) {
            const int s = s0 + threadIdx.x, u = s0 == 0 ? u0 : units_at(s);
            int inc = u;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int x = __shfl_up_sync(~0u, inc, o);
                if (lane >= o) inc += x;
            }
            __syncthreads();
            if (lane == 31) scan[warp] = inc;
            __syncthreads();
            int at = before + inc - u;
            for (int w = 0; w < kJoinWarps; ++w) {
                if (w < warp) at += scan[w];
                before += scan[w];
            }
            // Unit u of the list belongs to member ceil((u + 1) members / total) - 1.
            auto member_of = [&](int unit) { return (int)(((int64_t)(unit + 1) * members + total - 1) / total) - 1; };
            const int first = u ? member_of(at) : 0, last = u ? member_of(at + u - 1) : 0;
            const Join jn{s, first, last, (int64_t)first * total / members < at};
            const unsigned below = (1u << lane) - 1;
            const unsigned f = __ballot_sync(~0u, last > first && last - first < kFewPieces);
            const unsigned g = __ballot_sync(~0u, last - first >= kFewPieces);
            if (lane == 0) {
                found[0][warp] = __popc(f);
                found[1][warp] = __popc(g);
            }
            __syncthreads();
            int nf = few + __popc(f & below), nm = many + __popc(g & below);
            for (int w = 0; w < kJoinWarps; ++w) {
                if (w < warp) {
                    nf += found[0][w];
                    nm += found[1][w];
                }
                few += found[0][w];
                many += found[1][w];
            }
            if (f >> lane & 1) list[nf] = jn;
            if (g >> lane & 1) list[kMaxJoins - 1 - nm] = jn;
        }
    }
    __syncthreads();
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // The slot of piece k of a sequence in a group of rows.
    auto slot_of = [&](const Join& jn, int group, int k) {
        return 2 * ((int64_t)(jn.member + k) * p.groups + group) + (k == 0 ? jn.second : 0);
    };
    const int per_row = p.R / 8;                             // threads a row
    const int64_t slot_floats = (int64_t)NB * (2 + p.R);
    const int steps = (NB * per_row + kJoinThreads - 1) / kJoinThreads;
    for (int it = blockIdx.x; it < few * p.groups * steps; it += gridDim.x) {
        const Join jn = list[it / steps / p.groups];
        const int group = it / steps % p.groups, pieces = jn.last - jn.member + 1;
        const int at = it % steps * kJoinThreads + threadIdx.x;
        const int row = at / per_row, e = at % per_row * 8, r = group * NB + row;
        if (row >= NB || r >= p.rows) continue;
        float top = -INFINITY, l = 0.0f;
        float4 o0 = make_float4(0, 0, 0, 0), o1 = o0;
        for (int k0 = 0; k0 < pieces; k0 += 4) {
            float mx[4], lx[4];
            float4 v[4][2];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int k = k0 + q;
                mx[q] = -INFINITY;
                lx[q] = 0.0f;
                v[q][0] = v[q][1] = make_float4(0, 0, 0, 0);
                if (k < pieces && dbg_in_bytes(p.parts + slot_of(jn, group, k) * slot_floats, 4 * slot_floats, p.sw,
                                               &g_wait_status)) {
                    const float* src = p.parts + slot_of(jn, group, k) * slot_floats;
                    mx[q] = src[row];
                    lx[q] = src[NB + row];
                    const float4* o = reinterpret_cast<const float4*>(src + 2 * NB + (int64_t)row * p.R + e);
                    v[q][0] = o[0];
                    v[q][1] = o[1];
                }
            }
            float now = top;
#pragma unroll
            for (int q = 0; q < 4; ++q) now = fmaxf(now, mx[q]);
            const float f = top == -INFINITY ? 0.0f : exp2f(top - now);
            l *= f;
            o0 = scale4(o0, f);
            o1 = scale4(o1, f);
            top = now;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float w = mx[q] == -INFINITY ? 0.0f : exp2f(mx[q] - top);
                l = fmaf(w, lx[q], l);
                add4(o0, w, v[q][0]);
                add4(o1, w, v[q][1]);
            }
        }
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        T* out = static_cast<T*>(p.O) + jn.seq * p.bsO + r / p.heads * p.tsO + r % p.heads * p.hsO + e;
        if (!dbg_in_bytes(out, 8 * sizeof(T), p.so, &g_wait_status)) continue;
        store4(out, scale4(o0, inv), p.o_vec);
        store4(out + 4, scale4(o1, inv), p.o_vec);
    }
    const int quarters = p.R / 128;
    for (int it = blockIdx.x; it < many * p.groups * NB * quarters; it += gridDim.x) {
        const Join jn = list[kMaxJoins - 1 - it / (NB * quarters) / p.groups];
        const int group = it / (NB * quarters) % p.groups, pieces = jn.last - jn.member + 1;
        const int row = it / quarters % NB, e = it % quarters * 128 + lane * 4, r = group * NB + row;
        if (r >= p.rows) continue;
        auto piece = [&](int k) { return p.parts + slot_of(jn, group, k) * slot_floats; };
        // This warp's pieces: a running maximum over groups of four.
        float top = -INFINITY, l = 0.0f;
        float4 o = make_float4(0, 0, 0, 0);
        for (int k0 = warp; k0 < pieces; k0 += 32) {
            float mx[4], lx[4];
            float4 v[4];
            float now = top;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int k = k0 + 8 * q;
                mx[q] = -INFINITY;
                lx[q] = 0.0f;
                v[q] = make_float4(0, 0, 0, 0);
                if (k < pieces && dbg_in_bytes(piece(k), 4 * slot_floats, p.sw, &g_wait_status)) {
                    const float* src = piece(k);
                    mx[q] = src[row];
                    lx[q] = src[NB + row];
                    v[q] = *reinterpret_cast<const float4*>(src + 2 * NB + (int64_t)row * p.R + e);
                }
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) now = fmaxf(now, mx[q]);
            const float f = top == -INFINITY ? 0.0f : exp2f(top - now);
            l *= f;
            o = scale4(o, f);
            top = now;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float w = mx[q] == -INFINITY ? 0.0f : exp2f(mx[q] - top);
                l = fmaf(w, lx[q], l);
                add4(o, w, v[q]);
            }
        }
        __syncthreads();                                     // the last item's sums are read
        sums[warp][lane] = o;
        if (lane == 0) {
            tops[warp] = top;
            ls[warp] = l;
        }
        __syncthreads();
        if (warp == 0) {
            top = -INFINITY;
            for (int k = 0; k < 8; ++k) top = fmaxf(top, tops[k]);
            l = 0.0f;
            o = make_float4(0, 0, 0, 0);
            for (int k = 0; k < 8; ++k) {
                const float w = tops[k] == -INFINITY ? 0.0f : exp2f(tops[k] - top);
                l = fmaf(w, ls[k], l);
                add4(o, w, sums[k][lane]);
            }
            const float inv = l == 0.0f ? 0.0f : 1.0f / l;
            T* out = static_cast<T*>(p.O) + jn.seq * p.bsO + r / p.heads * p.tsO + r % p.heads * p.hsO + e;
            if (dbg_in_bytes(out, 4 * sizeof(T), p.so, &g_wait_status)) store4(out, scale4(o, inv), p.o_vec);
        }
    }
}

int rows_block(int64_t rows) { return rows <= 16 ? 16 : rows <= 32 ? 32 : 64; }

size_t part_bytes(int nb, int64_t R) { return (size_t)nb * (2 + R) * 4; }

template <typename T, int NB>
cudaError_t launch(const CUtensorMap& map, const Params& p, int sms, cudaStream_t stream) {
    static std::atomic<uint64_t> attr_done{0};
    constexpr size_t most_bytes = smem_bytes<NB>(kMaxChunks);
    static_assert(most_bytes <= 232448, "shared memory per CTA");
    int dev = 0;
    cudaGetDevice(&dev);
    const uint64_t bit = 1ull << (dev & 63);
    if (!(attr_done.load() & bit)) {
        const cudaError_t e = cudaFuncSetAttribute(decode_kernel<T, NB>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   (int)most_bytes);
        if (e != cudaSuccess) return e;
        attr_done.fetch_or(bit);
    }
    decode_kernel<T, NB><<<(unsigned)(p.groups * p.per_group), kThreads, smem_bytes<NB>(p.chunks), stream>>>(map, p);
    cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess && p.split) {
        cudaLaunchAttribute early{};
        early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
        early.val.programmaticStreamSerializationAllowed = 1;
        cudaLaunchConfig_t cfg{};
        // No more blocks than there can be rows to join.
        const int64_t most = (int64_t)std::min(p.n_seqs, p.per_group - 1) * p.groups * NB * (p.R / 128);
        cfg.gridDim = dim3((unsigned)std::min<int64_t>((int64_t)sms * kJoinBlocks<NB>, most));
        cfg.blockDim = dim3(kJoinThreads);
        cfg.stream = stream;
        cfg.attrs = &early;
        cfg.numAttrs = 1;
        e = cudaLaunchKernelEx(&cfg, join_kernel<T, NB>, p);
    }
    return e;
}

template <typename T>
cudaError_t launch_rows(int nb, const CUtensorMap& map, const Params& p, int sms, cudaStream_t stream) {
    if (nb == 16) return launch<T, 16>(map, p, sms, stream);
    if (nb == 32) return launch<T, 32>(map, p, sms, stream);
    return launch<T, 64>(map, p, sms, stream);
}

bool vec16(const void* base, int64_t a, int64_t b, int64_t c) {
    return reinterpret_cast<uintptr_t>(base) % 16 == 0 && a % 8 == 0 && b % 8 == 0 && c % 8 == 0;
}

}  // namespace

size_t latent_decode_workspace_bytes(int sms) { return 2 * (size_t)sms * part_bytes(64, 512); }

bool launch_latent_decode(const LatentPaged& a, int sms, cudaStream_t stream, cudaError_t* err) {
    if (a.R % 128 != 0 || a.R > 512 || a.P % 8 != 0 || a.P > 64) return false;
    if (!vec16(a.Q, a.heads > 1 ? a.hsQ : 0, a.q_len > 1 ? a.tsQ : 0, a.n_seqs > 1 ? a.bsQ : 0) ||
        !vec16(a.cache, a.block_size > 1 ? a.rsC : 0, a.num_blocks > 1 ? a.psC : 0, 0))
        return false;
    const int64_t rows = a.q_len * a.heads;
    const int nb = rows_block(rows);
    const int64_t groups = (rows + nb - 1) / nb;
    if (groups > 65535 || (__int128)a.n_seqs * (a.N / 32 + 1) >= INT32_MAX) return false;
    Params p{};
    p.Q = a.Q; p.hsQ = a.hsQ; p.tsQ = a.tsQ; p.bsQ = a.bsQ;
    p.cache = a.cache; p.rsC = a.rsC; p.psC = a.psC;
    p.table = a.table; p.seq_lens = a.seq_lens;
    p.O = a.O; p.hsO = a.hsO; p.tsO = a.tsO; p.bsO = a.bsO;
    p.max_blocks = a.max_blocks;
    p.num_blocks = (int)a.num_blocks; p.block_size = (int)a.block_size;
    p.q_len = (int)a.q_len; p.heads = (int)a.heads; p.rows = (int)rows;
    p.N = (int)a.N; p.R = (int)a.R; p.P = (int)a.P; p.n_seqs = (int)a.n_seqs;
    p.o_vec = reinterpret_cast<uintptr_t>(a.O) % 8 == 0 && a.hsO % 4 == 0 && a.tsO % 4 == 0 && a.bsO % 4 == 0;
    p.chunks = (int)(a.R / 64 + (a.P > 0));
    p.rope_steps = (int)((a.P + 15) / 16);
    p.groups = (int)groups;
    p.scale_log2 = a.alpha * 1.4426950408889634f;
    p.causal = a.causal;
    p.sq = a.sq; p.sc = a.sc; p.so = a.so;
    p.sw = ByteSpan{reinterpret_cast<uintptr_t>(a.workspace), reinterpret_cast<uintptr_t>(a.workspace) + a.workspace_bytes};
    const bool bf = a.type == SBGEMM_TYPE_BF16;
    p.idesc_s = idesc16(bf, nb, false, false, 64);
    p.idesc_o = idesc16(bf, nb, true, true);
    // Runs of rows that lie in one page wherever a block begins; whole groups
    // of 8 rows, the swizzle's period.
    CUtensorMap map{};
    int run = nb == 64 ? Shape<64>::BT : Shape<32>::BT;
    for (const int bt = run; a.block_size % run != 0 || bt % run != 0;) --run;
    const int64_t row_stride = a.block_size > 1 ? a.rsC : (a.R + a.P + 7) / 8 * 8;
    const int64_t page_stride = a.num_blocks > 1 ? a.psC : row_stride;
    const int64_t lim = (int64_t)1 << 39;
    if (run % 8 == 0 && row_stride > 0 && page_stride > 0 && row_stride < lim && page_stride < lim) {
        const uint64_t dims[3] = {(uint64_t)(a.R + a.P), (uint64_t)a.block_size, (uint64_t)a.num_blocks};
        const uint64_t strides[2] = {(uint64_t)row_stride * 2, (uint64_t)page_stride * 2};
        const uint32_t box[3] = {64, (uint32_t)run, 1};
        if (!encode_tmap_16(&map, a.cache, 3, dims, strides, box)) {
            *err = cudaErrorInvalidValue;
            return true;
        }
        p.run = run;
    }
    // CTAs for each group of rows: an SM each, as far as the workspace has two
    // slots for every one of them; without it whole sequences.
    int64_t each = std::max<int64_t>(1, sms / groups);
    const int64_t slots = a.workspace ? (int64_t)(a.workspace_bytes / part_bytes(nb, a.R)) : 0;
    each = std::min(each, slots / (2 * groups));
    if (each > 1 && each * groups <= kMaxJoins) {
        p.split = 1;
        p.parts = static_cast<float*>(a.workspace);
    } else {
        each = std::min<int64_t>(std::max<int64_t>(1, sms / groups), a.n_seqs);
    }
    p.per_group = (int)each;
    *err = bf ? launch_rows<__nv_bfloat16>(nb, map, p, sms, stream)
              : launch_rows<__half>(nb, map, p, sms, stream);
    return true;
}

unsigned int* status_word_latent_decode() { return word_address(&g_wait_status); }

}  // namespace sbg
