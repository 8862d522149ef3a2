// The 16-bit strided product on the tensor cores (sbgemm_half): C = alpha A B
// (+ C), fp32 accumulation in TMEM, for operands that a tensor map describes.
//
// Persistent CTAs, one an SM, over tiles of 128 x NT outputs.  A tile's 128
// rows (the MMA's M) are rows of C, or columns of C (the product computed as
// C^T = B^T A^T), whichever pads and reads less: a decode batch has few rows
// of C, and then the weights fill the MMA's M and the tokens its N.  K goes by
// in blocks of 64 (one 128-byte swizzled row) through a ring of TMA stages
// that runs on over the tiles; either operand may be unit-stride along K or
// along its other index, the MMA reads both orders from the same swizzled
// boxes, so no layout is transposed on the way.
//
// Roles: warp 8 issues the TMA loads, warp 9 the MMAs, warps 0-3 and 4-7 take
// the accumulator (one of two in TMEM, so that the next tile's MMAs run
// meanwhile) in turns of 64 columns, round it once and send it out by TMA
// through swizzled 16 KB buffers, two for each group (128 products of
// 64 x 512 x 128: 8.3 us, 10.3 with one buffer each); a C without a
// tensor map, or one that is added to, goes straight from registers.
//
// Products of long K run on CTA pairs (cta_group::2): one MMA of 256 x 256 x 16
// over both CTAs' shared memory, each holding its 128 rows of the tile and half
// of its columns' operand.  Alone, a 128 x 256 tile moves 24 KB through shared
// memory a K step (12 KB in by TMA, 12 KB out to the MMA), 192 of its cycles for
// 130 of the MMA's; a pair's CTA moves 16 KB.  bf16: 4096 x 4096 x 4096 96 us on
// single CTAs, 86 on pairs; 8192 x 8192 x 2048 with an N-major B 194 and 174;
// but 4096 x 8192 x 512 31 and 32, and 128 products of 512 x 512 x 128 24 and
// 29, the pair's two epilogues ending together: hence pairs from K = 1024.
//
// Bound: at K of a few hundred by the bytes of A, B and C; each tile reads
// (128 + NT) K elements from L2 for 128 NT K products.
#include <algorithm>
#include <atomic>

#include "debug_check.cuh"
#include "serving.h"
#include "tc16.cuh"

namespace sbg {
namespace {

constexpr int BX = 128, BK = 64;
constexpr int kGroups = 2, kTmaWarp = 4 * kGroups, kMmaWarp = kTmaWarp + 1;
constexpr int kThreads = (kMmaWarp + 1) * 32;
constexpr int kOutBytes = 128 * 64 * 2;      // one buffer of the way out
__device__ unsigned int g_wait_status = 0;

struct Params {
    void* C; int64_t rsC, bsC;     // unit stride along C's columns
    int64_t rows, cols;            // of C
    int64_t x_tiles, y_tiles, tiles;
    int k_blocks;
    float alpha;
    int accumulate, swapped;       // swapped: the MMA's M runs along C's columns
    int x_mn, y_mn;                // operand unit-stride along M / N instead of K
    int x_batch, y_batch;          // the batch coordinate moves (else shared)
    int c_tma;                     // C goes out through its tensor map
    uint32_t idesc;
    ByteSpan sc;                   // debug builds: what C occupies
};

template <int NT, bool kPair>
struct Shape {
    static constexpr int kYRows = kPair ? NT / 2 : NT;              // this CTA's share
    static constexpr int kYBytes = (kYRows < 64 ? 64 : kYRows) * BK * 2;    // an MN-major box is 64 wide
    static constexpr int kStage = BX * BK * 2 + kYBytes;
    static constexpr int kStages = kYRows == 256 ? 4 : kYRows == 128 ? 5 : 6;
    static constexpr int kBufs = kYRows == 256 ? 1 : 2;             // on the way out, for each group
    // With 256 columns a fourth stage and a second buffer do not both fit; up to
    // three blocks of K have no use for the stage (128 products of 64 x 512 x
    // 128: 10.3 us with four stages, 8.3 with two buffers; 4099 x 8192 x 512:
    // 30.8 and 33.8).
    __host__ __device__ static constexpr int stages(int k_blocks) { return kYRows == 256 && k_blocks <= 3 ? 3 : kStages; }
    __host__ __device__ static constexpr int bufs(int k_blocks) { return kYRows == 256 && k_blocks <= 3 ? 2 : kBufs; }
    static constexpr int kSmem = kStages * kStage + kBufs * kGroups * kOutBytes + 1024;
    static_assert(kSmem <= 232448 - 1024, "shared memory per CTA");
};

// Barriers of the four warps of an epilogue group.
__device__ __forceinline__ void group_sync(int g) { asm volatile("bar.sync %0, 128;" ::"r"(1 + g) : "memory"); }
__device__ __forceinline__ bool all_of_group(int g, bool v) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred a, b;\n\tsetp.ne.b32 a, %1, 0;\n\t"
        "barrier.cta.red.and.pred b, %2, 128, a;\n\tselp.u32 %0, 1, 0, b;\n\t}"
        : "=r"(r) : "r"((uint32_t)v), "r"(1 + g) : "memory");
    return r != 0;
}

template <typename T, int NT, bool kPair>
__global__ void __launch_bounds__(kThreads, 1)
half_tc_kernel(const __grid_constant__ CUtensorMap tx, const __grid_constant__ CUtensorMap ty,
               const __grid_constant__ CUtensorMap to, const __grid_constant__ Params p) {
    using S = Shape<NT, kPair>;
    constexpr int kCtas = kPair ? 2 : 1;
    const int rank = kPair ? (int)(cluster_rank() & 1) : 0;
    extern __shared__ uint8_t raw[];
    uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
    const int stages = S::stages(p.k_blocks), bufs = S::bufs(p.k_blocks);
    uint8_t* out = ring + stages * S::kStage;
    __shared__ uint64_t full[S::kStages], empty[S::kStages], acc_full[2], acc_free[2], done;
    __shared__ uint32_t tmem_base;
    const int warp = uniform_warp(), lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S::kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&acc_full[i], 1);
            mbar_init(&acc_free[i], 4 * kGroups * kCtas);
        }
        mbar_init(&done, 1);
        fence_mbar_init_cluster();
        prefetch_tensormap(&tx);
        prefetch_tensormap(&ty);
        if (p.c_tma) prefetch_tensormap(&to);
    }
    if (warp == kMmaWarp) {
        if constexpr (kPair) {
            tmem_alloc_pair(&tmem_base, kTmemAll);
            tmem_relinquish_pair();
        } else {
            tmem_alloc(&tmem_base, kTmemAll);
            tmem_relinquish();
        }
    }
    tc_fence_before();
    __syncthreads();
    // A pair's barriers and TMEM are there in both CTAs before either uses the other's.
    if constexpr (kPair) cluster_sync();
    tc_fence_after();
    const int64_t first = blockIdx.x / kCtas, stride = gridDim.x / kCtas;
    // Tile t: x fastest, so that CTAs side by side share the Y operand's tile.
    auto place = [&](int64_t t, int* x0, int* y0, int* b) {
        *x0 = (int)(t % p.x_tiles) * (BX * kCtas) + BX * rank;
        *y0 = (int)(t / p.x_tiles % p.y_tiles) * NT;
        *b = (int)(t / p.x_tiles / p.y_tiles);
    };

    if (warp == kTmaWarp) {
        if (lane == 0) {
            const int y_boxes = p.y_mn ? (S::kYRows + 63) / 64 : 1;
            const uint32_t bytes = BX * BK * 2 + (p.y_mn ? y_boxes * 64 : S::kYRows) * BK * 2;
            // A pair's copies all complete on its first CTA's barriers.
            auto load = [&](void* dst, const CUtensorMap* map, int s, int c0, int c1, int c2) {
                if constexpr (kPair) tma_load_3d_pair(dst, map, cluster_addr(&full[s], 0), c0, c1, c2);
                else tma_load_3d(dst, map, &full[s], c0, c1, c2);
            };
            // Stage and round of the ring, by counting (a division a block of K is
            // what such a loop has no time for).
            int s = 0, issued = 0;
            uint32_t round = 0;
            bool ok = true;
            for (int64_t t = first; t < p.tiles && ok; t += stride) {
                int x0, y0, b;
                place(t, &x0, &y0, &b);
                const int zx = p.x_batch ? b : 0, zy = p.y_batch ? b : 0;
                for (int j = 0; j < p.k_blocks; ++j) {
                    if (round > 0 && !bar_wait(&empty[s], (round - 1) & 1)) {
                        record_status(&g_wait_status, kWaitEmpty);
                        ok = false;
                        break;
                    }
                    uint8_t* x = ring + s * S::kStage;
                    uint8_t* y = x + BX * BK * 2;
                    if (rank == 0) mbar_arrive_expect_tx(&full[s], bytes * kCtas);
                    if (p.x_mn) {
                        load(x, &tx, s, x0, j * BK, zx);
                        load(x + 64 * BK * 2, &tx, s, x0 + 64, j * BK, zx);
                    } else {
                        load(x, &tx, s, j * BK, x0, zx);
                    }
                    const int yr = y0 + S::kYRows * rank;
                    if (p.y_mn) {
                        for (int q = 0; q < y_boxes; ++q)
                            load(y + q * 64 * BK * 2, &ty, s, yr + 64 * q, j * BK, zy);
                    } else {
                        load(y, &ty, s, j * BK, yr, zy);
                    }
                    if (issued < stages) ++issued;
                    if (++s == stages) {
                        s = 0;
                        ++round;
                    }
                }
            }
            // Copies still landing keep the CTA's shared memory (a pair's first
            // CTA waits for both).
            for (int q = 0; rank == 0 && q < issued; ++q) {
                if (--s < 0) {
                    s = stages - 1;
                    --round;
                }
                if (!bar_wait(&full[s], round & 1)) {
                    record_status(&g_wait_status, kWaitDrain);
                    break;
                }
            }
        }
    } else if (warp == kMmaWarp) {
        if (rank == 0 && elect_one()) {
            const uint32_t x_step = p.x_mn ? kStepMN : kStepK, y_step = p.y_mn ? kStepMN : kStepK;
            int s = 0, n = 0;                      // stage; tiles begun
            uint32_t round = 0;
            bool ok = true;
            for (int64_t t = first; t < p.tiles && ok; t += stride, ++n) {
                if (n >= 2) {
                    const uint32_t ph = (uint32_t)((n / 2 - 1) & 1);
                    if (!(kPair ? mbar_wait_cluster(&acc_free[n & 1], ph) : bar_wait(&acc_free[n & 1], ph))) {
                        record_status(&g_wait_status, kWaitAccFree);
                        break;
                    }
                    tc_fence_after();
                }
                const uint32_t acc = kTmemBase + (uint32_t)(n & 1) * NT;
                for (int j = 0; j < p.k_blocks; ++j) {
                    if (!bar_wait(&full[s], round & 1)) {
                        record_status(&g_wait_status, kWaitFull);
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t x = smem_u32(ring + s * S::kStage);
                    uint64_t dx = desc16(x, 64 * BK * 2), dy = desc16(x + BX * BK * 2, 64 * BK * 2);
#pragma unroll
                    for (int k = 0; k < BK / 16; ++k) {
                        if constexpr (kPair) mma16_ss_pair(acc, dx, dy, p.idesc, (j | k) ? 1u : 0u);
                        else mma16_ss(acc, dx, dy, p.idesc, (j | k) ? 1u : 0u);
                        dx += x_step;
                        dy += y_step;
                    }
                    if constexpr (kPair) mma_commit_pair_both(&empty[s]);
                    else mma_commit(&empty[s]);
                    if (++s == stages) {
                        s = 0;
                        ++round;
                    }
                }
                if (!ok) break;
                if constexpr (kPair) mma_commit_pair_both(&acc_full[n & 1]);
                else mma_commit(&acc_full[n & 1]);
            }
            // Nothing may still be writing TMEM when it is freed.
            if constexpr (kPair) mma_commit_pair_local(&done);
            else mma_commit(&done);
            if (!bar_wait(&done, 0)) record_status(&g_wait_status, kWaitMma);
        }
    } else {
        // The way out in chunks of 64 accumulator columns (32 where NT is).
        constexpr int kChunk = NT < 64 ? NT : 64;
        constexpr int kHalves = kChunk / 32;
        const int g = warp >> 2, row = threadIdx.x & 127;
        int n = 0, sent = 0;
        for (int64_t t = first; t < p.tiles; t += stride, ++n) {
            int x0, y0, b;
            place(t, &x0, &y0, &b);
            const bool in = bar_wait(&acc_full[n & 1], (uint32_t)((n / 2) & 1));
            if (!in) record_status(&g_wait_status, kWaitMma);
            if (!all_of_group(g, in)) break;          // they meet at barriers below: all go on or none
            tc_fence_after();
            const uint32_t acc = kTmemBase + (uint32_t)(n & 1) * NT + ((uint32_t)((warp & 3) * 32) << 16);
            const int x = x0 + row;
            T* C = static_cast<T*>(p.C) + b * p.bsC;
#pragma unroll 1
            for (int c = g * kChunk; c < NT; c += kGroups * kChunk) {
                uint8_t* buf = out + (bufs * g + (bufs == 2 ? sent & 1 : 0)) * kOutBytes;
                if (p.c_tma) {
                    // The buffer's last store has read it.
                    if (row == 0) {
                        if (bufs == 2) bulk_wait_read_all_but_one();
                        else bulk_wait_read_all();
                    }
                    group_sync(g);
                }
#pragma unroll
                for (int h = 0; h < kHalves; ++h) {
                    float v[32];
                    tmem_ld<32>(acc + c + 32 * h, v);
                    if (!p.c_tma) {
                        // No tensor map, or added to C: rounded once, element by element.
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            const int y = y0 + c + 32 * h + i;
                            const int64_t m = p.swapped ? y : x, nn = p.swapped ? x : y;
                            if (m < p.rows && nn < p.cols) {
                                T* o = C + m * p.rsC + nn;
                                if (!dbg_in_bytes(o, sizeof(T), p.sc, &g_wait_status)) continue;
                                *o = from_float<T>(p.accumulate ? fmaf(p.alpha, v[i], to_float(*o)) : p.alpha * v[i]);
                            }
                        }
                    } else if (p.swapped) {
                        // Two boxes [kChunk rows of C][64 columns]: this thread's column.
                        uint8_t* box = buf + (row >> 6) * (kChunk * 128);
                        const uint32_t at = (row & 63) * 2;
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            const uint32_t r = 32 * h + i;
                            *reinterpret_cast<T*>(box + r * 128 + (at ^ ((r & 7) << 4))) = from_float<T>(p.alpha * v[i]);
                        }
                    } else {
                        // One box [128 rows of C][64 columns]: this thread's row.
                        const uint32_t r = row;
#pragma unroll
                        for (int i = 0; i < 32; i += 8)
                            *reinterpret_cast<uint4*>(buf + r * 128 + ((uint32_t)((32 * h + i) * 2) ^ ((r & 7) << 4))) =
                                make_uint4(pack2<T>(p.alpha * v[i], p.alpha * v[i + 1]),
                                           pack2<T>(p.alpha * v[i + 2], p.alpha * v[i + 3]),
                                           pack2<T>(p.alpha * v[i + 4], p.alpha * v[i + 5]),
                                           pack2<T>(p.alpha * v[i + 6], p.alpha * v[i + 7]));
                    }
                }
                if (p.c_tma) {
                    fence_proxy_async_smem();
                    group_sync(g);
                    if (row == 0) {
                        const int y = y0 + c;
                        if (p.swapped) {
                            if (y < p.rows && x0 < p.cols) {
                                tma_store_3d(&to, buf, x0, y, b);
                                if (x0 + 64 < p.cols) tma_store_3d(&to, buf + kChunk * 128, x0 + 64, y, b);
                            }
                        } else if (y < p.cols && x0 < p.rows) {
                            tma_store_3d(&to, buf, y, x0, b);
                        }
                        bulk_commit();
                    }
                    ++sent;
                }
            }
            // The group's share of the accumulator is read.
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (kPair && rank != 0) mbar_arrive_remote(&acc_free[n & 1], 0);
                else mbar_arrive(&acc_free[n & 1]);
            }
        }
        if (p.c_tma && row == 0) bulk_wait_read_all();   // shared memory outlives the stores' reads
    }
    tc_fence_before();
    __syncthreads();
    // Neither CTA of a pair leaves while the other may use its memory.
    if constexpr (kPair) cluster_sync();
    if (warp == kMmaWarp) {
        tc_fence_after();
        if constexpr (kPair) tmem_dealloc_pair(kTmemBase, kTmemAll);
        else tmem_dealloc(kTmemBase, kTmemAll);
    }
}

// An operand as [batch][outer][inner] with a unit stride along inner.
struct View { const void* base; int64_t inner, outer, outer_stride, batch, batch_stride; };

bool mappable(const View& v) {
    if (reinterpret_cast<uintptr_t>(v.base) % 16 != 0) return false;
    const int64_t lim = (int64_t)1 << 31;
    if (v.inner >= lim || v.outer >= lim || v.batch >= lim) return false;
    auto ok = [](int64_t s) { return s > 0 && s % 8 == 0 && s < ((int64_t)1 << 39); };
    if (v.outer > 1 && !ok(v.outer_stride)) return false;
    return v.batch == 1 || v.batch_stride == 0 || ok(v.batch_stride);
}

bool make_map(CUtensorMap* map, const View& v, uint32_t box_outer) {
    const bool moves = v.batch > 1 && v.batch_stride != 0;
    const uint64_t inner_bytes = (uint64_t)(v.inner * 2 + 15) / 16 * 16;
    const uint64_t dims[3] = {(uint64_t)v.inner, (uint64_t)v.outer, moves ? (uint64_t)v.batch : 1};
    const uint64_t so = v.outer > 1 ? (uint64_t)v.outer_stride * 2 : inner_bytes;
    const uint64_t strides[2] = {so, moves ? (uint64_t)v.batch_stride * 2 : so};
    const uint32_t box[3] = {64, box_outer, 1};
    return encode_tmap_16(map, v.base, 3, dims, strides, box);
}

// Operand rows x K with strides (rs, cs, bs): K-major or MN-major view.
bool view_of(const void* base, int64_t rows, int64_t K, int64_t rs, int64_t cs, int64_t bs, int64_t batch, View* v,
             bool* mn) {
    *v = View{base, K, rows, rs, batch, bs};
    *mn = false;
    if ((cs == 1 || K == 1) && mappable(*v)) return true;
    *v = View{base, rows, K, cs, batch, bs};
    *mn = true;
    return (rs == 1 || rows == 1) && mappable(*v);
}

// C^T = B^T A^T as a problem of its own.
HalfProblem transposed(const HalfProblem& p) {
    HalfProblem t = p;
    t.A = p.B; t.rsA = p.csB; t.csA = p.rsB; t.bsA = p.bsB;
    t.B = p.A; t.rsB = p.csA; t.csB = p.rsA; t.bsB = p.bsA;
    t.rsC = p.csC; t.csC = p.rsC;
    t.M = p.N; t.N = p.M;
    return t;
}

template <typename T, int NT, bool kPair>
cudaError_t launch(const Params& p, const CUtensorMap& tx, const CUtensorMap& ty, const CUtensorMap& to, int sms,
                   cudaStream_t stream) {
    using S = Shape<NT, kPair>;
    static std::atomic<int> ready[64];           // 0: not asked yet; else the CTAs (or pairs) that fit, or -1
    int dev = 0;
    cudaGetDevice(&dev);
    cudaLaunchConfig_t cfg{};
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = S::kSmem;
    cfg.stream = stream;
    cudaLaunchAttribute cluster{};
    cluster.id = cudaLaunchAttributeClusterDimension;
    cluster.val.clusterDim.x = 2;
    cluster.val.clusterDim.y = cluster.val.clusterDim.z = 1;
    cfg.attrs = &cluster;
    cfg.numAttrs = kPair ? 1 : 0;
    int fit = ready[dev & 63].load();
    if (fit == 0) {
        const cudaError_t e = cudaFuncSetAttribute(half_tc_kernel<T, NT, kPair>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
        if (e != cudaSuccess) return e;
        fit = sms;
        if (kPair) {
            cfg.gridDim = dim3((unsigned)(sms / 2 * 2));
            if (cudaOccupancyMaxActiveClusters(&fit, half_tc_kernel<T, NT, kPair>, &cfg) != cudaSuccess || fit <= 0) {
                cudaGetLastError();
                fit = sms / 2;
            }
        }
        ready[dev & 63].store(fit);
    }
    cfg.gridDim = dim3((unsigned)(std::min<int64_t>(p.tiles, fit) * (kPair ? 2 : 1)));
    return cudaLaunchKernelEx(&cfg, half_tc_kernel<T, NT, kPair>, tx, ty, to, p);
}

template <typename T>
cudaError_t launch_nt(int nt, bool pair, const Params& p, const CUtensorMap& tx, const CUtensorMap& ty,
                      const CUtensorMap& to, int sms, cudaStream_t stream) {
    if (pair) return launch<T, 256, true>(p, tx, ty, to, sms, stream);
    switch (nt) {
        case 32: return launch<T, 32, false>(p, tx, ty, to, sms, stream);
        case 64: return launch<T, 64, false>(p, tx, ty, to, sms, stream);
        case 128: return launch<T, 128, false>(p, tx, ty, to, sms, stream);
        default: return launch<T, 256, false>(p, tx, ty, to, sms, stream);
    }
}

}  // namespace

// The tile's N and orientation, and single CTAs or pairs: the fewest elements
// read by an SM, (128 + its columns) a tile, over the waves of tiles; a pair's
// tile counts as 340 for the times above.
bool launch_half_tc(const HalfProblem& given, int sms, cudaStream_t stream, cudaError_t* err) {
    // Unit stride along C's columns.
    const HalfProblem p = given.csC == 1 || given.N == 1 ? given : transposed(given);
    if (!(p.csC == 1 || p.N == 1) || p.K <= 0) return false;
    View va, vb;
    bool a_mn, b_mn;
    if (!view_of(p.A, p.M, p.K, p.rsA, p.csA, p.bsA, p.batch, &va, &a_mn) ||
        !view_of(p.B, p.N, p.K, p.csB, p.rsB, p.bsB, p.batch, &vb, &b_mn))
        return false;
    int64_t best = 0;
    int nt = 0;
    bool swapped = false, pair = false;
    Params q{};
    for (int s = 0; s < 2; ++s)
        for (int n : {32, 64, 128, 256, 512}) {
            if (!s && n == 32) continue;       // an upright box on the way out is 64 columns wide
            const bool two = n == 512;         // a pair's tile of 256 x 256
            if (two && p.K < 1024) continue;
            const int64_t bx = two ? 2 * BX : BX, by = two ? 256 : n;
            const int64_t xs = ((s ? p.N : p.M) + bx - 1) / bx, ys = ((s ? p.M : p.N) + by - 1) / by;
            if ((double)xs * (double)ys * (double)p.batch > 1e15) return false;
            const int64_t at_once = two ? sms / 2 : sms;
            const int64_t cost = (xs * ys * p.batch + at_once - 1) / at_once * (two ? 340 : BX + n);
            if (nt == 0 || cost < best) {
                best = cost;
                nt = (int)by;
                pair = two;
                swapped = s != 0;
                q.x_tiles = xs;
                q.y_tiles = ys;
                q.tiles = xs * ys * p.batch;
            }
        }
    const View& vx = swapped ? vb : va;
    const View& vy = swapped ? va : vb;
    q.x_mn = swapped ? b_mn : a_mn;
    q.y_mn = swapped ? a_mn : b_mn;
    CUtensorMap tx, ty, to{};
    const View vc{p.C, p.N, p.M, p.rsC, p.batch, p.bsC};
    // Bulk stores clip a row of C to whole 16-byte pieces.
    q.c_tma = !p.accumulate && p.N % 8 == 0 && mappable(vc) && (p.batch == 1 || p.bsC != 0);
    if (!make_map(&tx, vx, q.x_mn ? 64 : BX) || !make_map(&ty, vy, q.y_mn ? 64 : (uint32_t)(pair ? nt / 2 : nt)) ||
        (q.c_tma && !make_map(&to, vc, swapped ? (uint32_t)(nt < 64 ? nt : 64) : BX))) {
        *err = cudaErrorInvalidValue;
        return true;
    }
    q.C = p.C; q.rsC = p.rsC; q.bsC = p.bsC; q.sc = p.sc;
    q.rows = p.M; q.cols = p.N;
    q.k_blocks = (int)((p.K + BK - 1) / BK);
    q.alpha = p.alpha;
    q.accumulate = p.accumulate;
    q.swapped = swapped;
    q.x_batch = p.batch > 1 && vx.batch_stride != 0;
    q.y_batch = p.batch > 1 && vy.batch_stride != 0;
    q.idesc = idesc16(p.type == SBGEMM_TYPE_BF16, nt, q.x_mn, q.y_mn, pair ? 256 : 128);
    *err = p.type == SBGEMM_TYPE_BF16 ? launch_nt<__nv_bfloat16>(nt, pair, q, tx, ty, to, sms, stream)
                                      : launch_nt<__half>(nt, pair, q, tx, ty, to, sms, stream);
    return true;
}

unsigned int* status_word_half_tc() { return word_address(&g_wait_status); }

}  // namespace sbg
