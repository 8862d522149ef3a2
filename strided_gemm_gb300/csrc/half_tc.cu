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
// Roles: warp 4 issues the TMA loads, warp 5 the MMAs, warps 0-3 take the
// accumulator (one of two in TMEM, so that the next tile's MMAs run meanwhile),
// round it once and send it out by TMA through a swizzled 16 KB buffer (two of
// them); a C without a tensor map, or one that is added to, goes straight from
// registers.
//
// Bound: at K of a few hundred by the bytes of A, B and C; each tile reads
// (128 + NT) K elements from L2 for 128 NT K products.
#include <algorithm>
#include <atomic>

#include "serving.h"
#include "tc16.cuh"

namespace sbg {
namespace {

constexpr int BX = 128, BK = 64;
constexpr int kThreads = 192;
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
};

template <int NT>
struct Shape {
    static constexpr int kYBytes = (NT < 64 ? 64 : NT) * BK * 2;    // an MN-major box is 64 wide
    static constexpr int kStage = BX * BK * 2 + kYBytes;
    static constexpr int kStages = NT == 256 ? 4 : NT == 128 ? 6 : 8;
    static constexpr int kSmem = kStages * kStage + 2 * kOutBytes + 1024;
    static_assert(kSmem <= 232448 - 1024, "shared memory per CTA");
};

// The four epilogue warps' own barrier.
__device__ __forceinline__ void group_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }
__device__ __forceinline__ bool all_of_group(bool v) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred a, b;\n\tsetp.ne.b32 a, %1, 0;\n\t"
        "barrier.cta.red.and.pred b, 1, 128, a;\n\tselp.u32 %0, 1, 0, b;\n\t}"
        : "=r"(r) : "r"((uint32_t)v) : "memory");
    return r != 0;
}

template <typename T, int NT>
__global__ void __launch_bounds__(kThreads, 1)
half_tc_kernel(const __grid_constant__ CUtensorMap tx, const __grid_constant__ CUtensorMap ty,
               const __grid_constant__ CUtensorMap to, const __grid_constant__ Params p) {
    using S = Shape<NT>;
    extern __shared__ uint8_t raw[];
    uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
    uint8_t* out = ring + S::kStages * S::kStage;
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
            mbar_init(&acc_free[i], 4);
        }
        mbar_init(&done, 1);
        fence_mbar_init();
        prefetch_tensormap(&tx);
        prefetch_tensormap(&ty);
        if (p.c_tma) prefetch_tensormap(&to);
    }
    if (warp == 5) {
        tmem_alloc(&tmem_base, kTmemAll);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // Tile t: x fastest, so that CTAs side by side share the Y operand's tile.
    auto place = [&](int64_t t, int* x0, int* y0, int* b) {
        *x0 = (int)(t % p.x_tiles) * BX;
        *y0 = (int)(t / p.x_tiles % p.y_tiles) * NT;
        *b = (int)(t / p.x_tiles / p.y_tiles);
    };

    if (warp == 4) {
        if (lane == 0) {
            const int y_boxes = p.y_mn ? (NT + 63) / 64 : 1;
            const uint32_t bytes = BX * BK * 2 + (p.y_mn ? y_boxes * 64 : NT) * BK * 2;
            int64_t i = 0;                         // blocks issued
            bool ok = true;
            for (int64_t t = blockIdx.x; t < p.tiles && ok; t += gridDim.x) {
                int x0, y0, b;
                place(t, &x0, &y0, &b);
                const int zx = p.x_batch ? b : 0, zy = p.y_batch ? b : 0;
                for (int j = 0; j < p.k_blocks; ++j, ++i) {
                    const int s = (int)(i % S::kStages);
                    if (i >= S::kStages && !bar_wait(&empty[s], (uint32_t)((i / S::kStages - 1) & 1))) {
                        record_status(&g_wait_status, kWaitEmpty);
                        ok = false;
                        break;
                    }
                    uint8_t* x = ring + s * S::kStage;
                    uint8_t* y = x + BX * BK * 2;
                    mbar_arrive_expect_tx(&full[s], bytes);
                    if (p.x_mn) {
                        tma_load_3d(x, &tx, &full[s], x0, j * BK, zx);
                        tma_load_3d(x + 64 * BK * 2, &tx, &full[s], x0 + 64, j * BK, zx);
                    } else {
                        tma_load_3d(x, &tx, &full[s], j * BK, x0, zx);
                    }
                    if (p.y_mn) {
                        for (int q = 0; q < y_boxes; ++q)
                            tma_load_3d(y + q * 64 * BK * 2, &ty, &full[s], y0 + 64 * q, j * BK, zy);
                    } else {
                        tma_load_3d(y, &ty, &full[s], j * BK, y0, zy);
                    }
                }
            }
            // Copies still landing keep the CTA's shared memory.
            for (int64_t q = i > S::kStages ? i - S::kStages : 0; q < i; ++q)
                if (!bar_wait(&full[q % S::kStages], (uint32_t)((q / S::kStages) & 1))) {
                    record_status(&g_wait_status, kWaitDrain);
                    break;
                }
        }
    } else if (warp == 5) {
        if (elect_one()) {
            const uint32_t x_step = p.x_mn ? kStepMN : kStepK, y_step = p.y_mn ? kStepMN : kStepK;
            int64_t i = 0;
            int n = 0;                             // tiles begun
            bool ok = true;
            for (int64_t t = blockIdx.x; t < p.tiles && ok; t += gridDim.x, ++n) {
                if (n >= 2 && !bar_wait(&acc_free[n & 1], (uint32_t)((n / 2 - 1) & 1))) {
                    record_status(&g_wait_status, kWaitAccFree);
                    break;
                }
                const uint32_t acc = kTmemBase + (uint32_t)(n & 1) * NT;
                for (int j = 0; j < p.k_blocks; ++j, ++i) {
                    const int s = (int)(i % S::kStages);
                    if (!bar_wait(&full[s], (uint32_t)((i / S::kStages) & 1))) {
                        record_status(&g_wait_status, kWaitFull);
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t x = smem_u32(ring + s * S::kStage);
                    uint64_t dx = desc16(x, 64 * BK * 2), dy = desc16(x + BX * BK * 2, 64 * BK * 2);
#pragma unroll
                    for (int k = 0; k < BK / 16; ++k) {
                        mma16_ss(acc, dx, dy, p.idesc, (j | k) ? 1u : 0u);
                        dx += x_step;
                        dy += y_step;
                    }
                    mma_commit(&empty[s]);
                }
                if (ok) mma_commit(&acc_full[n & 1]);
            }
            // Nothing may still be writing TMEM when it is freed.
            mma_commit(&done);
            if (!bar_wait(&done, 0)) record_status(&g_wait_status, kWaitMma);
        }
    } else {
        // The way out in chunks of 64 accumulator columns (32 where NT is).
        constexpr int kChunk = NT < 64 ? NT : 64;
        constexpr int kHalves = kChunk / 32;
        int n = 0, sent = 0;
        for (int64_t t = blockIdx.x; t < p.tiles; t += gridDim.x, ++n) {
            int x0, y0, b;
            place(t, &x0, &y0, &b);
            const bool in = bar_wait(&acc_full[n & 1], (uint32_t)((n / 2) & 1));
            if (!in) record_status(&g_wait_status, kWaitMma);
            if (!all_of_group(in)) break;          // they meet at barriers below: all go on or none
            tc_fence_after();
            const uint32_t acc = kTmemBase + (uint32_t)(n & 1) * NT + ((uint32_t)(warp * 32) << 16);
            const int x = x0 + threadIdx.x;
            T* C = static_cast<T*>(p.C) + b * p.bsC;
#pragma unroll 1
            for (int c = 0; c < NT; c += kChunk) {
                uint8_t* buf = out + (sent & 1) * kOutBytes;
                if (p.c_tma) {
                    // The buffer's last store (two chunks ago) has read it.
                    if (threadIdx.x == 0) bulk_wait_read_all_but_one();
                    group_sync();
                }
#pragma unroll
                for (int h = 0; h < kHalves; ++h) {
                    float v[32];
                    tmem_ld32(acc + c + 32 * h, v);
                    if (!p.c_tma) {
                        // No tensor map, or added to C: rounded once, element by element.
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            const int y = y0 + c + 32 * h + i;
                            const int64_t m = p.swapped ? y : x, nn = p.swapped ? x : y;
                            if (m < p.rows && nn < p.cols) {
                                T* o = C + m * p.rsC + nn;
                                *o = from_float<T>(p.accumulate ? fmaf(p.alpha, v[i], to_float(*o)) : p.alpha * v[i]);
                            }
                        }
                    } else if (p.swapped) {
                        // Two boxes [kChunk rows of C][64 columns]: this thread's column.
                        uint8_t* box = buf + (threadIdx.x >> 6) * (kChunk * 128);
                        const uint32_t at = (threadIdx.x & 63) * 2;
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            const uint32_t r = 32 * h + i;
                            *reinterpret_cast<T*>(box + r * 128 + (at ^ ((r & 7) << 4))) = from_float<T>(p.alpha * v[i]);
                        }
                    } else {
                        // One box [128 rows of C][64 columns]: this thread's row.
                        const uint32_t r = threadIdx.x;
#pragma unroll
                        for (int i = 0; i < 32; i += 8)
                            *reinterpret_cast<uint4*>(buf + r * 128 + ((uint32_t)((32 * h + i) * 2) ^ ((r & 7) << 4))) =
                                make_uint4(pack2<T>(p.alpha * v[i], p.alpha * v[i + 1]),
                                           pack2<T>(p.alpha * v[i + 2], p.alpha * v[i + 3]),
                                           pack2<T>(p.alpha * v[i + 4], p.alpha * v[i + 5]),
                                           pack2<T>(p.alpha * v[i + 6], p.alpha * v[i + 7]));
                    }
                }
                if (c + kChunk >= NT) {            // the accumulator is read: free it
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&acc_free[n & 1]);
                }
                if (p.c_tma) {
                    fence_proxy_async_smem();
                    group_sync();
                    if (threadIdx.x == 0) {
                        const int y = y0 + c;
                        if (p.swapped) {
                            if (y < p.rows) {
                                tma_store_3d(&to, buf, x0, y, b);
                                if (x0 + 64 < p.cols) tma_store_3d(&to, buf + kChunk * 128, x0 + 64, y, b);
                            }
                        } else if (y < p.cols) {
                            tma_store_3d(&to, buf, y, x0, b);
                        }
                        bulk_commit();
                    }
                    ++sent;
                }
            }
        }
        if (p.c_tma && threadIdx.x == 0) bulk_wait_read_all();   // shared memory outlives the stores' reads
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 5) {
        tc_fence_after();
        tmem_dealloc(kTmemBase, kTmemAll);
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

template <typename T, int NT>
cudaError_t launch(const Params& p, const CUtensorMap& tx, const CUtensorMap& ty, const CUtensorMap& to, int sms,
                   cudaStream_t stream) {
    static std::atomic<uint64_t> attr_done{0};
    int dev = 0;
    cudaGetDevice(&dev);
    const uint64_t bit = 1ull << (dev & 63);
    if (!(attr_done.load() & bit)) {
        const cudaError_t e = cudaFuncSetAttribute(half_tc_kernel<T, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   Shape<NT>::kSmem);
        if (e != cudaSuccess) return e;
        attr_done.fetch_or(bit);
    }
    half_tc_kernel<T, NT><<<(unsigned)std::min<int64_t>(p.tiles, sms), kThreads, Shape<NT>::kSmem, stream>>>(tx, ty, to, p);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_nt(int nt, const Params& p, const CUtensorMap& tx, const CUtensorMap& ty, const CUtensorMap& to,
                      int sms, cudaStream_t stream) {
    switch (nt) {
        case 32: return launch<T, 32>(p, tx, ty, to, sms, stream);
        case 64: return launch<T, 64>(p, tx, ty, to, sms, stream);
        case 128: return launch<T, 128>(p, tx, ty, to, sms, stream);
        default: return launch<T, 256>(p, tx, ty, to, sms, stream);
    }
}

}  // namespace

// The tile's N and orientation: the fewest elements read, (128 + NT) a tile,
// over the waves of one tile an SM.
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
    bool swapped = false;
    Params q{};
    for (int s = 0; s < 2; ++s)
        for (int n : {32, 64, 128, 256}) {
            if (!s && n == 32) continue;       // an upright box on the way out is 64 columns wide
            const int64_t xs = ((s ? p.N : p.M) + BX - 1) / BX, ys = ((s ? p.M : p.N) + n - 1) / n;
            if ((double)xs * (double)ys * (double)p.batch > 1e15) return false;
            const int64_t cost = (xs * ys * p.batch + sms - 1) / sms * (BX + n);
            if (nt == 0 || cost < best) {
                best = cost;
                nt = n;
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
    if (!make_map(&tx, vx, q.x_mn ? 64 : BX) || !make_map(&ty, vy, q.y_mn ? 64 : (uint32_t)nt) ||
        (q.c_tma && !make_map(&to, vc, swapped ? (uint32_t)(nt < 64 ? nt : 64) : BX))) {
        *err = cudaErrorInvalidValue;
        return true;
    }
    q.C = p.C; q.rsC = p.rsC; q.bsC = p.bsC;
    q.rows = p.M; q.cols = p.N;
    q.k_blocks = (int)((p.K + BK - 1) / BK);
    q.alpha = p.alpha;
    q.accumulate = p.accumulate;
    q.swapped = swapped;
    q.x_batch = p.batch > 1 && vx.batch_stride != 0;
    q.y_batch = p.batch > 1 && vy.batch_stride != 0;
    q.idesc = idesc16(p.type == SBGEMM_TYPE_BF16, nt, q.x_mn, q.y_mn);
    *err = p.type == SBGEMM_TYPE_BF16 ? launch_nt<__nv_bfloat16>(nt, q, tx, ty, to, sms, stream)
                                      : launch_nt<__half>(nt, q, tx, ty, to, sms, stream);
    return true;
}

unsigned int read_and_clear_status_half_tc(cudaStream_t stream) {
    return read_and_clear_word(reinterpret_cast<const void*>(&g_wait_status), stream);
}

}  // namespace sbg
