// The product of 8-bit floats with block scales on the tensor cores
// (sbgemm_fp8), for operands with unit stride along K that a tensor map
// describes.
//
// K goes by in blocks of 128, one 128-byte swizzled row of each operand and one
// scale each, through a ring of TMA stages: a block's products (four MMAs of
// K = 32, kind::f8f6f4) start a fresh accumulator in TMEM, one of two, and the
// epilogue warps add it, times the two scales, to fp32 sums in registers while
// the next block's MMAs run. So no scale has to be a power of two, and no more
// than 128 products are summed by the tensor core.
//
// A tile is 128 rows (the MMA's M) by NT columns. Its rows are rows of C, or
// columns of C (C^T = B^T A^T): a decode batch's few tokens are the columns and
// the weights fill the rows. Large products run on CTA pairs, one MMA of 256 x
// 256 x 32 over both CTAs' shared memory, which then moves 32 KB a block of K
// and CTA, in and out, instead of 48. Few tiles with a long K are split along K
// over the CTAs of a cluster: each sums its blocks and hands every other CTA
// its share of the columns through distributed shared memory, added there in
// the order of the CTAs.
//
// Roles: warps 8 and 10 issue the TMA loads of an operand each, warp 9 the MMAs; warps
// 0-3 and 4-7 hold the sums of the tile's two column halves, a thread one row.
// C goes out through shared memory and its tensor map (what fp32 sums are added to is
// brought there first, so that every output is rounded once; boxes added by the map's
// own additions would round alpha's product before them and lose what is below 2^-126:
// 131 us for the 146 below), else in 16-byte vectors, else from shared memory row by row,
// or by the element.
//
// Measured on a GB300, device time in a graph, bf16 out, a scale a row of A and
// 128 x 128 of B: 4099 x 7168 x 4096 110 us (2.18 PFLOP/s), 4096 x 4096 x 4096 64 us,
// a scale a row of both 118; 1024 x 4096 x 4096 19.1 us; 2560 x 960 x 8192, a scale a
// row of both, fp32 47.5 us, added to C 51.7; 4099 x 7168 x 4096 fp32 123 us, added
// to C 146 (702 by the element), bf16 added to C 179; 16 x 7168 x 4096 7.4 us from L2, 9.7 from memory.
// Bound: large products by the epilogue. A block's 256 x 256 x 128 take the
// tensor cores 513 cycles and the eight warps that scale it 850, of which 270 wait for
// their loads from TMEM; with a scale for each column twice the arithmetic, 1600.
// (Without effect or slower: two commits a block for half the columns each 118 us,
// scales' addresses moved on 147, scales staged in shared memory 140 to 146.) Few rows
// by the weights' bytes and the start and end of a cluster's CTAs.
#include <algorithm>
#include <atomic>

#include "debug_check.cuh"
#include "f32x2.cuh"
#include "layers.h"
#include "tc16.cuh"

namespace sbg {
namespace {

constexpr int BX = 128, BK = kScaleBlock;
constexpr int kGroups = 2, kTmaWarp = 4 * kGroups, kMmaWarp = kTmaWarp + 1, kTmaWarpY = kTmaWarp + 2;
constexpr int kChunk = 8;        // blocks of K whose column scales come in together: a 32-byte sector of a row's
constexpr int kThreads = 4 * (kGroups + 1) * 32;      // whole warpgroups: registers move between them
// Named barriers: 0 the CTA, 1 and 2 the epilogue groups, 3 the start, of its own
// since the TMA warp, which only arrives there, may come to the CTA's next one
// before the others have passed it.
constexpr int kStartBarrier = 3;
__device__ unsigned int g_status = 0;

// Scales of one operand; shift: 7 where one covers 128 rows, else 0.
struct Scales { const float* at; int64_t rs, ks, bs; int rows, shift; ByteSpan span; };

struct Params {
    void* C; int64_t cx, cy, cb;   // C's strides along the tile's rows, its columns and the batch
    int type_c;
    int64_t rows, cols;            // of the product's tiles: x < rows, y < cols
    uint32_t x_tiles, y_tiles, tiles;
    int k_blocks, split;           // split: CTAs of a cluster that share a tile's blocks
    float alpha;
    int accumulate;
    int vec;                       // columns go out as 16-byte vectors
    int vec_rows;                  // ... and a split tile's as vectors of four rows
    int c_tma;                     // C goes out through its tensor map
    int c_rows;                    // rows that are not whole vectors: a row's columns by a warp's lanes
    int x_batch, y_batch;          // the batch coordinate moves (else shared)
    uint32_t idesc;
    Scales sx, sy;
    ByteSpan sc;                   // debug builds: what C occupies
};

template <int NT, bool kYScales, bool kPair>
struct Shape {
    static constexpr int kYRows = kPair ? NT / 2 : NT;              // this CTA's share of Y
    static constexpr int kStage = (BX + kYRows) * BK;
    // Two CTAs an SM for up to 64 columns: the weights' bytes want to be in flight.
    static constexpr int kCtas = NT <= 64 ? 2 : 1;
    static constexpr int kStages = NT <= 32 ? 5 : NT == 64 ? 4 : kYScales ? 5 : 6;
    // Accumulators in TMEM: few columns are read long after their MMAs were quick.
    static constexpr int kAccs = NT <= 64 ? 4 : 2;
    static constexpr uint32_t kCols = kAccs * NT;
    // Buffers of the way out, [128 rows][128 bytes] for each group.
    static constexpr int kOut = NT >= 128 ? kGroups * BX * 128 : 0;
    static constexpr int kSmem = kStages * kStage + kOut + 1024;
    static_assert(NT > 128 || 2 * NT * BX * 4 <= kStages * kStage, "a split tile's sums, here and from the cluster");
    static_assert((kSmem + (kYScales ? 8 * kChunk * NT : 0) + 512) * kCtas <= 232448, "shared memory");
};

// kind::f8f6f4, D fp32, both operands K-major.
uint32_t idesc8(bool x_e5m2, bool y_e5m2, int n, int m) {
    return (1u << 4) | ((x_e5m2 ? 1u : 0u) << 7) | ((y_e5m2 ? 1u : 0u) << 10) | ((uint32_t)(n >> 3) << 17) |
           ((uint32_t)(m >> 4) << 24);
}

template <bool kPair>
__device__ __forceinline__ void mma8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    if constexpr (kPair)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}"
            ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}"
            ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
            : "memory");
}

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

// Shared memory of this CTA to that of a CTA of the cluster (shared::cluster
// addresses of the destination and of its barrier).
__device__ __forceinline__ void bulk_copy_to_cta(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                 ::"r"(dst), "r"(smem_u32(src)), "r"(bytes), "r"(bar) : "memory");
}

__device__ __forceinline__ void cp_async4(float* dst, const float* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}

// 16 bytes, or zeros.
__device__ __forceinline__ void cp_async16(void* dst, const void* src, bool read) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(read ? 16 : 0) : "memory");
}

__device__ __forceinline__ float get(const float* c) { return *c; }
template <typename T> __device__ __forceinline__ float get(const T* c) { return to_float(*c); }
__device__ __forceinline__ void put(float* c, float v) { *c = v; }
template <typename T> __device__ __forceinline__ void put(T* c, float v) { *c = from_float<T>(v); }
// 16 bytes of a row.
__device__ __forceinline__ void put_vector(float* c, const uint64_t* v, float alpha) {
    *reinterpret_cast<float4*>(c) =
        make_float4(alpha * lower(v[0]), alpha * upper(v[0]), alpha * lower(v[1]), alpha * upper(v[1]));
}
template <typename T> __device__ __forceinline__ void put_vector(T* c, const uint64_t* v, float alpha) {
    *reinterpret_cast<uint4*>(c) = make_uint4(
        pack2<T>(alpha * lower(v[0]), alpha * upper(v[0])), pack2<T>(alpha * lower(v[1]), alpha * upper(v[1])),
        pack2<T>(alpha * lower(v[2]), alpha * upper(v[2])), pack2<T>(alpha * lower(v[3]), alpha * upper(v[3])));
}
// The same added to what is there.
__device__ __forceinline__ void add_vector(float* c, const uint64_t* v, float alpha) {
    const float4 o = *reinterpret_cast<const float4*>(c);
    *reinterpret_cast<float4*>(c) = make_float4(fmaf(alpha, lower(v[0]), o.x), fmaf(alpha, upper(v[0]), o.y),
                                                fmaf(alpha, lower(v[1]), o.z), fmaf(alpha, upper(v[1]), o.w));
}
template <typename T> __device__ __forceinline__ void add_vector(T* c, const uint64_t* v, float alpha) {
    const uint4 o = *reinterpret_cast<const uint4*>(c);
    auto added = [&](uint32_t w, uint64_t x) {
        const float2 f = unpack2<T>(w);
        return pack2<T>(fmaf(alpha, lower(x), f.x), fmaf(alpha, upper(x), f.y));
    };
    *reinterpret_cast<uint4*>(c) = make_uint4(added(o.x, v[0]), added(o.y, v[1]), added(o.z, v[2]), added(o.w, v[3]));
}
template <typename T>
__device__ __forceinline__ void put_one(const Params& p, T* c, float v) {
    if (dbg_in_bytes(c, sizeof(T), p.sc, &g_status)) put(c, p.accumulate ? fmaf(p.alpha, v, get(c)) : p.alpha * v);
}

// Sums v of the columns y .. y + n - 1 of row x go out.
template <typename T, int n>
__device__ __forceinline__ void emit_as(const Params& p, int64_t b, int64_t x, int64_t y, const uint64_t (&v)[n / 2]) {
    if (x >= p.rows) return;
    T* c = static_cast<T*>(p.C) + b * p.cb + x * p.cx + y * p.cy;
    constexpr int w = 16 / sizeof(T);
    if constexpr (n % w == 0) {
        if (p.vec) {                 // unit stride along the columns, whole vectors
#pragma unroll
            for (int i = 0; i < n; i += w)
                if (y + i < p.cols && dbg_in_bytes(c + i, 16, p.sc, &g_status)) {
                    if (p.accumulate) add_vector(c + i, v + i / 2, p.alpha);
                    else put_vector(c + i, v + i / 2, p.alpha);
                }
            return;
        }
    }
#pragma unroll
    for (int i = 0; i < n; ++i, c += p.cy)
        if (y + i < p.cols) put_one(p, c, i & 1 ? upper(v[i / 2]) : lower(v[i / 2]));
}
// The sums of four rows from x on of column y.
template <typename T>
__device__ __forceinline__ void emit_rows_as(const Params& p, int64_t b, int x, int y, const float4& v) {
    T* c = static_cast<T*>(p.C) + b * p.cb + x * p.cx + y * p.cy;
    if (p.vec_rows && x + 3 < p.rows) {
        if (!dbg_in_bytes(c, 4 * sizeof(T), p.sc, &g_status)) return;
        float4 o = make_float4(p.alpha * v.x, p.alpha * v.y, p.alpha * v.z, p.alpha * v.w);
        if (p.accumulate) {
            float4 old;
            if constexpr (sizeof(T) == 4) {
                old = *reinterpret_cast<const float4*>(c);
            } else {
                const uint2 w = *reinterpret_cast<const uint2*>(c);
                const float2 a = unpack2<T>(w.x), d = unpack2<T>(w.y);
                old = make_float4(a.x, a.y, d.x, d.y);
            }
            o = make_float4(fmaf(p.alpha, v.x, old.x), fmaf(p.alpha, v.y, old.y), fmaf(p.alpha, v.z, old.z),
                            fmaf(p.alpha, v.w, old.w));
        }
        if constexpr (sizeof(T) == 4) *reinterpret_cast<float4*>(c) = o;
        else *reinterpret_cast<uint2*>(c) = make_uint2(pack2<T>(o.x, o.y), pack2<T>(o.z, o.w));
        return;
    }
    const float each[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i, c += p.cx)
        if (x + i < p.rows) put_one(p, c, each[i]);
}
__device__ __forceinline__ void emit_rows(const Params& p, int64_t b, int x, int y, const float4& v) {
    if (y >= p.cols) return;
    if (p.type_c == SBGEMM_TYPE_BF16) emit_rows_as<__nv_bfloat16>(p, b, x, y, v);
    else if (p.type_c == SBGEMM_TYPE_FP16) emit_rows_as<__half>(p, b, x, y, v);
    else emit_rows_as<float>(p, b, x, y, v);
}
template <int n>
__device__ __forceinline__ void emit(const Params& p, int64_t b, int64_t x, int64_t y, const uint64_t (&v)[n / 2]) {
    if (p.type_c == SBGEMM_TYPE_BF16) emit_as<__nv_bfloat16, n>(p, b, x, y, v);
    else if (p.type_c == SBGEMM_TYPE_FP16) emit_as<__half, n>(p, b, x, y, v);
    else emit_as<float, n>(p, b, x, y, v);
}

// The same of all 128 rows of a group's columns through shared memory and C's
// tensor map, in boxes of 128 bytes a row: a thread's own vectors would touch 32
// rows an instruction, half a sector each.
template <typename T, int n, bool kAdded>
__device__ __forceinline__ void send_as(const Params& p, const CUtensorMap& to, uint8_t* buf, int g, int row, int b, int x0,
                                        int y, const uint64_t (&v)[n / 2]) {
    constexpr int w = 16 / sizeof(T), box = 128 / sizeof(T);
#pragma unroll
    for (int c = 0; c < n; c += box) {
        if (row == 0) bulk_wait_read_all();              // the buffer's last store has read it
        group_sync(g);
        if constexpr (kAdded) {
            // What the sums are added to comes in first, 8 threads a row.
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int r = 16 * i + (row >> 3), e = (row & 7) * w;
                const T* at = static_cast<const T*>(p.C) + b * p.cb + (int64_t)(x0 + r) * p.cx + (y + c + e);
                const bool there = x0 + r < p.rows && y + c + e < p.cols && dbg_in_bytes(at, 16, p.sc, &g_status);
                cp_async16(buf + r * 128 + ((e * 4) ^ ((r & 7) << 4)), there ? at : static_cast<const T*>(p.C), there);
            }
            asm volatile("cp.async.commit_group;\n\tcp.async.wait_group 0;" ::: "memory");
            group_sync(g);
        }
#pragma unroll
        for (int i = 0; i < box; i += w) {
            T* at = reinterpret_cast<T*>(buf + row * 128 + ((i / w * 16) ^ ((row & 7) << 4)));
            if constexpr (kAdded) add_vector(at, v + (c + i) / 2, p.alpha);
            else put_vector(at, v + (c + i) / 2, p.alpha);
        }
        fence_proxy_async_smem();
        group_sync(g);
        if (row == 0) {
            if (y + c < p.cols && x0 < p.rows) tma_store_3d(&to, buf, (y + c) * (int)sizeof(T), x0, b);
            bulk_commit();
        }
    }
}
template <int n>
__device__ __forceinline__ void send(const Params& p, const CUtensorMap& to, uint8_t* buf, int g, int row, int b, int x0,
                                     int y, const uint64_t (&v)[n / 2]) {
    if constexpr (n >= 64) {
        if (p.type_c == SBGEMM_TYPE_BF16) send_as<__nv_bfloat16, n, false>(p, to, buf, g, row, b, x0, y, v);
        else if (p.type_c == SBGEMM_TYPE_FP16) send_as<__half, n, false>(p, to, buf, g, row, b, x0, y, v);
        else if (p.accumulate) send_as<float, n, true>(p, to, buf, g, row, b, x0, y, v);
        else send_as<float, n, false>(p, to, buf, g, row, b, x0, y, v);
    }
}

// Where rows of C are not whole vectors: 32 columns of the sums at a time through
// shared memory, then a row's by a warp's lanes. (4099 x 7168 x 4096, rows of 7169: 134
// us, 377 by a thread a row.)
template <typename T, int n>
__device__ __forceinline__ void spread_as(const Params& p, uint8_t* buf, int g, int row, int b, int x0, int y,
                                          const uint64_t (&v)[n / 2]) {
    const int lane = row & 31, r0 = row & ~31;
#pragma unroll
    for (int c = 0; c < n; c += 32) {
        group_sync(g);                                   // the buffer's last columns are read
#pragma unroll
        for (int i = 0; i < 32; i += 4)
            put_vector(reinterpret_cast<float*>(buf + row * 128 + ((i * 4) ^ ((row & 7) << 4))), v + (c + i) / 2, 1.0f);
        group_sync(g);
        T* at = static_cast<T*>(p.C) + b * p.cb + (int64_t)(x0 + r0) * p.cx + (y + c + lane);
        if (y + c + lane < p.cols) {
            for (int r = 0; r < 32; r += 16, at += 16 * p.cx) {
                auto mine = [&](int q) { return x0 + r0 + r + q < p.rows && dbg_in_bytes(at + q * p.cx, sizeof(T), p.sc, &g_status); };
                float old[16];                           // (all on their way before the first store)
#pragma unroll
                for (int q = 0; q < 16; ++q) old[q] = p.accumulate && mine(q) ? get(at + q * p.cx) : 0.0f;
#pragma unroll
                for (int q = 0; q < 16; ++q) {
                    const float v = *reinterpret_cast<const float*>(buf + (r0 + r + q) * 128 + ((lane * 4) ^ ((q & 7) << 4)));
                    if (mine(q)) put(at + q * p.cx, p.accumulate ? fmaf(p.alpha, v, old[q]) : p.alpha * v);
                }
            }
        }
    }
}
template <int n>
__device__ __forceinline__ void spread(const Params& p, uint8_t* buf, int g, int row, int b, int x0, int y,
                                       const uint64_t (&v)[n / 2]) {
    if constexpr (n >= 64) {
        if (p.type_c == SBGEMM_TYPE_BF16) spread_as<__nv_bfloat16, n>(p, buf, g, row, b, x0, y, v);
        else if (p.type_c == SBGEMM_TYPE_FP16) spread_as<__half, n>(p, buf, g, row, b, x0, y, v);
        else spread_as<float, n>(p, buf, g, row, b, x0, y, v);
    }
}

// (An ordinary load: the kernel before may write scales while this one is resident
// already, and what comes by the read-only path is not ordered behind the wait for it.)
__device__ __forceinline__ float load_scale(const float* at, const ByteSpan& span) {
    return dbg_in_bytes(at, 4, span, &g_status) ? *at : 0.0f;
}

// kYScales: Y has a scale for each of its rows (the tile's columns), else one
// for each 128 of them, which a half of the tile's columns lies in.
template <int NT, bool kYScales, bool kPair>
__global__ void __launch_bounds__(kThreads, Shape<NT, kYScales, kPair>::kCtas)
fp8_tc_kernel(const __grid_constant__ CUtensorMap tx, const __grid_constant__ CUtensorMap ty,
              const __grid_constant__ CUtensorMap to, const __grid_constant__ Params p) {
    using S = Shape<NT, kYScales, kPair>;
    constexpr int kCtas = kPair ? 2 : 1;
    constexpr int CPG = NT / kGroups;            // columns of a group
    const int rank = kPair || p.split > 1 ? (int)cluster_rank() : 0;
    const int pair_rank = kPair ? rank : 0, k_rank = kPair ? 0 : rank;
    extern __shared__ uint8_t raw[];
    uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
    // mma_done: a stage's MMAs are through, for the TMA warp that fills it again and
    // for the epilogue that reads their sums (one commit a block: a second one
    // behind it holds the issuing thread for some 360 cycles).
    __shared__ uint64_t full[S::kStages], mma_done[S::kStages], acc_free[S::kAccs], sums_full;
    __shared__ uint32_t tmem_base;
    // Scales of the columns for kChunk blocks of K, two chunks a group.
    __shared__ alignas(16) float ys[kYScales ? kGroups : 1][2][kYScales ? kChunk : 1][kYScales ? CPG : 4];
    const int warp = uniform_warp(), lane = threadIdx.x & 31;

    if (threadIdx.x == kTmaWarp * 32) {
        for (int s = 0; s < S::kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&mma_done[s], 1);
        }
        for (int i = 0; i < S::kAccs; ++i) mbar_init(&acc_free[i], 4 * kGroups * kCtas);
        mbar_init(&sums_full, 1);
        fence_mbar_init_cluster();
        prefetch_tensormap(&tx);
        prefetch_tensormap(&ty);
        if (p.c_tma) prefetch_tensormap(&to);
    }
    if (warp == kMmaWarp) {
        if constexpr (kPair) {
            tmem_alloc_pair(&tmem_base, S::kCols);
            tmem_relinquish_pair();
        } else {
            tmem_alloc(&tmem_base, S::kCols);
            tmem_relinquish();
        }
        // From here on: a kernel that starts early and waits for this one may hold TMEM
        // on this SM, which this one must not wait for.
        asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    }
    if constexpr (kPair) {
        tc_fence_before();
        __syncthreads();
        // A pair's barriers and TMEM are there in both CTAs before either uses the other's.
        cluster_sync();
        tc_fence_after();
    } else if (warp == kTmaWarp) {
        // The loads need the barriers alone, which this warp has made: on without waiting.
        __syncwarp();
        asm volatile("bar.arrive %0, %1;" ::"n"(kStartBarrier), "n"(kThreads) : "memory");
    } else {
        tc_fence_before();
        asm volatile("bar.sync %0, %1;" ::"n"(kStartBarrier), "n"(kThreads) : "memory");
        tc_fence_after();
    }
    // Launched while the kernel before may still run (what it writes may be an operand).
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // (That TMA warp, which may be ahead of the allocation, does not use it.)
    const uint32_t tmem = S::kCols == kTmemAll ? kTmemBase : warp == kTmaWarp ? 0 : tmem_base;
    const int share = kPair ? 2 : p.split;       // CTAs a tile
    const uint32_t first = blockIdx.x / share, stride = gridDim.x / share;
    const int j0 = k_rank * p.k_blocks / p.split, j1 = (k_rank + 1) * p.k_blocks / p.split;
    // (32 bits: a 64-bit division takes hundreds of cycles.)
    auto place = [&](uint32_t t, int* x0, int* y0, int* b) {
        *x0 = (int)(t % p.x_tiles) * (BX * kCtas) + BX * pair_rank;
        *y0 = (int)(t / p.x_tiles % p.y_tiles) * NT;
        *b = (int)(t / p.x_tiles / p.y_tiles);
    };

    // (Sums of a split tile's threads, kept over the cluster's barriers below.)
    uint64_t acc[CPG / 2];
    const int g = warp >> 2, row = threadIdx.x & 127;
    int x = 0, y = 0, b = 0;
    // 256 x 216 + 128 x 64 registers are within the 384 x 168 of the launch.
    if (warp >= kTmaWarp) {
        if constexpr (CPG == 128) asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
        if (warp == kTmaWarp || warp == kTmaWarpY) {
            // A warp an operand: a load takes its issuer some 250 cycles.
            const bool is_x = warp == kTmaWarp;
            if (lane == 0) {
                auto load = [&](void* dst, const CUtensorMap* map, int s, int c0, int c1, int c2) {
                    if constexpr (kPair) tma_load_3d_pair(dst, map, cluster_addr(&full[s], 0), c0, c1, c2);
                    else tma_load_3d(dst, map, &full[s], c0, c1, c2);
                };
                int s = 0, issued = 0;
                uint32_t round = 0;
                bool ok = true;
                for (uint32_t t = first; t < p.tiles && ok; t += stride) {
                    int x0, y0, b;
                    place(t, &x0, &y0, &b);
                    const int zx = p.x_batch ? b : 0, zy = p.y_batch ? b : 0;
                    for (int j = j0; j < j1; ++j) {
                        if (round > 0 && !bar_wait(&mma_done[s], (round - 1) & 1)) {
                            record_status(&g_status, kWaitEmpty);
                            ok = false;
                            break;
                        }
                        uint8_t* x = ring + s * S::kStage;
                        if (is_x) {
                            if (pair_rank == 0) mbar_arrive_expect_tx(&full[s], S::kStage * kCtas);
                            load(x, &tx, s, j * BK, x0, zx);
                        } else {
                            load(x + BX * BK, &ty, s, j * BK, y0 + S::kYRows * pair_rank, zy);
                        }
                        if (issued < S::kStages) ++issued;
                        if (++s == S::kStages) {
                            s = 0;
                            ++round;
                        }
                    }
                }
                // Copies still landing keep the CTA's shared memory (a pair's first
                // CTA waits for both).
                for (int q = 0; is_x && pair_rank == 0 && q < issued; ++q) {
                    if (--s < 0) {
                        s = S::kStages - 1;
                        --round;
                    }
                    if (!bar_wait(&full[s], round & 1)) {
                        record_status(&g_status, kWaitDrain);
                        break;
                    }
                }
            }
            __syncwarp();
        } else if (warp == kMmaWarp) {
            if (pair_rank == 0 && elect_one()) {
                int s = 0, n = 0, last = -1;           // stage; blocks begun; the last one's stage
                uint32_t round = 0, last_round = 0;
                bool ok = true;
                for (uint32_t t = first; t < p.tiles && ok; t += stride) {
                    for (int j = j0; j < j1; ++j, ++n) {
                        // The operands first: what follows the accumulator's wait is on
                        // the way from its last reader to the next block's sums.
                        if (!bar_wait(&full[s], round & 1)) {
                            record_status(&g_status, kWaitFull);
                            ok = false;
                            break;
                        }
                        const int a = n % S::kAccs;
                        if (n >= S::kAccs) {
                            const uint32_t ph = (uint32_t)((n / S::kAccs - 1) & 1);
                            if (!(kPair ? bar_wait_cluster(&acc_free[a], ph) : bar_wait(&acc_free[a], ph))) {
                                record_status(&g_status, kWaitAccFree);
                                ok = false;
                                break;
                            }
                        }
                        tc_fence_after();
                        const uint32_t acc = tmem + (uint32_t)a * NT;
                        const uint32_t x = smem_u32(ring + s * S::kStage);
                        uint64_t dx = desc16(x), dy = desc16(x + BX * BK);
#pragma unroll
                        for (int k = 0; k < BK / 32; ++k) {      // 32 bytes of K a step
                            mma8<kPair>(acc, dx, dy, p.idesc, k ? 1u : 0u);
                            dx += kStepK;
                            dy += kStepK;
                        }
                        if constexpr (kPair) mma_commit_pair_both(&mma_done[s]);
                        else mma_commit(&mma_done[s]);
                        last = s;
                        last_round = round;
                        if (++s == S::kStages) {
                            s = 0;
                            ++round;
                        }
                    }
                }
                // Nothing may still be writing TMEM when it is freed.
                if (last >= 0 && !bar_wait(&mma_done[last], last_round & 1)) record_status(&g_status, kWaitMma);
            }
            __syncwarp();
        }
    } else {
        if constexpr (CPG == 128) asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        int n = 0, s = 0;
        uint32_t round = 0;
        bool ok = true;
        for (uint32_t t = first; t < p.tiles; t += stride) {
            int x0, y0;
            place(t, &x0, &y0, &b);
            x = x0 + row;
            y = y0 + g * CPG;
            // This thread's row's scales, two blocks ahead in registers, and the
            // columns' common one likewise, or each column's through shared memory.
            // Rows past the end take the last one's.
            const float* sx = p.sx.at + b * p.sx.bs + (min(x, p.sx.rows - 1) >> p.sx.shift) * p.sx.rs;
            const float* sy = p.sy.at + b * p.sy.bs + (kYScales ? 0 : (min(y, p.sy.rows - 1) >> p.sy.shift) * p.sy.rs);
            // (Multiplied when they are used: a product here would wait for the loads.)
            auto row_scale = [&](int j) { return j < j1 ? load_scale(sx + j * p.sx.ks, p.sx.span) : 0.0f; };
            auto col_scale = [&](int j) { return !kYScales && j < j1 ? load_scale(sy + j * p.sy.ks, p.sy.span) : 1.0f; };
            auto fetch = [&](int c) {            // the columns' scales of chunk c
                for (int i = row; i < kChunk * CPG; i += 128) {
                    const int k = i % kChunk, col = i / kChunk, j = j0 + c * kChunk + k;
                    const float* at = sy + min(y + col, p.sy.rows - 1) * p.sy.rs + j * p.sy.ks;
                    if (j < j1 && dbg_in_bytes(at, 4, p.sy.span, &g_status)) cp_async4(&ys[g][c & 1][k][col], at);
                }
                asm volatile("cp.async.commit_group;" ::: "memory");
            };
            float fx[2] = {row_scale(j0), row_scale(j0 + 1)}, fy[2] = {col_scale(j0), col_scale(j0 + 1)};
            if constexpr (kYScales) {
                group_sync(g);                   // the last tile's scales are read
                fetch(0);
            }
            if (S::kOut && p.c_tma && p.accumulate && x < p.rows) {
                // What the sums are added to, on its way into L2 under the products.  (Without:
                // 157 us, for 149 at the time.)
                const float* at = static_cast<const float*>(p.C) + b * p.cb + x * p.cx + y;
                for (int i = 0; i < CPG && y + i < p.cols; i += 32) asm volatile("prefetch.global.L2 [%0];" ::"l"(at + i) : "memory");
            }
#pragma unroll
            for (int i = 0; i < CPG / 2; ++i) acc[i] = 0;
            for (int j = j0; j < j1; ++j, ++n) {
                const float f = kYScales ? fx[0] : fx[0] * fy[0];
                const uint64_t ff = pair_of(f, f);
                fx[0] = fx[1];
                fy[0] = fy[1];
                fx[1] = row_scale(j + 2);
                fy[1] = col_scale(j + 2);
                if constexpr (kYScales) {
                    if ((j - j0) % kChunk == 0) {
                        // A chunk is in for all, and all are through with the one before.
                        asm volatile("cp.async.wait_group 0;" ::: "memory");
                        group_sync(g);
                        if (j + kChunk < j1) fetch((j - j0) / kChunk + 1);
                    }
                }
                const float* yscale = ys[kYScales ? g : 0][kYScales ? (j - j0) / kChunk & 1 : 0][kYScales ? (j - j0) % kChunk : 0];
                if (ok && !bar_wait(&mma_done[s], round & 1)) {
                    record_status(&g_status, kWaitMma);
                    ok = false;
                }
                if (++s == S::kStages) {
                    s = 0;
                    ++round;
                }
                // (A warp whose wait ran out goes on without waiting, so that all come to
                // the same barriers; its group's tiles are not stored from then on.)
                tc_fence_after();
                // The accumulator in pieces, the next one on its way under a piece's sums.
                constexpr int W = CPG < 16 ? CPG : CPG <= 32 || !kYScales ? 16 : 32;     // (as registers allow without spills)
                uint32_t v[2][W];
                const int a = n % S::kAccs;
                const uint32_t at = tmem + lanes + (uint32_t)(a * NT + g * CPG);
                tmem_ld_begin<W>(at, v[0]);
#pragma unroll
                for (int c = 0; c < CPG; c += W) {
                    uint32_t (&now)[W] = v[c / W & 1];
                    tmem_ld_end<W>(now);
                    if (c + W < CPG) {
                        tmem_ld_begin<W>(at + c + W, v[(c / W + 1) & 1]);
                    } else {
                        // The accumulator is read: the next block's MMAs may have it.
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) {
                            if (kPair && pair_rank != 0) mbar_arrive_remote_relaxed(&acc_free[a], 0);
                            else mbar_arrive(&acc_free[a]);
                        }
                    }
                    if constexpr (kYScales) {
#pragma unroll
                        for (int i = 0; i < W; i += 4) {
                            const ulonglong2 z = *reinterpret_cast<const ulonglong2*>(yscale + c + i);
                            fma2(acc[(c + i) / 2], pair_of(now[i], now[i + 1]), mul2(ff, z.x));
                            fma2(acc[(c + i) / 2 + 1], pair_of(now[i + 2], now[i + 3]), mul2(ff, z.y));
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < W; i += 2)
                            fma2(acc[(c + i) / 2], pair_of(now[i], now[i + 1]), ff);
                    }
                }
            }
            ok = all_of_group(g, ok);
            if (ok && (kPair || p.split == 1)) {
                if (S::kOut && p.c_tma) send<CPG>(p, to, ring + S::kStages * S::kStage + g * BX * 128, g, row, b, x0, y, acc);
                else if (S::kOut && p.c_rows) spread<CPG>(p, ring + S::kStages * S::kStage + g * BX * 128, g, row, b, x0, y, acc);
                else emit<CPG>(p, b, x, y, acc);
            }
        }
        if (S::kOut && p.c_tma && row == 0) bulk_wait_read_all();    // shared memory outlives the stores' reads

    }
    if constexpr (!kPair && NT <= 128) {
        if (p.split > 1) {
            // One tile a cluster.  This CTA's ring is idle: its sums go there, column
            // by column, and once every CTA's is, each one's share of the columns
            // to it by a bulk copy, all CTAs' behind one another.
            const int each = NT / p.split;       // columns this CTA adds up
            uint8_t* mine = ring;
            uint8_t* theirs = ring + NT * BX * 4;
            __syncwarp();
            if (warp < kTmaWarp) {
#pragma unroll
                for (int i = 0; i < CPG; ++i)
                    reinterpret_cast<float*>(mine)[(g * CPG + i) * BX + row] = i & 1 ? upper(acc[i / 2]) : lower(acc[i / 2]);
                fence_proxy_async_smem();
            }
            __syncthreads();
            cluster_sync();
            const uint32_t bytes = (uint32_t)(each * BX * 4);
            if (threadIdx.x == 0) {
                mbar_arrive_expect_tx(&sums_full, bytes * p.split);
                for (int r = 0; r < p.split; ++r)
                    bulk_copy_to_cta(cluster_addr(theirs + k_rank * bytes, r), mine + r * bytes, bytes,
                                     cluster_addr(&sums_full, r));
            }
            if (warp < kTmaWarp) {
                const bool in = bar_wait(&sums_full, 0);
                if (!in) record_status(&g_status, kWaitPartial);
                const float* sums = reinterpret_cast<const float*>(theirs);
                // A warp a column, a lane four of its rows.
                const int x4 = x - row + 4 * lane, y0 = y - g * CPG + k_rank * each;
#pragma unroll 2
                for (int c = warp; in && c < each; c += 4 * kGroups) {
                    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    for (int r = 0; r < p.split; ++r) {
                        const float4 w = *reinterpret_cast<const float4*>(sums + (r * each + c) * BX + 4 * lane);
                        v.x += w.x;
                        v.y += w.y;
                        v.z += w.z;
                        v.w += w.w;
                    }
                    emit_rows(p, b, x4, y0 + c, v);
                }
            }
            // Nobody leaves while a copy may still read its memory.
            __syncwarp();
            cluster_sync();
        }
    }
    tc_fence_before();
    __syncthreads();
    // Neither CTA of a pair leaves while the other may use its memory.
    if constexpr (kPair) cluster_sync();
    if (warp == kMmaWarp) {
        tc_fence_after();
        if constexpr (kPair) tmem_dealloc_pair(tmem, S::kCols);
        else tmem_dealloc(tmem, S::kCols);
    }
}

bool mappable(const Fp8Operand& o, int64_t K, int64_t batch) {
    if (o.ks != 1 && K > 1) return false;
    if (reinterpret_cast<uintptr_t>(o.data) % 16 != 0) return false;
    auto ok = [](int64_t s) { return s > 0 && s % 16 == 0 && s < ((int64_t)1 << 39); };
    if (o.rows > 1 && !ok(o.rs)) return false;
    return batch == 1 || o.bs == 0 || ok(o.bs);
}

bool make_map(CUtensorMap* map, const Fp8Operand& o, int64_t K, int64_t batch, uint32_t box_rows) {
    const bool moves = batch > 1 && o.bs != 0;
    const uint64_t dims[3] = {(uint64_t)K, (uint64_t)o.rows, moves ? (uint64_t)batch : 1};
    const uint64_t rs = o.rows > 1 ? (uint64_t)o.rs : (uint64_t)(K + 15) / 16 * 16;
    const uint64_t strides[2] = {rs, moves ? (uint64_t)o.bs : rs};
    const uint32_t box[3] = {BK, box_rows, 1};
    return encode_tmap_8(map, o.data, 3, dims, strides, box);
}

Scales scales_of(const Fp8Operand& o) {
    return Scales{o.scale, o.rsS, o.ksS, o.bsS, (int)o.rows, o.group == 1 ? 0 : 7, o.ss};
}

template <int NT, bool kYScales, bool kPair>
cudaError_t launch(const Params& p, const CUtensorMap& tx, const CUtensorMap& ty, const CUtensorMap& to, int sms,
                   cudaStream_t stream) {
    using S = Shape<NT, kYScales, kPair>;
    static std::atomic<int> ready[64];           // 0: not asked yet; else the pairs that fit (or 1)
    int dev = 0;
    cudaGetDevice(&dev);
    const int size = kPair ? 2 : p.split;
    cudaLaunchConfig_t cfg{};
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = S::kSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attrs[2] = {};
    attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attrs[0].val.programmaticStreamSerializationAllowed = 1;
    attrs[1].id = cudaLaunchAttributeClusterDimension;
    attrs[1].val.clusterDim.x = (unsigned)size;
    attrs[1].val.clusterDim.y = attrs[1].val.clusterDim.z = 1;
    cfg.attrs = attrs;
    cfg.numAttrs = size > 1 ? 2 : 1;
    int fit = ready[dev & 63].load();
    if (fit == 0) {
        const cudaError_t e = cudaFuncSetAttribute(fp8_tc_kernel<NT, kYScales, kPair>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
        if (e != cudaSuccess) return e;
        fit = 1;
        if (kPair) {
            cfg.gridDim = dim3((unsigned)(sms / 2 * 2));
            if (cudaOccupancyMaxActiveClusters(&fit, fp8_tc_kernel<NT, kYScales, kPair>, &cfg) != cudaSuccess ||
                fit <= 0) {
                cudaGetLastError();
                fit = sms / 2;
            }
        }
        ready[dev & 63].store(fit);
    }
    // A split tile is its cluster's only one; others go round the CTAs (or pairs) that are resident.
    const int64_t at_once = p.split > 1 ? p.tiles : kPair ? fit : (int64_t)sms * S::kCtas;
    cfg.gridDim = dim3((unsigned)(std::min<int64_t>(p.tiles, at_once) * size));
    return cudaLaunchKernelEx(&cfg, fp8_tc_kernel<NT, kYScales, kPair>, tx, ty, to, p);
}

template <bool kYScales>
cudaError_t launch_nt(int nt, bool pair, const Params& p, const CUtensorMap& tx, const CUtensorMap& ty,
                      const CUtensorMap& to, int sms, cudaStream_t stream) {
    if (pair) return launch<256, kYScales, true>(p, tx, ty, to, sms, stream);
    switch (nt) {
        case 16: return launch<16, kYScales, false>(p, tx, ty, to, sms, stream);
        case 32: return launch<32, kYScales, false>(p, tx, ty, to, sms, stream);
        case 64: return launch<64, kYScales, false>(p, tx, ty, to, sms, stream);
        default: return launch<128, kYScales, false>(p, tx, ty, to, sms, stream);
    }
}

// Cycles of a block of K in a tile, measured: with one scale for the columns or
// one each (twice the epilogue's arithmetic), and for tiles of up to 64 columns
// with one CTA on an SM or two. 4096 x 4096 x 4096: pairs 67 and 116 us, tiles of
// 128 columns 74 and 122, of 64 columns 120 and 163; 2560 x 960 x 8192 with scales
// a column: 47 us on 300 tiles of 64 columns in one wave, 58 on 40 pairs, 68 on 160
// tiles of 128 columns in two waves.
int block_cycles(int nt, bool pair, int on_sm, bool y_scales) {
    if (pair) return y_scales ? 1600 : 850;
    switch (nt) {
        case 16: return y_scales ? (on_sm == 2 ? 900 : 610) : on_sm == 2 ? 650 : 560;
        case 32: return y_scales ? (on_sm == 2 ? 1000 : 650) : on_sm == 2 ? 700 : 600;
        case 64: return y_scales ? (on_sm == 2 ? 1200 : 850) : on_sm == 2 ? 920 : 760;
        default: return y_scales ? 930 : 535;
    }
}

}  // namespace

bool launch_fp8_tc(const Fp8Problem& p, int sms, cudaStream_t stream, cudaError_t* err) {
    // (Indexes of a tile past the last one still are ints.)
    if (p.a.rows > INT32_MAX - 1024 || p.b.rows > INT32_MAX - 1024) return false;
    if (p.K <= 0 || !mappable(p.a, p.K, p.batch) || !mappable(p.b, p.K, p.batch)) return false;
    const int k_blocks = (int)((p.K + BK - 1) / BK);
    // Orientation, columns of a tile, pairs, and the split of K: the fewest
    // cycles, by the blocks of K that an SM goes through, 2500 cycles for a tile's
    // start and end (a pair's 4000), and 4500 for joining a split one.  (16 x 7168 x
    // 4096, 16 columns a tile: 13.7, 10.8 and 9.8 us split by 1, 2 and 4; 128 x 7168
    // x 4096: 13.1 us upright, 16.9 turned and split by 2.)
    double best = 0;
    int nt = 0;
    bool swapped = false, pair = false;
    Params q{};
    for (int s = 0; s < 2; ++s)
        for (int n : {16, 32, 64, 128, 256}) {
            const bool two = n == 256;       // CTA pairs, 256 x 256
            const int64_t bx = two ? 2 * BX : BX, by = n;
            const int64_t xs = ((s ? p.b.rows : p.a.rows) + bx - 1) / bx, ys = ((s ? p.a.rows : p.b.rows) + by - 1) / by;
            if ((double)xs * (double)ys * (double)p.batch > 1e9) continue;
            const int64_t tiles = xs * ys * p.batch, per_sm = n <= 64 ? 2 : 1;
            const int64_t slots = two ? sms / 2 : sms * per_sm;
            for (int split : {1, 2, 4, 8}) {
                // (A split tile goes out a row a lane: along C's unit stride.)
                if (split > 1 && (s ? p.csC : p.rsC) != 1 && (s ? p.rsC : p.csC) == 1) break;
                if (split > 1 && (n > 128 || tiles * split > slots || split > k_blocks || by / split < 2)) break;
                const int64_t waves = (tiles * split + slots - 1) / slots;
                const int on_sm = per_sm == 2 && tiles * split > sms ? 2 : 1;
                const double cost = waves * ((double)((k_blocks + split - 1) / split) * block_cycles((int)by, two, on_sm, (s ? p.a : p.b).group == 1) +
                                             (two ? 4000 : 2500) + (split > 1 ? 4500 : 0));
                if (nt == 0 || cost < best) {
                    best = cost;
                    nt = (int)by;
                    pair = two;
                    swapped = s != 0;
                    q.x_tiles = (uint32_t)xs;
                    q.y_tiles = (uint32_t)ys;
                    q.tiles = (uint32_t)tiles;
                    q.split = split;
                }
            }
        }
    if (nt == 0) return false;
    const Fp8Operand& ox = swapped ? p.b : p.a;
    const Fp8Operand& oy = swapped ? p.a : p.b;
    CUtensorMap tx, ty, to{};
    if (!make_map(&tx, ox, p.K, p.batch, BX) || !make_map(&ty, oy, p.K, p.batch, (uint32_t)(pair ? nt / 2 : nt))) return false;
    q.C = p.C;
    q.cx = swapped ? p.csC : p.rsC;
    q.cy = swapped ? p.rsC : p.csC;
    q.cb = p.bsC;
    q.type_c = p.type_c;
    q.rows = ox.rows;
    q.cols = oy.rows;
    q.k_blocks = k_blocks;
    q.alpha = p.alpha;
    q.accumulate = p.accumulate;
    const int64_t w = p.type_c == SBGEMM_TYPE_FP32 ? 4 : 8;
    q.vec = q.cy == 1 && q.cols % w == 0 && (q.rows == 1 || q.cx % w == 0) &&
            (p.batch == 1 || q.cb % w == 0) && reinterpret_cast<uintptr_t>(p.C) % 16 == 0;
    q.vec_rows = q.cx == 1 && (q.cols == 1 || q.cy % 4 == 0) && (p.batch == 1 || q.cb % 4 == 0) &&
                 reinterpret_cast<uintptr_t>(p.C) % 16 == 0;
    // Whole vectors, and rows that a map can describe.  (What is added to 16-bit elements
    // goes by a thread's own vectors.)
    q.c_tma = q.vec && (!p.accumulate || p.type_c == SBGEMM_TYPE_FP32) && nt >= 128 && q.split == 1 && (q.rows == 1 || q.cx > 0) && (p.batch == 1 || q.cb > 0) &&
              q.cx < ((int64_t)1 << 37) && q.cb < ((int64_t)1 << 37) && q.cols < ((int64_t)1 << 29);
    q.c_rows = !q.vec && nt >= 128 && q.cy == 1;
    if (q.c_tma) {
        const int64_t e = 16 / w, row = q.rows > 1 ? q.cx * e : (q.cols * e + 15) / 16 * 16;
        const uint64_t strides[2] = {(uint64_t)row, p.batch > 1 ? (uint64_t)(q.cb * e) : (uint64_t)row};
        // Bytes: the map copies boxes of 128 of them whatever C's type is.
        const uint64_t dims[3] = {(uint64_t)(q.cols * e), (uint64_t)q.rows, (uint64_t)p.batch};
        const uint32_t box[3] = {128, BX, 1};
        q.c_tma = encode_tmap_8(&to, p.C, 3, dims, strides, box);        // (else by vectors)
    }
    q.x_batch = p.batch > 1 && ox.bs != 0;
    q.y_batch = p.batch > 1 && oy.bs != 0;
    q.idesc = idesc8(ox.type == SBGEMM_TYPE_E5M2, oy.type == SBGEMM_TYPE_E5M2, nt, pair ? 256 : 128);
    q.sx = scales_of(ox);
    q.sy = scales_of(oy);
    q.sc = p.sc;
    *err = oy.group == 1 ? launch_nt<true>(nt, pair, q, tx, ty, to, sms, stream)
                         : launch_nt<false>(nt, pair, q, tx, ty, to, sms, stream);
    return true;
}

unsigned int* status_word_fp8_tc() { return word_address(&g_status); }

}  // namespace sbg
