// Operations on the pages of a cache: copy, fork, append, free and compact
// (include/sbgemm.h).  All bookkeeping is done by kernels on the pool's device
// arrays, with integer results that do not depend on the order of threads:
// requests are admitted by their index (atomicMin claims, an ordered prefix
// sum of the pages they need), fresh pages are the free ones in ascending
// order, and counts change by integer atomics.
//
// What bounds them: copy and compact move pages and run at the memory's rate;
// fork, append and free touch little and are bound by the latency of their
// dependent steps, so each is one planning launch of one CTA (claims, checks,
// prefix sum, search of the free pages, all ordered by block barriers) and one
// launch over the GPU that moves the data.
//
// Data moves in pieces of 4 KB a warp (eight 16-byte loads in flight a lane,
// then eight stores).
#include <algorithm>
#include <atomic>
#include <climits>

#include "debug_check.cuh"
#include "half_util.cuh"
#include "ptx.cuh"
#include "serving.h"

namespace sbg {
namespace {

__device__ unsigned int g_status = 0;

constexpr int kPlanThreads = 1024;
constexpr int kPiece = 4096;                 // bytes a warp moves at a time
constexpr int kSegment = 1024;               // pages a block of the compaction counts
constexpr int kNoClaim = 0x7f7f7f7f;         // what memset leaves; above every request index

// A request of fork or append, as the planning kernel admitted it.
struct Request {
    int32_t ok;          // granted
    int32_t from, to;    // fork: parent, child; append: unused, sequence
    int32_t len;         // tokens before the call
    int32_t first;       // index of its first fresh page in the list of fresh pages
    int32_t need;        // fresh pages
    int32_t start, count;   // append: its tokens
};

struct Workspace {
    int32_t* head;       // [0] fresh pages found; compaction: [0] pages in use, [1] moved
    Request* req;        // [n]
    int32_t* fresh;      // [num_blocks] free pages in ascending order (compaction: the holes)
    int32_t* claim;      // [max(num_blocks, n_seqs)] lowest request with this destination
    int32_t* flag;       // [n_seqs] is some request's parent
    int32_t* rank;       // [num_blocks] compaction: rank among the pages in use
    int32_t* counts;     // [segments] compaction: pages in use of each segment
};

int64_t round256(int64_t b) { return (b + 255) / 256 * 256; }

Workspace layout(void* base, int64_t num_blocks, int64_t n_seqs, int64_t n, size_t* bytes) {
    int64_t at = 0;
    auto take = [&](int64_t size) {
        char* p = static_cast<char*>(base) + at;
        at += round256(size);
        return p;
    };
    Workspace w;
    w.head = reinterpret_cast<int32_t*>(take(256));
    w.req = reinterpret_cast<Request*>(take(n * (int64_t)sizeof(Request)));
    w.fresh = reinterpret_cast<int32_t*>(take(num_blocks * 4));
    w.claim = reinterpret_cast<int32_t*>(take(std::max(num_blocks, n_seqs) * 4));
    w.flag = reinterpret_cast<int32_t*>(take(n_seqs * 4));
    w.rank = reinterpret_cast<int32_t*>(take(num_blocks * 4));
    w.counts = reinterpret_cast<int32_t*>(take(((num_blocks + kSegment - 1) / kSegment) * 4));
    if (bytes) *bytes = (size_t)at;
    return w;
}

__device__ __forceinline__ int warp_inclusive(int v) {
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) {
        const int o = __shfl_up_sync(~0u, v, s);
        if ((threadIdx.x & 31) >= (unsigned)s) v += o;
    }
    return v;
}

// Exclusive prefix sum over the block (a whole number of warps, at most 32);
// *total receives the sum.  `sums` is 33 ints of shared memory.
__device__ __forceinline__ int block_exclusive(int v, int* sums, int* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int inc = warp_inclusive(v);
    __syncthreads();                          // the last use of sums is over
    if (lane == 31) sums[warp] = inc;
    __syncthreads();
    if (warp == 0) {
        const int s = warp_inclusive(lane < warps ? sums[lane] : 0);
        sums[lane] = s;                       // inclusive over warps; [31] is the total
    }
    __syncthreads();
    *total = sums[31];
    return inc - v + (warp ? sums[warp - 1] : 0);
}

// `bytes` (a multiple of 16, at most kPiece) moved by one warp.  Debug builds:
// between what `to` and `from` span.
__device__ __forceinline__ void move_piece(char* dst, const char* src, int bytes, const ByteSpan& to,
                                           const ByteSpan& from) {
    if (!dbg_in_bytes(dst, bytes, to, &g_status) || !dbg_in_bytes(src, bytes, from, &g_status)) return;
    constexpr int kLoads = kPiece / 512;
    const int lane = threadIdx.x & 31;
    uint4 v[kLoads];
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
        const int at = (lane + 32 * i) * 16;
        if (at < bytes) v[i] = *reinterpret_cast<const uint4*>(src + at);
    }
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
        const int at = (lane + 32 * i) * 16;
        if (at < bytes) *reinterpret_cast<uint4*>(dst + at) = v[i];
    }
}

__host__ __device__ __forceinline__ int64_t pieces_of(int64_t bytes) { return (bytes + kPiece - 1) / kPiece; }

// What cache i occupies.
__device__ __forceinline__ ByteSpan cache_span(const PageCaches& c, int i, int64_t num_blocks, int64_t block_size) {
    const uintptr_t base = reinterpret_cast<uintptr_t>(c.base[i]);
    return {base, base + (uintptr_t)(c.row_bytes[i] * block_size * num_blocks)};
}

// Debug builds: whether an entry of the counts or of the table is one.
__device__ __forceinline__ bool a_count(const PagePool& p, const int32_t* at) {
    const uintptr_t base = reinterpret_cast<uintptr_t>(p.refs);
    return dbg_in_bytes(at, 4, ByteSpan{base, base + (uintptr_t)(4 * p.num_blocks)}, &g_status);
}
__device__ __forceinline__ bool an_entry(const PagePool& p, const int32_t* at) {
    const uintptr_t base = reinterpret_cast<uintptr_t>(p.table);
    return dbg_in_bytes(at, 4, ByteSpan{base, base + (uintptr_t)(4 * p.n_seqs * p.max_blocks)}, &g_status);
}

// Piece `j` of the first `rows` rows of a page, over all caches: moved from
// page src to page dst by this warp.
__device__ __forceinline__ void move_page_piece(const PageCaches& c, int64_t num_blocks, int64_t block_size,
                                                int64_t rows, int64_t src, int64_t dst, int64_t j) {
    for (int i = 0; i < c.n; ++i) {
        const int64_t bytes = c.row_bytes[i] * rows, np = pieces_of(bytes);
        if (j < np) {
            const int64_t page = c.row_bytes[i] * block_size, at = j * kPiece;
            move_piece(c.base[i] + dst * page + at, c.base[i] + src * page + at,
                       (int)min((int64_t)kPiece, bytes - at), cache_span(c, i, num_blocks, block_size),
                       cache_span(c, i, num_blocks, block_size));
            return;
        }
        j -= np;
    }
}

// ---- copy --------------------------------------------------------------------

__device__ __forceinline__ bool in_pool(int64_t page, int64_t num_blocks) { return page >= 0 && page < num_blocks; }

// The lowest pair with each destination.
__device__ __forceinline__ void claim_pair(const int32_t* pairs, int64_t k, int64_t num_blocks, int32_t* claim) {
    const int src = pairs[2 * k], dst = pairs[2 * k + 1];
    if (in_pool(src, num_blocks) && in_pool(dst, num_blocks) && src != dst) atomicMin(&claim[dst], (int)k);
}

__global__ void copy_claim_kernel(const int32_t* pairs, int64_t n, int64_t num_blocks, int32_t* claim) {
    const int64_t k = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (k < n) claim_pair(pairs, k, num_blocks, claim);
}

// Few pairs of a small pool: every block makes the claims for itself in shared
// memory, and the copy is one launch (1500 pairs of 73.7 KB pages in a pool of 8192: 38.9
// us, 43.5 with a memset and a launch for them).
constexpr int64_t kOwnClaimPairs = 8192, kOwnClaimBlocks = 24576;

template <bool kOwnClaims>
__global__ void __launch_bounds__(512)
copy_move_kernel(const __grid_constant__ PageCaches c, const int32_t* pairs, int64_t n, int64_t num_blocks,
                 int64_t block_size, const int32_t* claims, int64_t pieces) {
    extern __shared__ int32_t own[];
    if (kOwnClaims) {
        for (int64_t i = threadIdx.x; i < num_blocks; i += blockDim.x) own[i] = kNoClaim;
        __syncthreads();
        for (int64_t k = threadIdx.x; k < n; k += blockDim.x) claim_pair(pairs, k, num_blocks, own);
        __syncthreads();
    }
    const int32_t* claim = kOwnClaims ? own : claims;
    const int64_t warps = (int64_t)gridDim.x * (blockDim.x >> 5);
    for (int64_t w = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); w < n * pieces; w += warps) {
        const int64_t k = w / pieces, j = w % pieces;
        const int src = pairs[2 * k], dst = pairs[2 * k + 1];
        const bool inside = in_pool(src, num_blocks) && in_pool(dst, num_blocks);
        if (inside && src == dst) continue;
        if (!inside || claim[dst] != k || claim[src] != kNoClaim) {
            if ((threadIdx.x & 31) == 0) record_status(&g_status, kPageRequest);
            continue;
        }
        move_page_piece(c, num_blocks, block_size, block_size, src, dst, j);
    }
}

// ---- fork and append: planning -------------------------------------------------

constexpr int kEach = 8;                     // pages a thread looks at in a round of the search

// Bit i: page at + i is free.
__device__ __forceinline__ unsigned free_pages(const int32_t* refs, int64_t num_blocks, int64_t at) {
    int v[kEach];
#pragma unroll
    for (int i = 0; i < kEach; ++i) v[i] = at + i < num_blocks ? refs[at + i] : 1;
    unsigned bits = 0;
#pragma unroll
    for (int i = 0; i < kEach; ++i) bits |= (v[i] == 0 ? 1u : 0u) << i;
    return bits;
}

// The free pages in ascending order, as many as `want`, into `fresh`; returns
// how many were found.  `first_bits`: this thread's pages of the first round,
// looked at beforehand.
__device__ int find_fresh(const int32_t* refs, int64_t num_blocks, int64_t want, unsigned first_bits,
                          int32_t* fresh, int* sums) {
    int64_t found = 0;
    for (int64_t base = 0; base < num_blocks && found < want; base += (int64_t)kPlanThreads * kEach) {
        const int64_t at = base + (int64_t)threadIdx.x * kEach;
        const unsigned bits = base == 0 ? first_bits : free_pages(refs, num_blocks, at);
        int total;
        int64_t to = found + block_exclusive(__popc(bits), sums, &total);
#pragma unroll
        for (int i = 0; i < kEach; ++i)
            if (bits >> i & 1) {
                if (to < want) fresh[to] = (int32_t)(at + i);
                ++to;
            }
        found += total;
    }
    return (int)min(found, want);
}

// Checks one request.  True: valid, with len, need (fresh pages), start and
// count filled in.
template <bool kFork>
__device__ __forceinline__ bool check_request(const PagePool& p, const int32_t* a, const int32_t* b,
                                              const Workspace& w, int64_t k, Request* r) {
    const int64_t bs = p.block_size;
    if (kFork) {
        r->from = a[k];
        r->to = b[k];
        if (r->from < 0 || r->from >= p.n_seqs || r->to < 0 || r->to >= p.n_seqs) return false;
        if (w.claim[r->to] != k || w.flag[r->to] || p.lens[r->to] != 0) return false;
        r->len = p.lens[r->from];
        if (r->len < 0 || r->len > p.max_blocks * bs) return false;
        const int64_t full = r->len / bs;
        r->need = r->len % bs != 0;
        return !r->need || in_pool(p.table[r->from * p.max_blocks + full], p.num_blocks);
    }
    r->to = a[k];
    r->start = b[k];
    r->count = b[k + 1] - b[k];
    if (r->to < 0 || r->to >= p.n_seqs) return false;
    if (w.claim[r->to] != k) return false;
    r->len = p.lens[r->to];
    if (r->len < 0 || (int64_t)r->len + r->count > min(p.max_blocks * bs, (int64_t)INT_MAX)) return false;
    const int64_t have = (r->len + bs - 1) / bs;
    r->need = (int32_t)(((int64_t)r->len + r->count + bs - 1) / bs - have);
    if (r->len % bs && r->count) {
        const int64_t last = p.table[r->to * p.max_blocks + have - 1];
        if (!in_pool(last, p.num_blocks) || p.refs[last] != 1) return false;
    }
    return true;
}

constexpr int kSharedSeqs = 4096;            // pools of up to so many sequences have their claims in shared memory

// One CTA: claims, checks, the prefix sum of the pages needed, the search of
// the free pages, and what is granted.  Fork: a = parents, b = children;
// append: a = sequences, b = starts.  Lengths are read before any is written.
// A chain of dependent steps, so the first pages are looked at while the
// requests come in, claims are in shared memory where they fit, and a thread
// keeps its first request in registers.
template <bool kFork>
__global__ void __launch_bounds__(kPlanThreads)
plan_kernel(const PagePool p, const int32_t* a, const int32_t* b, int64_t n, int64_t total, Workspace w) {
    __shared__ int sums[33];
    __shared__ int32_t claims[kSharedSeqs], flags[kSharedSeqs];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (p.n_seqs <= kSharedSeqs) {
        w.claim = claims;
        w.flag = flags;
    }
    const int t = threadIdx.x;
    const unsigned first_bits = free_pages(p.refs, p.num_blocks, (int64_t)t * kEach);
    bool bad_starts = false;
    for (int64_t k = t; k < n; k += kPlanThreads) {
        const int to = kFork ? b[k] : a[k];
        if (to >= 0 && to < p.n_seqs) {
            w.claim[to] = kNoClaim;
            w.flag[to] = 0;
        }
        if (!kFork) bad_starts |= b[k] < 0 || b[k + 1] < b[k] || b[k + 1] > total;
    }
    // Tokens are found by their place among the starts: without an order none is.
    bad_starts = __syncthreads_or(bad_starts);
    for (int64_t k = t; k < n; k += kPlanThreads) {
        const int to = kFork ? b[k] : a[k];
        if (to >= 0 && to < p.n_seqs) atomicMin(&w.claim[to], (int)k);
        // Flags of sequences that are no child are never read.
        if (kFork && a[k] >= 0 && a[k] < p.n_seqs) w.flag[a[k]] = 1;
    }
    __syncthreads();
    int64_t want = 0;
    Request mine{};
    for (int64_t base = 0; base < n; base += kPlanThreads) {
        const int64_t k = base + t;
        Request r{};
        r.ok = k < n && !bad_starts && check_request<kFork>(p, a, b, w, k, &r);
        if (!r.ok) r.need = 0;
        int sum;
        const int64_t before = want + block_exclusive(r.need, sums, &sum);
        // Past the pool's size nothing can be granted: keep the sum in range.
        r.first = (int32_t)min(before, (int64_t)INT_MAX / 2);
        want += sum;
        if (k < n && !r.ok) record_status(&g_status, kPageRequest);
        if (base == 0) mine = r;
        else if (k < n) w.req[k] = r;
    }
    __syncthreads();
    const int found = find_fresh(p.refs, p.num_blocks, min(want, p.num_blocks), first_bits, w.fresh, sums);
    for (int64_t k = t; k < n; k += kPlanThreads) {
        Request r = k < kPlanThreads ? mine : w.req[k];
        if (r.ok && (int64_t)r.first + r.need > found) {
            r.ok = 0;
            record_status(&g_status, kPageExhausted);
        }
        w.req[k] = r;
        if (r.ok) p.lens[r.to] = r.len + (kFork ? 0 : r.count);
    }
}

// ---- fork and append: moving -----------------------------------------------------

// One row of blocks a request: the child's table row and the counts of the
// shared pages (blockIdx.y == 0), and the rows of the last page.
__global__ void __launch_bounds__(256)
fork_move_kernel(const __grid_constant__ PageCaches c, const PagePool p, const Workspace w, int64_t pieces) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const Request r = w.req[blockIdx.x];
    if (!r.ok) return;
    const int64_t full = r.len / p.block_size, rest = r.len % p.block_size;
    const int32_t* from = p.table + r.from * p.max_blocks;
    int32_t* to = p.table + r.to * p.max_blocks;
    if (blockIdx.y == 0) {
        for (int64_t i = threadIdx.x; i < full; i += blockDim.x) {
            if (!an_entry(p, from + i) || !an_entry(p, to + i)) continue;
            const int page = from[i];
            to[i] = page;
            if (in_pool(page, p.num_blocks)) atomicAdd(&p.refs[page], 1);
            else record_status(&g_status, kPageRequest);
        }
    }
    if (r.need) {
        const int64_t src = from[full], dst = w.fresh[r.first];
        if (blockIdx.y == 0 && threadIdx.x == 0) {
            if (an_entry(p, to + full)) to[full] = (int32_t)dst;
            if (a_count(p, p.refs + dst)) p.refs[dst] = 1;
        }
        const int warps = (blockDim.x >> 5) * gridDim.y;
        for (int64_t j = blockIdx.y * (blockDim.x >> 5) + (threadIdx.x >> 5); j < pieces; j += warps)
            move_page_piece(c, p.num_blocks, p.block_size, rest, src, dst, j);
    }
}

// One warp a token and cache.
__global__ void __launch_bounds__(256)
append_move_kernel(const __grid_constant__ PageCaches c, const __grid_constant__ PageRows rows, const PagePool p,
                   const Workspace w, const int32_t* starts, int64_t n, int64_t total) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int64_t warps = (int64_t)gridDim.x * (blockDim.x >> 5);
    const int lane = threadIdx.x & 31;
    const int64_t per = c.n ? c.n : 1;
    for (int64_t i = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); i < total * per; i += warps) {
        const int64_t j = i / per;
        const int cache = (int)(i % per);
        // The last request that starts at or before token j and holds it;
        // evenly spread requests are found at the first look.
        int64_t k = j * n / total;
        if (!(starts[k] <= j && j < starts[k + 1])) {
            int64_t lo = 0, hi = n;                    // starts[lo] <= j < starts[hi] where monotone
            while (hi - lo > 1) {
                const int64_t mid = (lo + hi) / 2;
                if (starts[mid] <= j) lo = mid;
                else hi = mid;
            }
            k = lo;
        }
        const Request r = w.req[k];
        if (!r.ok || j < r.start || j >= (int64_t)r.start + r.count) continue;   // in no granted request
        const int64_t pos = r.len + (j - r.start), idx = pos / p.block_size, off = pos % p.block_size;
        const int64_t have = (r.len + p.block_size - 1) / p.block_size;
        int32_t* slot = p.table + r.to * p.max_blocks + idx;
        const int64_t page = idx < have ? *slot : w.fresh[r.first + (idx - have)];
        // The token that opens a page enters it.
        if (idx >= have && off == 0 && cache == 0 && lane == 0) {
            if (an_entry(p, slot)) *slot = (int32_t)page;
            if (a_count(p, p.refs + page)) p.refs[page] = 1;
        }
        if (c.n == 0) continue;
        const int64_t rb = c.row_bytes[cache];
        char* dst = c.base[cache] + (page * p.block_size + off) * rb;
        const char* src = rows.base[cache] + j * rows.stride[cache];
        const int64_t reach = rows.stride[cache] * (total - 1);
        const uintptr_t first = reinterpret_cast<uintptr_t>(rows.base[cache]);
        const ByteSpan given{first + (uintptr_t)min(reach, (int64_t)0), first + (uintptr_t)(max(reach, (int64_t)0) + rb)};
        for (int64_t at = 0; at < rb; at += kPiece)
            move_piece(dst + at, src + at, (int)min((int64_t)kPiece, rb - at),
                       cache_span(c, cache, p.num_blocks, p.block_size), given);
    }
}

// ---- free ------------------------------------------------------------------------

__global__ void __launch_bounds__(256) free_kernel(const PagePool p, const int32_t* seqs) {
    __shared__ int64_t pages;
    const int64_t s = seqs[blockIdx.x];
    if (threadIdx.x == 0) {
        pages = 0;
        if (s < 0 || s >= p.n_seqs) {
            record_status(&g_status, kPageRequest);
        } else {
            // The first block to come takes the length: a sequence given twice is freed once.
            const int64_t len = atomicExch(&p.lens[s], 0);
            pages = (len + p.block_size - 1) / p.block_size;
            if (len < 0 || pages > p.max_blocks) {
                record_status(&g_status, kPageRequest);
                pages = len < 0 ? 0 : p.max_blocks;
            }
        }
    }
    __syncthreads();
    for (int64_t i = threadIdx.x; i < pages; i += blockDim.x) {
        const int64_t page = p.table[s * p.max_blocks + i];
        if (!in_pool(page, p.num_blocks)) {
            record_status(&g_status, kPageRequest);
        } else if (atomicSub(&p.refs[page], 1) <= 0) {
            atomicAdd(&p.refs[page], 1);
            record_status(&g_status, kPageRequest);
        }
    }
}

// ---- compact ---------------------------------------------------------------------

constexpr int64_t kOwnCounts = 32;           // segments that every ranking block counts for itself

__global__ void __launch_bounds__(256) compact_count_kernel(const int32_t* refs, int64_t num_blocks, int32_t* counts) {
    __shared__ int sums[33];
    int used = 0;
#pragma unroll
    for (int i = 0; i < kSegment / 256; ++i) {
        const int64_t at = (int64_t)blockIdx.x * kSegment + i * 256 + threadIdx.x;
        used += at < num_blocks && refs[at] > 0;
    }
    int total;
    block_exclusive(used, sums, &total);
    if (threadIdx.x == 0) counts[blockIdx.x] = total;
}

// Each segment's pages: holes (free, index < U) into w.fresh by their rank,
// movers (in use, index >= U) into w.claim by theirs, and each page's rank
// among those in use.  The movers are the last h of the U pages in use, so
// mover k is w.claim[U - h + k] and goes to w.fresh[k].
__global__ void __launch_bounds__(256)
compact_rank_kernel(const int32_t* refs, int64_t num_blocks, int64_t segments, const Workspace w) {
    __shared__ int sums[33];
    const int t = threadIdx.x;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    int part_before = 0, part_all = 0;
    if (segments <= kOwnCounts) {
#pragma unroll 8
        for (int64_t i = t; i < num_blocks; i += 256) {
            const int v = refs[i] > 0;
            part_all += v;
            if (i < (int64_t)blockIdx.x * kSegment) part_before += v;
        }
    } else {
        for (int64_t s = t; s < segments; s += 256) {
            const int v = w.counts[s];
            part_all += v;
            if (s < blockIdx.x) part_before += v;
        }
    }
    int before, U;
    block_exclusive(part_all, sums, &U);
    block_exclusive(part_before, sums, &before);
    constexpr int kEach = kSegment / 256;
    const int64_t at = (int64_t)blockIdx.x * kSegment + (int64_t)t * kEach;
    int used[kEach], sum = 0;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        used[i] = at + i < num_blocks && refs[at + i] > 0;
        sum += used[i];
    }
    int total;
    int rank = before + block_exclusive(sum, sums, &total);
    if (blockIdx.x == 0 && t == 0) {
        w.head[0] = U;
        if (U == 0) w.head[1] = 0;
    }
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const int64_t page = at + i;
        if (page >= num_blocks) break;
        if (used[i] && page >= U) w.claim[rank] = (int32_t)page;
        if (!used[i] && page < U) w.fresh[page - rank] = (int32_t)page;
        w.rank[page] = used[i] ? rank : -1;
        rank += used[i];
        if (page == U - 1) w.head[1] = U - rank;       // holes up to U
    }
}

__global__ void __launch_bounds__(256)
compact_move_kernel(const __grid_constant__ PageCaches c, const PagePool p, const Workspace w, int64_t pieces,
                    int32_t* moved) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int U = w.head[0], h = w.head[1];
    const int64_t threads = (int64_t)gridDim.x * blockDim.x, t = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (t == 0 && moved) *moved = h;
    for (int64_t k = t; k < h; k += threads) {
        const int src = w.claim[U - h + k], dst = w.fresh[k];
        if (!a_count(p, p.refs + dst) || !a_count(p, p.refs + src)) continue;
        p.refs[dst] = p.refs[src];
        p.refs[src] = 0;
    }
    for (int64_t e = t; e < p.n_seqs * p.max_blocks; e += threads) {
        const int64_t s = e / p.max_blocks, i = e % p.max_blocks;
        if (i * p.block_size >= p.lens[s]) continue;
        const int page = p.table[e];
        if (page < U && page >= 0) continue;
        const int rank = in_pool(page, p.num_blocks) ? w.rank[page] : -1;
        if (rank < 0) record_status(&g_status, kPageRequest);    // out of range or not in use
        else p.table[e] = w.fresh[rank - (U - h)];
    }
    const int64_t warps = threads >> 5;
    for (int64_t i = t >> 5; i < h * pieces; i += warps)
        move_page_piece(c, p.num_blocks, p.block_size, p.block_size, w.claim[U - h + i / pieces], w.fresh[i / pieces],
                        i % pieces);
}

int64_t page_pieces(const PageCaches& c, int64_t block_size) {
    int64_t n = 0;
    for (int i = 0; i < c.n; ++i) n += pieces_of(c.row_bytes[i] * block_size);
    return n;
}

// Blocks of 8 warps for `warps` warps of work, at most eight a SM.
unsigned move_grid(int64_t warps, int sms) {
    return (unsigned)std::max<int64_t>(1, std::min<int64_t>((warps + 7) / 8, (int64_t)sms * 8));
}

// A launch that may begin before the one ahead of it ends; the kernel waits for
// that one's results itself (griddepcontrol.wait).
template <typename... P, typename... A>
cudaError_t launch_early(void (*kernel)(P...), dim3 grid, int threads, cudaStream_t stream, A... args) {
    cudaLaunchAttribute early{};
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.stream = stream;
    cfg.attrs = &early;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}

}  // namespace

size_t pages_workspace_bytes(int64_t num_blocks, int64_t n_seqs, int64_t n) {
    size_t bytes = 0;
    layout(nullptr, num_blocks, n_seqs, n, &bytes);
    return bytes;
}

cudaError_t launch_pages_copy(const PageCaches& c, const PagePool& p, const int32_t* pairs, int64_t n, void* ws,
                              int sms, cudaStream_t stream) {
    const int64_t pieces = page_pieces(c, p.block_size);
    // Blocks of 16 warps, two a SM.
    const unsigned grid = (unsigned)std::max<int64_t>(1, std::min<int64_t>((n * pieces + 15) / 16, (int64_t)sms * 2));
    if (n <= kOwnClaimPairs && p.num_blocks <= kOwnClaimBlocks) {
        static std::atomic<uint64_t> attr_done{0};
        int dev = 0;
        cudaGetDevice(&dev);
        const uint64_t bit = 1ull << (dev & 63);
        if (!(attr_done.load() & bit)) {
            const cudaError_t e = cudaFuncSetAttribute(copy_move_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                       (int)(kOwnClaimBlocks * 4));
            if (e != cudaSuccess) return e;
            attr_done.fetch_or(bit);
        }
        copy_move_kernel<true><<<grid, 512, (size_t)p.num_blocks * 4, stream>>>(c, pairs, n, p.num_blocks, p.block_size,
                                                                              nullptr, pieces);
        return cudaGetLastError();
    }
    const Workspace w = layout(ws, p.num_blocks, 0, 0, nullptr);
    const cudaError_t e = cudaMemsetAsync(w.claim, 0x7f, (size_t)p.num_blocks * 4, stream);
    if (e != cudaSuccess) return e;
    copy_claim_kernel<<<(unsigned)((n + 255) / 256), 256, 0, stream>>>(pairs, n, p.num_blocks, w.claim);
    copy_move_kernel<false><<<grid, 512, 0, stream>>>(c, pairs, n, p.num_blocks, p.block_size, w.claim, pieces);
    return cudaGetLastError();
}

cudaError_t launch_pages_fork(const PageCaches& c, const PagePool& p, const int32_t* parents,
                              const int32_t* children, int64_t n, void* ws, int sms, cudaStream_t stream) {
    const Workspace w = layout(ws, p.num_blocks, p.n_seqs, n, nullptr);
    plan_kernel<true><<<1, kPlanThreads, 0, stream>>>(p, parents, children, n, 0, w);
    const int64_t pieces = page_pieces(c, p.block_size);
    // A block moves 8 pieces at a time; at most two blocks a SM in all.
    const int64_t y = std::min<int64_t>((pieces + 7) / 8, std::max<int64_t>(1, 2 * sms / n));
    const cudaError_t e = launch_early(fork_move_kernel, dim3((unsigned)n, (unsigned)std::max<int64_t>(1, y)), 256,
                                       stream, c, p, w, pieces);
    return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_pages_append(const PageCaches& c, const PagePool& p, const int32_t* seqs, const int32_t* starts,
                                int64_t n, const PageRows& rows, int64_t total, void* ws, int sms,
                                cudaStream_t stream) {
    const Workspace w = layout(ws, p.num_blocks, p.n_seqs, n, nullptr);
    plan_kernel<false><<<1, kPlanThreads, 0, stream>>>(p, seqs, starts, n, total, w);
    if (total > 0) {
        const cudaError_t e = launch_early(append_move_kernel, dim3(move_grid(total * std::max(c.n, 1), sms)), 256,
                                           stream, c, rows, p, w, starts, n, total);
        if (e != cudaSuccess) return e;
    }
    return cudaGetLastError();
}

cudaError_t launch_pages_free(const PagePool& p, const int32_t* seqs, int64_t n, cudaStream_t stream) {
    free_kernel<<<(unsigned)n, 256, 0, stream>>>(p, seqs);
    return cudaGetLastError();
}

cudaError_t launch_pages_compact(const PageCaches& c, const PagePool& p, int32_t* moved, void* ws, int sms,
                                 cudaStream_t stream) {
    const Workspace w = layout(ws, p.num_blocks, p.n_seqs, 0, nullptr);
    const int64_t segments = (p.num_blocks + kSegment - 1) / kSegment;
    if (segments > kOwnCounts)
        compact_count_kernel<<<(unsigned)segments, 256, 0, stream>>>(p.refs, p.num_blocks, w.counts);
    compact_rank_kernel<<<(unsigned)segments, 256, 0, stream>>>(p.refs, p.num_blocks, segments, w);
    const cudaError_t e = launch_early(compact_move_kernel, dim3((unsigned)(sms * 8)), 256, stream, c, p, w,
                                       page_pieces(c, p.block_size), moved);
    return e != cudaSuccess ? e : cudaGetLastError();
}

unsigned int* status_word_pages() { return word_address(&g_status); }

}  // namespace sbg
