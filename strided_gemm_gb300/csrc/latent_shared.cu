// Latent attention over a paged cache for groups of sequences with a shared
// prefix (sbgemm_latent_attention_shared): the plan.
//
// Starts are taken as a running maximum of their values clamped to [0, n_seqs], so
// that every kernel sees the same, sound groups whatever stands in device memory;
// what was clamped is reported here.  For the row kernel the plan is each
// sequence's first key of its own and the sequence whose table row has the keys
// before.  For the tensor cores it is a list of items besides, up to nb query rows
// against a run of keys, and each item's place in a list of blocks of keys that the
// CTAs share equally: items of each sequence's own keys, then those of the
// prefixes, a group's rows of all its sequences side by side, so that a block of the
// prefix is read once for nb rows where the sequences alone would read it each for
// their own.  One CTA makes it (two running sums, over sequences and over groups),
// launched before the kernel that uses it and waited for there.
//
// Measured on a GB300, R = 512, P = 64, plan and join included, device time in a
// graph: 64 sequences with 250 to 1000 keys of their own behind 16001, 16 heads, bf16 76
// us (each for itself 180; with 1000 each 84); 4 documents of 8192 keys with 16 questions
// of 175 to 700, 128 heads, fp16, pages of 64 235 us, of 16 277; 4 samples of 50 to 200
// behind 1500 20 us; 64 sequences of 250 to 1000 and no prefix 31 us, of 1000 35; 300
// groups of 5 with 60 behind 500 270 us. The
// plan of up to 1024 sequences takes 5.5 us on its own, caches cold.
#include <algorithm>

#include "debug_check.cuh"
#include "serving.h"

namespace sbg {
namespace {

__device__ unsigned int g_status = 0;
constexpr int kPlanThreads = 1024;

struct PrefixPlan {
    LatentShared g;
    int32_t* prefix_item;                // nullptr: no items are wanted
    int32_t* head;
    LatentItem* items;
    int nb, keys, rows, own;             // query rows and keys a block; rows of a sequence; its items
};

__device__ __forceinline__ int clamped(int v, int lo, int hi, bool report) {
    const int c = min(max(v, lo), hi);
    if (c != v && report) record_status(&g_status, kPagedInput);
    return c;
}

struct Pair { int a, b; };
// Sums over the CTA's threads up to and with this one, and of all.
__device__ __forceinline__ Pair running(Pair v, Pair (&shared)[kPlanThreads / 32], Pair* all) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int a = __shfl_up_sync(~0u, v.a, o), b = __shfl_up_sync(~0u, v.b, o);
        if (lane >= o) {
            v.a += a;
            v.b += b;
        }
    }
    __syncthreads();
    if (lane == 31) shared[warp] = v;
    __syncthreads();
    // The warps before, by each warp's lanes.
    const Pair mine = shared[lane];
    const int below = warp > lane;
    Pair before{(int)__reduce_add_sync(~0u, below ? mine.a : 0), (int)__reduce_add_sync(~0u, below ? mine.b : 0)};
    *all = Pair{(int)__reduce_add_sync(~0u, mine.a), (int)__reduce_add_sync(~0u, mine.b)};
    return Pair{v.a + before.a, v.b + before.b};
}

__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const __grid_constant__ PrefixPlan p) {
    struct Group { int lo, hi, prefix, item, unit; };
    __shared__ Group group[kPlanThreads];
    __shared__ Pair sums[kPlanThreads / 32];
    __shared__ int tops[kPlanThreads / 32], so_far;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const LatentShared& g = p.g;
    const LatentPaged& a = g.paged;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, n_seqs = (int)a.n_seqs;
    const bool items = p.items != nullptr;
    auto length = [&](int s, bool report) { return a.seq_lens ? clamped(a.seq_lens[s], 0, (int)a.N, report) : (int)a.N; };
    auto put = [&](int32_t* at, int v) {
        if (dbg_in_bytes(at, 4, g.sw, &g_status)) *at = v;
    };
    auto put_item = [&](int i, const LatentItem& it) {
        if (dbg_in_bytes(p.items + i, sizeof(it), g.sw, &g_status)) p.items[i] = it;
    };
    for (int s = tid; s < n_seqs; s += kPlanThreads) {
        put(g.first + s, s);
        put(g.prefix + s, 0);
        if (items) put(p.prefix_item + s, -1);
    }
    // The groups, kPlanThreads at a time: f(how many, this thread's group).
    auto groups = [&](bool report, auto f) {
        if (tid == 0) so_far = 0;
        __syncthreads();
        for (int64_t g0 = 0; g0 < g.n_groups; g0 += kPlanThreads) {
            const int64_t i = g0 + tid;
            const bool mine = i < g.n_groups;
            // From the running maximum up to this group's start to that up to the next one's.
            const int at = mine ? clamped(g.group_starts[i], 0, n_seqs, report) : 0;
            const int next = mine ? clamped(g.group_starts[i + 1], 0, n_seqs, report) : 0;
            int top = at;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int x = __shfl_up_sync(~0u, top, o);
                if (lane >= o) top = max(top, x);
            }
            if (lane == 31) tops[warp] = top;
            __syncthreads();
            int lo = max(so_far, top);
            for (int w = 0; w < warp; ++w) lo = max(lo, tops[w]);
            const int hi = max(lo, next);
            __syncthreads();
            if (tid == kPlanThreads - 1) so_far = lo;
            Group mine_is{lo, hi, 0, 0, 0};
            if (mine) {
                const int given = g.prefix_lens[i];
                if (report && (lo != at || hi != next || given < 0)) record_status(&g_status, kPagedInput);
                if (lo < hi) mine_is.prefix = clamped(given, 0, length(lo, false), report);
            } else {
                mine_is.hi = lo;
            }
            f((int)min((int64_t)kPlanThreads, g.n_groups - g0), mine_is);
            __syncthreads();
        }
    };
    groups(true, [&](int count, const Group& mine) {
        group[tid] = mine;
        __syncthreads();
        for (int i = warp; i < count; i += kPlanThreads / 32)
            for (int s = group[i].lo + lane; s < group[i].hi; s += 32) {
                put(g.first + s, group[i].lo);
                put(g.prefix + s, group[i].prefix);
            }
    });
    __syncthreads();

    // Each sequence's own keys, from its prefix on.
    Pair total{0, n_seqs * p.own};           // units, items
    for (int s0 = 0; s0 < n_seqs; s0 += kPlanThreads) {
        const int s = s0 + tid;
        const int len = s < n_seqs ? length(s, true) : 0;       // (reports every length)
        if (!items) continue;
        const int lo = s < n_seqs ? g.prefix[s] : 0, units = len > lo ? (len + p.keys - 1) / p.keys - lo / p.keys : 0;
        Pair all;
        const int cost = latent_item_cost(units), at = total.a + running(Pair{cost * p.own, 0}, sums, &all).a - cost * p.own;
        if (s < n_seqs)
            for (int k = 0; k < p.own; ++k)
                put_item(s * p.own + k, LatentItem{at + k * cost, units, s, lo, len, s, k * p.nb,
                                                   min(p.nb, p.rows - k * p.nb)});
        total.a += all.a;
        __syncthreads();
    }
    if (!items) return;
    groups(false, [&](int count, Group mine) {
        const int rows = (mine.hi - mine.lo) * p.rows;
        const int blocks = mine.prefix > 0 ? (rows + p.nb - 1) / p.nb : 0;
        const int cost = latent_item_cost((mine.prefix + p.keys - 1) / p.keys);
        Pair all;
        const Pair at = running(Pair{blocks * cost, blocks}, sums, &all);
        mine.unit = total.a + at.a - blocks * cost;
        mine.item = total.b + at.b - blocks;
        group[tid] = mine;
        __syncthreads();
        for (int i = warp; i < count; i += kPlanThreads / 32) {
            const Group it = group[i];
            if (it.prefix <= 0) continue;
            const int rows = (it.hi - it.lo) * p.rows, units = (it.prefix + p.keys - 1) / p.keys;
            for (int s = it.lo + lane; s < it.hi; s += 32) put(p.prefix_item + s, it.item);
            for (int k = lane; k * p.nb < rows; k += 32)
                put_item(it.item + k, LatentItem{it.unit + k * latent_item_cost(units), units, it.lo, 0, it.prefix, it.lo, k * p.nb,
                                                 min(p.nb, rows - k * p.nb)});
        }
        total.a += all.a;
        total.b += all.b;
    });
    if (tid == 0) {
        put(p.head, total.a);
        put(p.head + 1, total.b);
    }
}

// The same for batches of up to kPlanThreads sequences and groups, a thread each:
// everything is loaded at once and stays in shared memory (plan_kernel's rounds
// through global memory and its passes over the groups take twice as long).
__global__ void __launch_bounds__(kPlanThreads) small_plan_kernel(const __grid_constant__ PrefixPlan p) {
    struct Sums { int own, units, items; };
    __shared__ int lens[kPlanThreads], firsts[kPlanThreads], prefixes[kPlanThreads], prefix_items[kPlanThreads];
    __shared__ int los[kPlanThreads], his[kPlanThreads], given[kPlanThreads], tops[kPlanThreads / 32];
    __shared__ Sums sums[kPlanThreads / 32];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const LatentShared& g = p.g;
    const LatentPaged& a = g.paged;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, n_seqs = (int)a.n_seqs, n_groups = (int)g.n_groups;
    const int warps = blockDim.x / 32;
    const bool is_seq = tid < n_seqs, is_group = tid < n_groups;
    const int len_in = is_seq && a.seq_lens ? a.seq_lens[tid] : (int)a.N;
    const int at_in = is_group ? g.group_starts[tid] : 0, next_in = is_group ? g.group_starts[tid + 1] : 0;
    const int prefix_in = is_group ? g.prefix_lens[tid] : 0;
    const int len = clamped(len_in, 0, (int)a.N, true);
    const int at = clamped(at_in, 0, n_seqs, true), next = clamped(next_in, 0, n_seqs, true);
    lens[tid] = len;
    firsts[tid] = tid;
    prefixes[tid] = 0;
    prefix_items[tid] = -1;
    // From the running maximum up to this group's start to that up to the next one's.
    int lo = at;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(~0u, lo, o);
        if (lane >= o) lo = max(lo, x);
    }
    if (lane == 31) tops[warp] = lo;
    __syncthreads();
    for (int w = 0; w < warp; ++w) lo = max(lo, tops[w]);
    const int hi = is_group ? max(lo, next) : lo;
    int prefix = 0;
    if (is_group) {
        if (lo != at || hi != next || prefix_in < 0) record_status(&g_status, kPagedInput);
        if (lo < hi) prefix = clamped(prefix_in, 0, lens[lo], true);
        los[tid] = lo;
        his[tid] = hi;
        given[tid] = prefix;
    }
    const int group_rows = (hi - lo) * p.rows;
    const int blocks = p.items && prefix > 0 ? (group_rows + p.nb - 1) / p.nb : 0, units = (prefix + p.keys - 1) / p.keys;
    __syncthreads();
    // A group's number of items and units needs no other group's; its sequences do
    // need its prefix.
    for (int i = warp; i < n_groups; i += warps)
        for (int s = los[i] + lane; s < his[i]; s += 32) {
            firsts[s] = los[i];
            prefixes[s] = given[i];
            prefix_items[s] = given[i] > 0 ? i : -1;         // the group, for now
        }
    __syncthreads();
    const int from = prefixes[tid], own_units = is_seq && len > from ? (len + p.keys - 1) / p.keys - from / p.keys : 0;
    if (is_seq) {
        if (dbg_in_bytes(g.first + tid, 4, g.sw, &g_status)) g.first[tid] = firsts[tid];
        if (dbg_in_bytes(g.prefix + tid, 4, g.sw, &g_status)) g.prefix[tid] = from;
    }
    if (!p.items) return;
    // Running sums: own units over the sequences, prefix units and items over the groups.
    const int own_cost = latent_item_cost(own_units);
    Sums v{own_cost * p.own, blocks * latent_item_cost(units), blocks};
    const Sums self = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(~0u, v.own, o), y = __shfl_up_sync(~0u, v.units, o), z = __shfl_up_sync(~0u, v.items, o);
        if (lane >= o) {
            v.own += x;
            v.units += y;
            v.items += z;
        }
    }
    if (lane == 31) sums[warp] = v;
    __syncthreads();
    Sums all{0, 0, 0}, before{0, 0, 0};
    for (int w = 0; w < warps; ++w) {
        const Sums x = sums[w];
        all.own += x.own;
        all.units += x.units;
        all.items += x.items;
        if (w < warp) {
            before.own += x.own;
            before.units += x.units;
            before.items += x.items;
        }
    }
    auto put_item = [&](int i, const LatentItem& it) {
        if (dbg_in_bytes(p.items + i, sizeof(it), g.sw, &g_status)) p.items[i] = it;
    };
    if (is_seq)
        for (int k = 0; k < p.own; ++k)
            put_item(tid * p.own + k, LatentItem{before.own + v.own - self.own + k * own_cost, own_units, tid, from, len, tid,
                                                 k * p.nb, min(p.nb, p.rows - k * p.nb)});
    // The groups' places, where their starts were.
    __syncthreads();
    int* unit_of = lens;
    int* item_of = firsts;
    if (is_group) {
        unit_of[tid] = all.own + before.units + v.units - self.units;
        item_of[tid] = n_seqs * p.own + before.items + v.items - self.items;
    }
    __syncthreads();
    if (is_seq) {
        const int of = prefix_items[tid];
        if (dbg_in_bytes(p.prefix_item + tid, 4, g.sw, &g_status)) p.prefix_item[tid] = of < 0 ? -1 : item_of[of];
    }
    for (int i = warp; i < n_groups; i += warps) {
        const int keys = given[i], rows = (his[i] - los[i]) * p.rows, n = (keys + p.keys - 1) / p.keys;
        if (keys <= 0) continue;
        for (int k = lane; k * p.nb < rows; k += 32)
            put_item(item_of[i] + k, LatentItem{unit_of[i] + k * latent_item_cost(n), n, los[i], 0, keys, los[i], k * p.nb,
                                                min(p.nb, rows - k * p.nb)});
    }
    if (tid == 0 && dbg_in_bytes(p.head, 8, g.sw, &g_status)) {
        p.head[0] = all.own + all.units;
        p.head[1] = n_seqs * p.own + all.items;
    }
}

size_t round256(size_t n) { return (n + 255) / 256 * 256; }

// What goes where in the workspace: arrays of a number a sequence (first, prefix,
// prefix_item), the head, the items, and a slot for every piece: an item that begins
// in a CTA has its index and the CTA's as its slot, so that there are as many as
// items and CTAs together.
struct Layout {
    int nb;
    int64_t own, most;                   // items of a sequence's own keys; items at most
    size_t each, items, parts, bytes;    // bytes an array; offsets
};
Layout layout_with(int nb, int sms, int64_t n_seqs, int64_t n_groups, int64_t rows, int64_t R) {
    Layout l{};
    l.nb = nb;
    l.own = (rows + l.nb - 1) / l.nb;
    l.most = n_seqs * l.own + n_seqs * rows / l.nb + n_groups;
    l.each = round256((size_t)n_seqs * 4);
    l.items = 3 * l.each + 256;
    l.parts = l.items + round256((size_t)l.most * sizeof(LatentItem));
    l.bytes = l.parts + (R > 0 ? (size_t)(l.most + sms) * latent_part_bytes(l.nb, R) : 0);
    return l;
}
Layout layout_of(int sms, int64_t n_seqs, int64_t n_groups, int64_t rows, int64_t R) {
    // Rows that a group has, were they all alike.
    const int64_t of = n_groups > 0 ? (n_seqs + n_groups - 1) / n_groups * rows : rows;
    return layout_with(latent_rows_block(std::max(of, rows)), sms, n_seqs, n_groups, rows, R);
}

}  // namespace

// What any call of up to these sizes needs: a block's query rows follow from the sizes
// (fewer groups have more rows each, and larger slots), and for one number of them
// nothing shrinks as the sizes grow.
size_t latent_shared_workspace_bytes(int sms, int64_t n_seqs, int64_t n_groups, int64_t q_len, int64_t heads, int64_t R) {
    const int64_t rows = q_len * heads;
    size_t most = 0;
    for (const int nb : {16, 32, 64}) {
        if (nb > latent_rows_block(n_seqs * rows)) break;
        most = std::max(most, layout_with(nb, sms, n_seqs, n_groups, rows, R).bytes);
    }
    return most;
}

cudaError_t launch_latent_shared(const LatentPaged& a, const int32_t* group_starts, const int32_t* prefix_lens,
                                 int64_t n_groups, int sms, cudaStream_t stream) {
    const int64_t rows = a.q_len * a.heads;
    const Layout l = layout_of(sms, a.n_seqs, n_groups, rows, a.R);
    char* ws = static_cast<char*>(a.workspace);
    PrefixPlan p{};
    p.g = LatentShared{a, group_starts, prefix_lens, n_groups, reinterpret_cast<int32_t*>(ws),
                       reinterpret_cast<int32_t*>(ws + l.each),
                       ByteSpan{reinterpret_cast<uintptr_t>(ws), reinterpret_cast<uintptr_t>(ws) + l.bytes}};
    p.nb = l.nb;
    p.keys = latent_block_keys(l.nb);
    p.rows = (int)rows;
    p.own = (int)l.own;
    // (Units and slots are ints.)
    const bool tc = latent_decode_takes(a) && (__int128)l.most * (a.N / p.keys + 2 + kLatentItemPad) < INT32_MAX &&
                    a.n_seqs * rows < INT32_MAX / 2;
    if (tc) {
        p.prefix_item = reinterpret_cast<int32_t*>(ws + 2 * l.each);
        p.head = reinterpret_cast<int32_t*>(ws + 3 * l.each);
        p.items = reinterpret_cast<LatentItem*>(ws + l.items);
    }
    cudaLaunchAttribute early{};
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(1);
    const int64_t most = std::max(a.n_seqs, n_groups);
    const bool small = most <= kPlanThreads;
    cfg.blockDim = dim3(small ? (unsigned)(most + 31) / 32 * 32 : kPlanThreads);
    cfg.stream = stream;
    cfg.attrs = &early;
    cfg.numAttrs = 1;
    if (const cudaError_t e = cudaLaunchKernelEx(&cfg, small ? small_plan_kernel : plan_kernel, p)) return e;
    if (!tc) return launch_latent_rows_shared(p.g, stream);
    const LatentItems items{p.g.first, p.prefix_item, p.head, p.items, p.own, (int)l.most};
    return launch_latent_decode_shared(a, items, l.nb, ws + l.parts, sms, stream);
}

unsigned int* status_word_latent_shared() { return word_address(&g_status); }

}  // namespace sbg
