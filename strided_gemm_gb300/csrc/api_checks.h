// Checks of arguments that the C entry points of the serving and layer operators
// share: spans, overlaps, device memory, options.
#pragma once

#include <cuda_runtime.h>

#include <algorithm>
#include <array>
#include <climits>
#include <initializer_list>

#include "internal.h"
#include "sbgemm.h"

namespace sbg {

using i128 = __int128;

inline bool aligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// Bytes [lo, hi) that an operand occupies.
struct Bytes { i128 lo, hi; };

struct Axis { int64_t stride, extent; };

// The bytes of an array of `esize`-byte elements over the axes' box (extents
// positive).  False if offsets do not fit comfortably in int64 bytes.
inline bool span_of(const void* base, int64_t esize, std::initializer_list<Axis> axes, Bytes* out) {
    i128 lo = 0, hi = 0;
    for (const Axis& a : axes) {
        const i128 d = (i128)a.stride * (a.extent - 1);
        if (d < 0) lo += d;
        else hi += d;
    }
    const i128 limit = (i128)1 << 60;
    if (lo < -limit || hi > limit) return false;
    const i128 b = (i128)reinterpret_cast<uintptr_t>(base);
    *out = {b + lo * esize, b + (hi + 1) * esize};
    return true;
}

// Distinct indices have distinct elements: sorted by stride, each stride
// exceeds what the smaller ones reach (sufficient, as for the fp32 product).
template <size_t n>
bool injective(std::array<Axis, n> a) {
    for (Axis& x : a) x.stride = x.stride < 0 ? -x.stride : x.stride;
    std::sort(a.begin(), a.end(), [](const Axis& x, const Axis& y) { return x.stride < y.stride; });
    i128 reach = 0;
    for (const Axis& x : a) {
        if (x.extent <= 1) continue;
        if ((i128)x.stride <= reach) return false;
        reach += (i128)x.stride * (x.extent - 1);
    }
    return true;
}

inline ByteSpan span_for_kernel(const Bytes& b) { return {(uintptr_t)b.lo, (uintptr_t)b.hi}; }

inline bool meet(const Bytes& a, const Bytes& b) { return a.lo < b.hi && b.lo < a.hi; }

// Each span lies inside one device-accessible allocation.  An allocation seen
// before in this call is not looked up again.
inline int in_device_memory(const Bytes* spans, size_t count) {
    std::array<Bytes, 8> seen;
    size_t n = 0;
    for (size_t k = 0; k < count; ++k) {
        const Bytes& s = spans[k];
        bool known = false;
        for (size_t i = 0; i < n && !known; ++i) known = s.lo >= seen[i].lo && s.hi <= seen[i].hi;
        if (known) continue;
        uintptr_t base = 0;
        size_t size = 0;
        if (!device_allocation_range(reinterpret_cast<const void*>((uintptr_t)s.lo), &base, &size))
            return SBGEMM_ERR_NOT_DEVICE_MEMORY;
        const Bytes a{(i128)base, (i128)base + (i128)size};
        if (s.lo < a.lo || s.hi > a.hi) return SBGEMM_ERR_NOT_DEVICE_MEMORY;
        if (n < seen.size()) seen[n++] = a;
    }
    return SBGEMM_OK;
}

inline int in_device_memory(std::initializer_list<Bytes> spans) { return in_device_memory(spans.begin(), spans.size()); }

// The options these operators read: a workspace, and no forced path.
inline int read_options(const sbgemm_options* opt, void** ws, size_t* bytes) {
    *ws = nullptr;
    *bytes = 0;
    if (!opt) return SBGEMM_OK;
    if (opt->math != SBGEMM_MATH_FP32 && opt->math != SBGEMM_MATH_TF32) return SBGEMM_ERR_INVALID_VALUE;
    if (opt->force_path < SBGEMM_PATH_AUTO || opt->force_path > SBGEMM_PATH_TMA_TF32)
        return SBGEMM_ERR_INVALID_VALUE;
    if (opt->force_path != SBGEMM_PATH_AUTO) return SBGEMM_ERR_UNSUPPORTED;
    if (opt->k_split < SBGEMM_KSPLIT_ANY || opt->k_split > SBGEMM_KSPLIT_NONE) return SBGEMM_ERR_INVALID_VALUE;
    for (int r : opt->reserved)
        if (r != 0) return SBGEMM_ERR_INVALID_VALUE;
    if (opt->workspace) {
        if (!aligned(opt->workspace, 256)) return SBGEMM_ERR_INVALID_VALUE;
        *ws = opt->workspace;
        *bytes = opt->workspace_bytes;
    }
    return SBGEMM_OK;
}

inline Bytes block(const void* p, int64_t bytes) {
    const i128 b = (i128)reinterpret_cast<uintptr_t>(p);
    return {b, b + bytes};
}

// The SMs of the current device, 0 on a CUDA error.
inline int current_sms() {
    int dev = 0;
    if (cudaGetDevice(&dev) == cudaSuccess) {
        if (const DeviceProps* d = device_props(dev)) return d->sm_count;
    }
    cudaGetLastError();
    return 0;
}

inline int finish(cudaError_t e) {
    if (e == cudaSuccess) return SBGEMM_OK;
    cudaGetLastError();
    return SBGEMM_ERR_CUDA;
}

constexpr int64_t kInt = INT_MAX;

}  // namespace sbg
