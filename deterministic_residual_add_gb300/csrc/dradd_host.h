// dradd_host.h -- what the C entry points share on the host: device limits,
// the kind of memory behind a pointer, and the byte ranges of buffers.  Not
// part of the public interface.
#pragma once

#include <atomic>
#include <cstdint>
#include <initializer_list>

#include <cuda_runtime.h>

#include "dradd.h"

namespace dradd {

constexpr int kMaxDevices = 64;
constexpr uint64_t kDefaultWaitLimitNs = 1000000000ull;  // 1 s

// Shared-memory and thread limits used to size grids and stages.  Defaults
// are GB300's; with a live device they come from the device.
struct DeviceLimits {
    int sm_count = 152;
    int smem_per_block_optin = 232448;  // 227 KiB
    int smem_per_sm = 233472;           // 228 KiB
    int max_threads_per_sm = 2048;
    int max_blocks_per_sm = 32;
};

inline std::atomic<int> g_limits_ready[kMaxDevices];
inline DeviceLimits g_limits[kMaxDevices];

inline dradd_status query_limits(DeviceLimits* out)
{
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess)
        return DRADD_ERR_CUDA;
    if (dev >= 0 && dev < kMaxDevices && g_limits_ready[dev].load(std::memory_order_acquire)) {
        *out = g_limits[dev];
        return DRADD_OK;
    }
    DeviceLimits L;
    if (cudaDeviceGetAttribute(&L.sm_count, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&L.smem_per_block_optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev) !=
            cudaSuccess ||
        cudaDeviceGetAttribute(&L.smem_per_sm, cudaDevAttrMaxSharedMemoryPerMultiprocessor, dev) !=
            cudaSuccess ||
        cudaDeviceGetAttribute(&L.max_threads_per_sm, cudaDevAttrMaxThreadsPerMultiProcessor, dev) !=
            cudaSuccess ||
        cudaDeviceGetAttribute(&L.max_blocks_per_sm, cudaDevAttrMaxBlocksPerMultiprocessor, dev) !=
            cudaSuccess)
        return DRADD_ERR_CUDA;
    if (dev >= 0 && dev < kMaxDevices) {
        g_limits[dev] = L;  // identical values if two threads race here
        g_limits_ready[dev].store(1, std::memory_order_release);
    }
    *out = L;
    return DRADD_OK;
}

// True when every non-NULL pointer is device memory.  Other memory the GPU
// can address (pinned or registered host memory, memory the GPU reaches
// through the host link, managed memory) is served by the register-load
// variant only: the staged variant's bulk copies are used on device memory.
inline bool all_device_memory(std::initializer_list<const void*> ptrs)
{
    for (const void* p : ptrs) {
        if (!p)
            continue;
        cudaPointerAttributes a;
        if (cudaPointerGetAttributes(&a, p) != cudaSuccess) {
            cudaGetLastError();  // not a sticky error; the pointer is simply not device memory
            return false;
        }
        if (a.type != cudaMemoryTypeDevice)
            return false;
    }
    return true;
}

// Byte ranges of the buffers of one call, for the overlap rules.
struct Range {
    uintptr_t lo = 0, hi = 0;  // [lo, hi)
    bool overlaps(const Range& o) const { return lo < o.hi && o.lo < hi; }
    bool same(const Range& o) const { return lo == o.lo && hi == o.hi; }
};

inline Range range_of(const void* p, int64_t bytes)
{
    Range r;
    r.lo = reinterpret_cast<uintptr_t>(p);
    r.hi = r.lo + static_cast<uintptr_t>(bytes);
    return r;
}

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// ------------------------------------------------------------ strided views
// A tensor of up to four dimensions with strides in elements; the last
// dimension of a real tensor has stride 1.
struct View {
    uintptr_t base = 0;
    int64_t elem = 1;
    int nd = 0;
    int64_t size[4] = {}, stride[4] = {};

    // Dimensions of more than one element, largest stride first.
    void add(int64_t n, int64_t s)
    {
        if (n <= 1)
            return;
        int i = nd++;
        for (; i > 0 && stride[i - 1] < s; --i) {
            size[i] = size[i - 1];
            stride[i] = stride[i - 1];
        }
        size[i] = n;
        stride[i] = s;
    }
    // Bytes from the first to past the last element of dimensions from, ...
    // (sizes and strides whose view_fits holds).
    int64_t span(int from = 0) const
    {
        int64_t e = 1;
        for (int i = from; i < nd; ++i)
            e += (size[i] - 1) * stride[i];
        return e * elem;
    }
    bool same(const View& o) const
    {
        if (base != o.base || elem != o.elem || nd != o.nd)
            return false;
        for (int i = 0; i < nd; ++i)
            if (size[i] != o.size[i] || stride[i] != o.stride[i])
                return false;
        return true;
    }
};

// Whether strides are >= 0 and every offset stays far inside 64 bits.
inline bool view_fits(const View& v)
{
    __int128 e = 1;
    for (int i = 0; i < v.nd; ++i) {
        if (v.stride[i] < 0 || v.size[i] < 0)
            return false;
        e += static_cast<__int128>(v.size[i] - 1) * v.stride[i];
        if (e > (static_cast<__int128>(1) << 58))
            return false;
    }
    return true;
}

// Whether two elements of one view may share memory.
inline bool view_overlaps_itself(const View& v)
{
    for (int i = 0; i < v.nd; ++i)
        if (v.stride[i] * v.elem < v.span(i + 1))
            return true;
    return false;
}

// Whether two views may share memory.  Disjoint byte ranges do not.  Where
// the ranges meet, the outermost dimensions have to agree in size and
// stride, and the rest of both views has to lie within one stride of it, so
// that only parts with the same index can meet; then the rest decides.
inline bool views_may_overlap(const View& a, const View& b)
{
    for (int i = 0;; ++i) {
        const uintptr_t a_end = a.base + static_cast<uintptr_t>(a.span(i));
        const uintptr_t b_end = b.base + static_cast<uintptr_t>(b.span(i));
        if (a_end <= b.base || b_end <= a.base)
            return false;
        if (i >= a.nd || i >= b.nd || a.size[i] != b.size[i] || a.stride[i] * a.elem != b.stride[i] * b.elem)
            return true;
        const uintptr_t lo = a.base < b.base ? a.base : b.base;
        const uintptr_t a_in = a.base + static_cast<uintptr_t>(a.span(i + 1));
        const uintptr_t b_in = b.base + static_cast<uintptr_t>(b.span(i + 1));
        if ((a_in > b_in ? a_in : b_in) - lo > static_cast<uintptr_t>(a.stride[i] * a.elem))
            return true;
    }
}

}  // namespace dradd
