// bss_host.h -- host side of the row operators around the attention step:
// alignment, launch sizes and the overlap of strided tensors.  No device code, so
// that a host program can compile and check it.
#pragma once
#include <cuda_runtime_api.h>

#include <cstdint>
#include <mutex>

#include "bss_internal.h"

namespace bss {

inline bool is_aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Blocks of a kernel that an SM holds at once with this much dynamic shared memory;
// the kernel may use it afterwards.  A kernel's limit is always set to all that a
// block may have beside the kernel's static memory, never to the size at hand: calls
// of other sizes, also in other threads, then leave it as it is.  (Below 48 KiB too:
// what a kernel may use unasked includes its static memory.)  The runtime is asked
// once per kernel, size and device, as long as the answer is among those kept: the
// last so many.
inline bss_status resident_blocks(const void* kernel, int threads, int smem, int* blocks) {
    struct Known {
        const void* kernel;
        int device, threads, smem, blocks;
    };
    constexpr int kKept = 512;
    static std::mutex mutex;
    static Known known[kKept];
    static int count = 0, next = 0;
    int device = 0;
    bss_status st = cuda_check(cudaGetDevice(&device), "current device");
    if (st != BSS_OK) return st;
    {
        std::lock_guard<std::mutex> lock(mutex);
        for (int i = 0; i < count; ++i) {
            const Known& k = known[i];
            if (k.kernel == kernel && k.device == device && k.threads == threads && k.smem == smem) {
                *blocks = k.blocks;
                return BSS_OK;
            }
        }
    }
    cudaFuncAttributes attributes = {};
    st = cuda_check(cudaFuncGetAttributes(&attributes, kernel), "kernel attributes");
    int most = 0, n = 0;
    if (st == BSS_OK)
        st = cuda_check(cudaDeviceGetAttribute(&most, cudaDevAttrMaxSharedMemoryPerBlockOptin, device), "shared memory of a block");
    most -= static_cast<int>(attributes.sharedSizeBytes);
    if (st == BSS_OK && attributes.maxDynamicSharedSizeBytes != most)
        st = cuda_check(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most), "shared memory size");
    if (st == BSS_OK)
        st = cuda_check(cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, threads, smem), "occupancy");
    if (st != BSS_OK) return st;
    *blocks = n < 1 ? 1 : n;
    std::lock_guard<std::mutex> lock(mutex);
    known[next] = {kernel, device, threads, smem, *blocks};
    next = (next + 1) % kKept;
    if (count < kKept) ++count;
    return BSS_OK;
}

// The bytes that a strided tensor touches: n0 times n1 runs of `width` bytes, s0 and
// s1 bytes apart (s0 the larger stride; a dimension of size 1 has stride 0).  Runs
// that touch or overlap are taken as one; where the n1 runs of one step reach into the
// next step's, or overlap it, the whole extent counts as one run.
struct Region {
    uintptr_t lo = 0;
    int64_t n0 = 0, s0 = 0, n1 = 1, s1 = 0, width = 0;
    bool self_overlap = false;  // the tensor names a byte twice, or its steps are interlaced
    int64_t inner() const { return (n1 - 1) * s1 + width; }
    uintptr_t hi() const { return lo + static_cast<uintptr_t>((n0 - 1) * s0 + inner()); }
    bool same_bytes(const Region& o) const {
        return lo == o.lo && n0 == o.n0 && s0 == o.s0 && n1 == o.n1 && s1 == o.s1 && width == o.width;
    }
};

// [n0][n1][width] elements with strides s0, s1
inline Region region_3d(const void* p, int64_t n0, int64_t s0, int64_t n1, int64_t s1, int64_t width, int64_t esize) {
    if (n0 <= 1) s0 = 0;
    if (n1 <= 1) s1 = 0;
    if (n1 > 1 && (n0 <= 1 || s1 > s0)) {
        int64_t t = n0;
        n0 = n1, n1 = t;
        t = s0, s0 = s1, s1 = t;
    }
    Region r;
    r.lo = reinterpret_cast<uintptr_t>(p);
    const int64_t inner = (n1 - 1) * s1 + width;
    r.self_overlap = (n1 > 1 && s1 < width) || (n0 > 1 && s0 < inner);
    if (n1 > 1 && s1 <= width) n1 = 1, s1 = 0, width = inner;
    if (n0 > 1 && s0 < inner) {
        width = (n0 - 1) * s0 + inner;
        n0 = n1 = 1, s0 = s1 = 0;
    }
    r.n0 = n0, r.s0 = s0 * esize;
    r.n1 = n1, r.s1 = s1 * esize;
    r.width = width * esize;
    return r;
}

// rows x width elements
inline Region region_2d(const void* p, int64_t rows, int64_t stride, int64_t width, int64_t esize) {
    return region_3d(p, rows, stride, 1, 0, width, esize);
}

// Whether two tensors certainly share no byte.  Exact for views of one tensor, whose
// strides are the same (column ranges of its rows, the Q, K and V of a projection
// packed token by token or head by head); others are told apart by their ends alone.
inline bool disjoint(const Region& a, const Region& b) {
    if (a.hi() <= b.lo || b.hi() <= a.lo) return true;
    if (a.n0 <= 1 || b.n0 <= 1 || a.s0 != b.s0 || (a.n1 > 1 && b.n1 > 1 && a.s1 != b.s1)) return false;
    // a run of b starts d + i s0 + j s1 bytes behind one of a, for |i| < n0 and |j| < n1;
    // a step's runs span at most s0, so few i come near
    const int64_t s0 = a.s0, s1 = a.n1 > 1 ? a.s1 : b.s1;
    const int64_t d = b.lo >= a.lo ? static_cast<int64_t>(b.lo - a.lo) : -static_cast<int64_t>(a.lo - b.lo);
    auto first_above = [](int64_t from, int64_t step, int64_t bound) {  // the least k with from + k step > bound
        const int64_t t = bound - from;
        return (t >= 0 ? t / step : -((-t + step - 1) / step)) + 1;
    };
    int64_t i = first_above(d, s0, -b.inner());
    if (i < 1 - a.n0) i = 1 - a.n0;
    for (; i < b.n0 && d + i * s0 < a.inner(); ++i) {
        const int64_t at = d + i * s0;
        int64_t j = s1 > 0 ? first_above(at, s1, -b.width) : 0;
        if (j < 1 - a.n1) j = 1 - a.n1;
        if (j < b.n1 && at + j * s1 > -b.width && at + j * s1 < a.width) return false;
    }
    return true;
}

}  // namespace bss
