// Host program of the checks in bss_host.h: disjoint() against the bytes of small
// strided tensors, and launch sizes against a runtime that keeps each kernel's limit.
#include <atomic>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <set>
#include <thread>
#include <vector>

#include "bss_host.h"

namespace bss {
bss_status set_error(bss_status st, const char*, ...) { return st; }
bss_status cuda_check(cudaError_t e, const char*) { return e == cudaSuccess ? BSS_OK : BSS_ERR_CUDA; }
}  // namespace bss

// The runtime, as far as it is asked: kernels with their static memory and limit.
namespace {
constexpr int kOptin = 232448, kKernels = 4;
struct Kernel {
    std::atomic<int> limit{48 * 1024};
    std::atomic<int> asked{0};
    int fixed = 0;
} kernels[kKernels];
Kernel& of(const void* k) { return kernels[reinterpret_cast<uintptr_t>(k) - 1]; }
}  // namespace
extern "C" {
cudaError_t cudaGetDevice(int* device) { return *device = 0, cudaSuccess; }
cudaError_t cudaDeviceGetAttribute(int* v, cudaDeviceAttr a, int) {
    *v = kOptin;
    return a == cudaDevAttrMaxSharedMemoryPerBlockOptin ? cudaSuccess : cudaErrorInvalidValue;
}
cudaError_t cudaFuncGetAttributes(cudaFuncAttributes* a, const void* k) {
    *a = {};
    a->sharedSizeBytes = of(k).fixed;
    a->maxDynamicSharedSizeBytes = of(k).limit;
    return cudaSuccess;
}
cudaError_t cudaFuncSetAttribute(const void* k, cudaFuncAttribute a, int v) {
    if (a != cudaFuncAttributeMaxDynamicSharedMemorySize || v + of(k).fixed > kOptin) return cudaErrorInvalidValue;
    of(k).limit = v;
    return cudaSuccess;
}
cudaError_t cudaOccupancyMaxActiveBlocksPerMultiprocessor(int* n, const void* k, int, size_t smem) {
    ++of(k).asked;
    *n = (kOptin + 1024) / (static_cast<int>(smem) + of(k).fixed + 1024);
    return cudaSuccess;
}
}

namespace {

uint64_t state = 1;
int64_t random_to(int64_t n) {  // 0 .. n
    state = state * 6364136223846793005ull + 1442695040888963407ull;
    return static_cast<int64_t>((state >> 33) % static_cast<uint64_t>(n + 1));
}

struct Tensor {
    int64_t at, n0, s0, n1, s1, width;
    std::multiset<int64_t> bytes() const {
        std::multiset<int64_t> b;
        for (int64_t i = 0; i < n0; ++i)
            for (int64_t j = 0; j < n1; ++j)
                for (int64_t c = 0; c < width; ++c) b.insert(at + i * s0 + j * s1 + c);
        return b;
    }
    bss::Region region() const {
        return bss::region_3d(reinterpret_cast<const void*>(static_cast<uintptr_t>(4096 + at)), n0, s0, n1, s1, width, 1);
    }
};

bool share(const Tensor& a, const Tensor& b) {
    const auto x = a.bytes();
    for (int64_t v : b.bytes())
        if (x.count(v)) return true;
    return false;
}

bool twice(const Tensor& a) {
    const auto x = a.bytes();
    for (int64_t v : x)
        if (x.count(v) > 1) return true;
    return false;
}

int fail(const char* what, const Tensor& a, const Tensor& b) {
    std::printf("%s: %lld [%lld %lld][%lld %lld] %lld, %lld [%lld %lld][%lld %lld] %lld\n", what, (long long)a.at,
                (long long)a.n0, (long long)a.s0, (long long)a.n1, (long long)a.s1, (long long)a.width, (long long)b.at,
                (long long)b.n0, (long long)b.s0, (long long)b.n1, (long long)b.s1, (long long)b.width);
    return 1;
}

// Random tensors: never called disjoint when they share a byte; and views of one
// tensor (whole steps, equal strides) always told apart when they do not.
int regions(int rounds) {
    int apart = 0, touching = 0;
    for (int k = 0; k < rounds; ++k) {
        Tensor a{random_to(40), 1 + random_to(3), random_to(24), 1 + random_to(3), random_to(24), 1 + random_to(5)};
        Tensor b{random_to(40), 1 + random_to(3), random_to(24), 1 + random_to(3), random_to(24), 1 + random_to(5)};
        if (random_to(2) > 0) b.s0 = a.s0, b.s1 = a.s1;
        if (bss::disjoint(a.region(), b.region()) && share(a, b)) return fail("called disjoint", a, b);
        if (bss::disjoint(a.region(), b.region()) != bss::disjoint(b.region(), a.region())) return fail("one way", a, b);
        if (twice(a) && !a.region().self_overlap) return fail("overlaps itself", a, a);
        // [n0][n1][gap] with either dimension outside, two ranges of the last
        const int64_t n0 = 2 + random_to(2), n1 = 1 + random_to(3), slot = 2 + random_to(8), pad = random_to(7);
        const int64_t outer = n1 * slot + pad;
        Tensor v[2];
        for (Tensor& t : v) {
            t.width = 1 + random_to(slot - 1);
            t.at = random_to(slot - t.width);
            t.n0 = n0, t.s0 = outer, t.n1 = n1, t.s1 = slot;
        }
        if (random_to(1)) {
            for (Tensor& t : v) std::swap(t.n0, t.n1), std::swap(t.s0, t.s1);
        }
        const bool hit = share(v[0], v[1]);
        (hit ? touching : apart) += 1;
        if (bss::disjoint(v[0].region(), v[1].region()) == hit) return fail("views of one tensor", v[0], v[1]);
    }
    std::printf("regions %d apart %d touching\n", apart, touching);
    return apart > rounds / 10 && touching > rounds / 10 ? 0 : 1;
}

bool may_launch(int kernel, int smem) {
    int blocks = 0;
    const void* k = reinterpret_cast<const void*>(static_cast<uintptr_t>(kernel + 1));
    return bss::resident_blocks(k, 128, smem, &blocks) == BSS_OK && blocks >= 1;
}

// More sizes than are kept, large ones followed by small ones: a kernel's limit covers
// its static memory and never falls below a size that was allowed (another thread may
// be about to launch it).
int limits() {
    for (int k = 0; k < kKernels; ++k) kernels[k].fixed = k * 700;
    for (int k = 0; k < kKernels; ++k) {
        for (int i = 0; i < 600; ++i)
            if (!may_launch(k, 64 + 32 * i)) return 1;
        const int large = kOptin - kernels[k].fixed;
        if (!may_launch(k, large) || kernels[k].limit < large) return 2;
        for (int i = 0; i < 600; ++i) {
            if (!may_launch(k, 96 + 16 * i)) return 3;
            if (kernels[k].limit < large) return 4;
        }
    }
    // a size in use is asked for once, whatever came before it
    const int before = kernels[0].asked;
    for (int i = 0; i < 100; ++i)
        if (!may_launch(0, 100000)) return 5;
    if (kernels[0].asked != before + 1) return 6;
    // threads with sizes of their own
    std::atomic<int> bad{0};
    std::vector<std::thread> threads;
    for (int t = 0; t < 4; ++t)
        threads.emplace_back([&bad, t] {
            for (int i = 0; i < 20000; ++i) {
                const int smem = t == 0 ? 200000 : 64 + (i * 4 + t) % 9001;
                if (!may_launch(1, smem) || kernels[1].limit < smem) ++bad;
            }
        });
    for (std::thread& t : threads) t.join();
    return bad == 0 ? 0 : 7;
}

}  // namespace

int main(int argc, char** argv) {
    if (argc > 1 && !std::strcmp(argv[1], "regions")) return regions(200000);
    if (argc > 1 && !std::strcmp(argv[1], "limits")) {
        const int bad = limits();
        std::printf("limits: check %d\n", bad);
        return bad;
    }
    return 2;
}
