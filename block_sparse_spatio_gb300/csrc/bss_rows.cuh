// bss_rows.cuh -- what the row operators around the attention step share:
// 8-channel vectors and packed arithmetic, sums over parts of a block and the
// launch of a kernel behind another (the rest of the host side: bss_host.h).
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "bss_block.h"
#include "bss_host.h"
#include "bss_internal.h"
#include "bss_ptx.cuh"

namespace bss {

// ---------------------------------------------------------------- vectors
// Row data is read once: keep it out of L1.
__device__ __forceinline__ uint4 ld_row(const void* p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p)
                 : "memory");
    return v;
}

__device__ __forceinline__ void st_row(void* p, const uint4& v) {
    asm volatile("st.global.cs.v4.u32 [%0], {%1,%2,%3,%4};" ::"l"(p), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
                 : "memory");
}

__device__ __forceinline__ uint32_t pack2(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// Parameters (weights, modulations) are shared by many rows: read through L1.
__device__ __forceinline__ void load_param8(const void* base, int64_t index, int dtype, float (&v)[8]) {
    if (dtype == BSS_DTYPE_F32) {
        const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + index);
        const float4 a = __ldg(p), b = __ldg(p + 1);
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
        const uint4 q = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(base) + index));
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
}

__device__ __forceinline__ float load_param(const void* base, int64_t index, int dtype) {
    return dtype == BSS_DTYPE_F32 ? __ldg(static_cast<const float*>(base) + index)
                                  : __bfloat162float(static_cast<const __nv_bfloat16*>(base)[index]);
}

// ---------------------------------------------------------------- packed arithmetic
// 8 channels as four pairs, computed two at a time (fma.rn.f32x2).
struct V8 {
    float2 p[4];
};

__device__ __forceinline__ float2 f2(float a) { return make_float2(a, a); }

// Pairs (0,1) (2,3) (4,5) (6,7), or for EO the even and odd channels apart:
// (0,2) (1,3) (4,6) (5,7).
template <bool EO>
__device__ __forceinline__ V8 unpack_bf16(const uint4& q) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
    V8 v;
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
        const float l0 = __uint_as_float(w[i] << 16), h0 = __uint_as_float(w[i] & 0xFFFF0000u);
        const float l1 = __uint_as_float(w[i + 1] << 16), h1 = __uint_as_float(w[i + 1] & 0xFFFF0000u);
        v.p[i] = EO ? make_float2(l0, l1) : make_float2(l0, h0);
        v.p[i + 1] = EO ? make_float2(h0, h1) : make_float2(l1, h1);
    }
    return v;
}

template <bool EO>
__device__ __forceinline__ uint4 pack_bf16(const V8& v) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
        w[i] = EO ? pack2(v.p[i].x, v.p[i + 1].x) : pack2(v.p[i].x, v.p[i].y);
        w[i + 1] = EO ? pack2(v.p[i].y, v.p[i + 1].y) : pack2(v.p[i + 1].x, v.p[i + 1].y);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

template <bool EO>
__device__ __forceinline__ V8 arrange(const float (&f)[8]) {
    V8 v;
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
        v.p[i] = EO ? make_float2(f[2 * i], f[2 * i + 2]) : make_float2(f[2 * i], f[2 * i + 1]);
        v.p[i + 1] = EO ? make_float2(f[2 * i + 1], f[2 * i + 3]) : make_float2(f[2 * i + 2], f[2 * i + 3]);
    }
    return v;
}

// The channel of pair i's first and second value.
template <bool EO>
__device__ __forceinline__ int channel_of(int i, int second) {
    return EO ? (i & 2) * 2 + (i & 1) + 2 * second : 2 * i + second;
}

__device__ __forceinline__ float dot(const V8& a, const V8& b) {
    float2 s = __fmul2_rn(a.p[0], b.p[0]);
#pragma unroll
    for (int i = 1; i < 4; ++i) s = __ffma2_rn(a.p[i], b.p[i], s);
    return s.x + s.y;
}

__device__ __forceinline__ V8 mul(const V8& a, const V8& b) {
    V8 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r.p[i] = __fmul2_rn(a.p[i], b.p[i]);
    return r;
}

__device__ __forceinline__ V8 mul(const V8& a, float b) {
    V8 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r.p[i] = __fmul2_rn(a.p[i], f2(b));
    return r;
}

// a * b + c
__device__ __forceinline__ V8 fma8(const V8& a, const V8& b, const V8& c) {
    V8 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r.p[i] = __ffma2_rn(a.p[i], b.p[i], c.p[i]);
    return r;
}

__device__ __forceinline__ V8 fma8(const V8& a, float b, const V8& c) {
    V8 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r.p[i] = __ffma2_rn(a.p[i], f2(b), c.p[i]);
    return r;
}

// ---------------------------------------------------------------- sums
// Sum over aligned groups of L lanes (L a power of two); every lane gets it.
template <int L>
__device__ __forceinline__ float lane_sum(float v) {
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// Sums of NV values over aligned groups of L lanes, NV <= L: while there are
// several values left the two halves of the group keep half of them each, so NV
// sums cost little more than one.  A lane ends with the sum of value
// scattered_index<NV, L>(lane).
template <int NV, int L>
__device__ __forceinline__ float scatter_sum(float (&v)[NV]) {
    int o = L / 2;
#pragma unroll
    for (int n = NV / 2; n >= 1; n /= 2, o /= 2) {
        const bool upper = (threadIdx.x & o) != 0;
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const float send = upper ? v[i] : v[i + n];
            v[i] = (upper ? v[i + n] : v[i]) + __shfl_xor_sync(0xFFFFFFFFu, send, o);
        }
    }
    if constexpr (NV < L)
#pragma unroll
        for (; o > 0; o /= 2) v[0] += __shfl_xor_sync(0xFFFFFFFFu, v[0], o);
    return v[0];
}

// The value a lane holds after scatter_sum, and whether it is the one to write it.
template <int NV, int L>
__device__ __forceinline__ int scattered_index() {
    return static_cast<int>(threadIdx.x % L) / (L / NV);
}
template <int NV, int L>
__device__ __forceinline__ bool scattered_writer() {
    return threadIdx.x % (L / NV) == 0;
}

// ---------------------------------------------------------------- integer division
// n / d for n < 2^31 by a multiplication (division by an invariant integer after
// Granlund and Montgomery, 1994): with 2^(L-1) < d <= 2^L and
// m = floor(2^32 (2^L - d) / d) + 1, n / d = (n m / 2^32 + n) / 2^L.
struct FastDiv {
    uint32_t d, m, shift;
    FastDiv() = default;
    explicit FastDiv(uint32_t by) : d(by), m(0), shift(0) {
        while (shift < 31 && (1u << shift) < by) ++shift;
        m = static_cast<uint32_t>(((uint64_t(1) << 32) * ((uint64_t(1) << shift) - by)) / by + 1);
    }
    __device__ __forceinline__ uint32_t div(uint32_t n) const { return (__umulhi(n, m) + n) >> shift; }
};

// ---------------------------------------------------------------- host side
// A kernel launched behind another one of the same stream, its launch overlapping
// that one's end: it calls cudaGridDependencySynchronize() before it reads what
// the other wrote, or writes anything.  With this much dynamic shared memory, in
// clusters of so many blocks.
template <typename... Params, typename... Args>
bss_status launch_behind_with(void (*kernel)(Params...), dim3 grid, int threads, int smem, int cluster, cudaStream_t stream,
                              const char* what, const Args&... args) {
    cudaLaunchConfig_t config = {};
    config.gridDim = grid;
    config.blockDim = dim3(static_cast<unsigned>(threads));
    config.dynamicSmemBytes = static_cast<size_t>(smem);
    config.stream = stream;
    cudaLaunchAttribute attributes[2] = {};
    attributes[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attributes[0].val.programmaticStreamSerializationAllowed = 1;
    attributes[1].id = cudaLaunchAttributeClusterDimension;
    attributes[1].val.clusterDim.x = static_cast<unsigned>(cluster);
    attributes[1].val.clusterDim.y = attributes[1].val.clusterDim.z = 1;
    config.attrs = attributes;
    config.numAttrs = cluster > 1 ? 2 : 1;
    return cuda_check(cudaLaunchKernelEx(&config, kernel, static_cast<Params>(args)...), what);
}

template <typename... Params, typename... Args>
bss_status launch_behind(void (*kernel)(Params...), dim3 grid, int threads, cudaStream_t stream, const char* what,
                         Args... args) {
    return launch_behind_with(kernel, grid, threads, 0, 1, stream, what, args...);
}

}  // namespace bss
