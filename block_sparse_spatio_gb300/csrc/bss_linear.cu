// bss_linear.cu -- linear layers: a matrix product with bias, activation, gate and
// residual in its epilogue, and its gradients.
//
//   z = x W^T + b,  out = a residual + gate * act(z)
//   dz = gate * dout * act'(z),  dx = dz W,  dW = dz^T x,  db = sum dz,
//   dgate = sum over a group's rows of dout * act(z)
//
// All three products are D[m][n] = sum over k of A[m][k] B[n][k]; an operand whose
// k is contiguous is K-major in shared memory, one whose m (or n) is contiguous
// MN-major, so nothing is transposed in memory:
//   z   A = x [rows][in]     K-major   B = W [out][in]  K-major
//   dx  A = dz [rows][out]   K-major   B = W [out][in]  MN-major
//   dW  A = dz [rows][out]   MN-major  B = x [rows][in] MN-major
//
// 75,600 x 1,280 -> 5,120 with GELU 636 us, 75,600 x 5,120 -> 1,280 with gate and residual
// 630 (1,558 and 1,574 TFLOP/s, 90 and 91% of what cuBLAS sustains under the power limit,
// which bounds both); the gradients of the former 1,539 (dz 300, dx and dW about 610 each).
#include <cuda.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstring>
#include <type_traits>

#include "bss_args.h"
#include "bss_rows.cuh"

namespace bss {
namespace {

constexpr int kMaxWidth = 65536;

// ---------------------------------------------------------------- activations
__device__ __forceinline__ float rcp_approx(float x) {  // 1 / infinity = 0
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// 1 / (1 + 2^a); 2^a past the float range gives 0 or infinity and the quotient its limit.
__device__ __forceinline__ float2 share_of(float2 a) {
    const float2 e = __fadd2_rn(make_float2(ex2_approx(a.x), ex2_approx(a.y)), f2(1.0f));
    return make_float2(rcp_approx(e.x), rcp_approx(e.y));
}

// tanh form: (1 + tanh u) / 2 = 1 / (1 + exp(-2 u)), which keeps the small values of
// negative z exact to a few roundings (1 + tanh u does not).
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kTanhC = 1.5957691216057308f;  // 2 sqrt(2 / pi)
constexpr float kTanhD = 0.044715f;

// The share of z that passes, of SiLU and the tanh form: w = z^2.
template <int ACT>
__device__ __forceinline__ float2 smooth_share(float2 z, float2 w) {
    if constexpr (ACT == BSS_ACT_GELU_TANH)
        return share_of(__fmul2_rn(z, __ffma2_rn(w, f2(-kTanhC * kTanhD * kLog2e), f2(-kTanhC * kLog2e))));
    else
        return share_of(__fmul2_rn(z, f2(-kLog2e)));
}

// The error function's form: the share of -|z| is e(z) g(|z|) with e = exp(-z^2 / 2) and g =
// erfc(|z| / sqrt(2)) / (2 e), smooth and like 1 / |z| far out: t times a polynomial of
// degree 8 in t = 1 / (1 + 0.34 |z|), fitted for the least relative error over 0..14.5 (5.7e-8
// with the coefficients as floats, 3e-7 with its roundings; e is 0 behind).  75,600 x 1,280 ->
// 5,120 with a bias: 682 us (the tanh form 627, no activation 549), with erfcf in its place 1,175.
constexpr float kErfSlope = 0.34f;

__device__ __forceinline__ float2 erf_share(float2 z, float2& e) {
    constexpr float kErfFit[9] = {0.1356215775f, 0.1360922903f, 0.1153511703f, 0.1147158891f, -0.0431121476f,
                                  0.1997268051f, -0.2708797455f, 0.1383616030f, -0.0258774385f};
    const float2 w = __fmul2_rn(z, z), by = __ffma2_rn(make_float2(fabsf(z.x), fabsf(z.y)), f2(kErfSlope), f2(1.0f));
    const float2 t = make_float2(rcp_approx(by.x), rcp_approx(by.y)), u = __fmul2_rn(w, f2(-0.5f * kLog2e));
    e = make_float2(ex2_approx(u.x), ex2_approx(u.y));
    float2 g = f2(kErfFit[8]);
#pragma unroll
    for (int i = 7; i >= 0; --i) g = __ffma2_rn(g, t, f2(kErfFit[i]));
    const float2 low = __fmul2_rn(__fmul2_rn(e, t), g), high = __ffma2_rn(low, f2(-1.0f), f2(1.0f));
    return make_float2(z.x < 0.0f ? low.x : high.x, z.y < 0.0f ? low.y : high.y);
}

// (z times the share, not a quotient: with an infinite exponential the share is 0)
template <int ACT>
__device__ __forceinline__ float2 activate(float2 z) {
    if constexpr (ACT == BSS_ACT_GELU) {
        float2 e;
        return __fmul2_rn(z, erf_share(z, e));
    } else if constexpr (ACT != BSS_ACT_NONE) return __fmul2_rn(z, smooth_share<ACT>(z, __fmul2_rn(z, z)));
    else return z;
}

template <int ACT>
__device__ __forceinline__ float activate(float z) { return activate<ACT>(make_float2(z, 0.0f)).x; }

template <int ACT>
__device__ __forceinline__ void activate8(float (&v)[8]) {
    if constexpr (ACT != BSS_ACT_NONE) {
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            const float2 y = activate<ACT>(make_float2(v[i], v[i + 1]));
            v[i] = y.x, v[i + 1] = y.y;
        }
    }
}

// Share and slope.  Beyond |z| = 20 (SiLU: 110) both are 0 or 1 to the last bit of a
// float's range; with z held there (t), no product of an overflowed factor and a zero can
// arise.  A NaN is not held: it stays in the share, and by it in the slope.
template <int ACT>
__device__ __forceinline__ void share_and_slope(float2 z, float2& share, float2& slope) {
    constexpr float kEnd = ACT == BSS_ACT_SILU ? 110.0f : 20.0f;
    const float2 t = make_float2(fminf(fmaxf(z.x, -kEnd), kEnd), fminf(fmaxf(z.y, -kEnd), kEnd));
    if constexpr (ACT == BSS_ACT_GELU) {
        float2 e;
        share = erf_share(z, e);
        slope = __ffma2_rn(__fmul2_rn(t, f2(0.39894228040143268f)), e, share);
    } else {
        // share (1 + (1 - share) u') with u' z times the derivative of the exponent
        const float2 w = __fmul2_rn(t, t);
        share = smooth_share<ACT>(z, w);
        float2 q = t;
        if constexpr (ACT == BSS_ACT_GELU_TANH) q = __fmul2_rn(t, __ffma2_rn(w, f2(3.0f * kTanhC * kTanhD), f2(kTanhC)));
        const float2 rest = __ffma2_rn(share, f2(-1.0f), f2(1.0f));
        slope = __fmul2_rn(share, __ffma2_rn(q, rest, f2(1.0f)));
    }
}

// ---------------------------------------------------------------- tile product
// A tile of 128 CG rows and columns is made by CG CTAs (a pair's MMA takes half of
// A and of B from each): warp 0 loads, warp 1 of the first CTA issues the MMAs,
// warps 4 to 11 of each bring the accumulators of its 128 rows from TMEM to memory,
// a warp 32 rows of half of the columns, 128 bytes a row at a time through a piece of
// shared memory of its own and a TMA store, which clips at the tensor's ends.
// Two accumulators a CTA: the MMAs of the next tile run during this one's stores.
// Bound by the tensor cores: one launch alone (37,800 x 5,120 -> 1,280) 1,857 TFLOP/s with the
// tensor pipe 92% active; pairs of CTAs because each then reads half of B from shared
// memory (a pair's block of 64 takes 0.38 us for four times the work of a single's 0.25).
constexpr int kTileK = 64;  // 128 bytes of bf16: one swizzle row
constexpr int kOperand = 128 * kTileK * 2;
constexpr int kStages = 5;
constexpr int kThreads = 384;
constexpr int kEpilogueWarps = 8;
// CTAs of a cluster that share a tile: with 8 not all clusters find room at once (256 x
// 1,280 -> 1,280: 18 us instead of 8).
constexpr int kMostJoined = 4;
constexpr int kPiece = 32 * 128;  // 32 rows of 128 bytes: a warp's two take turns

struct Epilogue {
    const void* bias;
    const void* gate;
    const void* residual;
    void* out;
    void* pre;
    int64_t gate_stride, residual_stride, out_stride, pre_stride;
    int32_t param_dtype, out_dtype, activation;
    float residual_scale;
    FastDiv by_rows;
};

struct GemmArgs {
    CUtensorMap a, b, out, pre, residual;
    int32_t m, n, kblocks;
    int32_t tiles_n, tiles, splits;  // of the contraction: split i takes the planes' sums i
    int* status;
    Epilogue e;
};

// The contraction's blocks of 64 that a split begins with.
__device__ __forceinline__ int split_begin(const GemmArgs& g, int split) {
    return static_cast<int>(static_cast<int64_t>(split) * g.kblocks / g.splits);
}

struct GemmSmem {
    static constexpr uint32_t kPieces = kStages * 2 * kOperand;
    static constexpr uint32_t kBars = kPieces + kEpilogueWarps * 2 * kPiece;
    // full, empty [kStages], accumulators full, empty [2], residual [kEpilogueWarps][2]
    static constexpr uint32_t kBytes = kBars + (2 * kStages + 4 + 2 * kEpilogueWarps) * 8 + 16;
    static constexpr uint32_t kAlloc = kBytes + 1024;  // the operands start on 1024 bytes
};

// 8 values of a row -> bf16 or float memory
__device__ __forceinline__ void store8(void* base, int64_t at, int dtype, const float (&v)[8]) {
    if (dtype == BSS_DTYPE_F32) {
        float4* p = reinterpret_cast<float4*>(static_cast<float*>(base) + at);
        p[0] = make_float4(v[0], v[1], v[2], v[3]);
        p[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
        *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(base) + at) =
            make_uint4(pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7]));
    }
}

// 8 values that another thread of this call may write afterwards: not through the
// read-only path.
__device__ __forceinline__ void load8(const void* base, int64_t at, int dtype, float (&v)[8]) {
    if (dtype == BSS_DTYPE_F32) {
        const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + at);
        const float4 a = p[0], b = p[1];
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
        const uint4 q = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(base) + at);
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
}

// 32 values of a lane's row in a piece: its 16-byte units are swizzled like the TMA's.
__device__ __forceinline__ uint8_t* unit_at(uint8_t* row, int unit) { return row + ((unit ^ (threadIdx.x & 7)) << 4); }

__device__ __forceinline__ void put32(uint8_t* row, int unit, const float2 (&v)[16]) {
#pragma unroll
    for (int k = 0; k < 4; ++k)
        *reinterpret_cast<uint4*>(unit_at(row, unit + k)) =
            make_uint4(pack2(v[4 * k].x, v[4 * k].y), pack2(v[4 * k + 1].x, v[4 * k + 1].y), pack2(v[4 * k + 2].x, v[4 * k + 2].y),
                       pack2(v[4 * k + 3].x, v[4 * k + 3].y));
}

__device__ __forceinline__ void put32_float(uint8_t* row, const float2 (&v)[16]) {
#pragma unroll
    for (int k = 0; k < 8; ++k)
        *reinterpret_cast<float4*>(unit_at(row, k)) = make_float4(v[2 * k].x, v[2 * k].y, v[2 * k + 1].x, v[2 * k + 1].y);
}

__device__ __forceinline__ void get32(uint8_t* row, int unit, float2 (&v)[16]) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const uint4 q = *reinterpret_cast<const uint4*>(unit_at(row, unit + k));
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) v[4 * k + i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
    }
}

__device__ __forceinline__ void get32_float(uint8_t* row, float2 (&v)[16]) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const float4 q = *reinterpret_cast<const float4*>(unit_at(row, k));
        v[2 * k] = make_float2(q.x, q.y), v[2 * k + 1] = make_float2(q.z, q.w);
    }
}

// A row's 32 parameters from a column on (NULL: all the same value).
__device__ __forceinline__ void load_params32(const void* base, int64_t at, int col, int n, int dtype, float none, float2 (&v)[16]) {
    if (base == nullptr) {
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = f2(none);
    } else if (dtype == BSS_DTYPE_F32) {
        const float* p = static_cast<const float*>(base) + at;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float4 q = __ldg(reinterpret_cast<const float4*>(p + min(col + 4 * k, n - 4)));
            v[2 * k] = make_float2(q.x, q.y), v[2 * k + 1] = make_float2(q.z, q.w);
        }
    } else {
        const __nv_bfloat16* p = static_cast<const __nv_bfloat16*>(base) + at;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint4 q = __ldg(reinterpret_cast<const uint4*>(p + min(col + 8 * k, n - 8)));
            const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) v[4 * k + i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
        }
    }
}

// From the product of 8 columns of a row to memory.
template <int ACT>
__device__ __forceinline__ void end_row8(const Epilogue& e, int row, int col, float (&v)[8], float (&w)[8]) {
    if (e.bias != nullptr) {
        load_param8(e.bias, col, e.param_dtype, w);
#pragma unroll
        for (int x = 0; x < 8; ++x) v[x] += w[x];
    }
    if (e.pre != nullptr) store8(e.pre, row * e.pre_stride + col, BSS_DTYPE_BF16, v);
    activate8<ACT>(v);
    if (e.gate != nullptr) {
        load_param8(e.gate, e.by_rows.div(row) * e.gate_stride + col, e.param_dtype, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] *= w[i];
    }
    if (e.residual != nullptr) {
        load8(e.residual, row * e.residual_stride + col, e.out_dtype, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = fmaf(e.residual_scale, w[i], v[i]);
    }
    store8(e.out, row * e.out_stride + col, e.out_dtype, v);
}

// JOIN: a cluster of `splits` CTAs makes one tile, each a share of the contraction; their
// sums meet through shared memory, each CTA taking as many of the rows to the end.
template <int CG, bool A_MN, bool B_MN, int ACT, bool JOIN>
__global__ void __launch_bounds__(kThreads, 1) gemm_kernel(const __grid_constant__ GemmArgs g) {
    using L = GemmSmem;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::kBars);
    uint64_t* empty = full + kStages;
    uint64_t* acc_full = empty + kStages;
    uint64_t* acc_empty = acc_full + 2;
    uint64_t* arrived = acc_empty + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(arrived + 2 * kEpilogueWarps);
    constexpr int kTile = 128 * CG;
    constexpr bool kPlain = A_MN || B_MN;    // a gradient: nothing behind the product
    constexpr uint32_t kAccCols = 128 * CG;  // a CTA's accumulator: its 128 rows, the tile's columns

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = CG == 2 ? cluster_rank() : 0;
    const int share = JOIN ? static_cast<int>(cluster_rank()) : 0;
    const int units = JOIN ? g.tiles : g.tiles * g.splits;
    const int first = JOIN ? blockIdx.x / g.splits : blockIdx.x / CG, step = JOIN ? g.tiles : gridDim.x / CG;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(full + s, 1);
            mbar_init(empty + s, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(acc_full + i, 1);
            mbar_init(acc_empty + i, kEpilogueWarps * CG);
        }
        for (int i = 0; i < 2 * kEpilogueWarps; ++i) mbar_init(arrived + i, 1);
        mbar_fence_init();
    }
    if (warp == 1) {
        if constexpr (CG == 2) tmem_alloc_pair(tmem_slot, 2 * kAccCols);
        else tmem_alloc(tmem_slot, 2 * kAccCols);
    }
    tc_fence_before();
    if constexpr (CG == 2) cluster_sync();
    else __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    cudaGridDependencySynchronize();

    if (warp == 0) {
        if (lane == 0) {
            tma_prefetch_desc(&g.a);
            tma_prefetch_desc(&g.b);
            auto load = [&](uint8_t* to, const CUtensorMap* map, int c0, int c1, uint64_t* bar) {
                if constexpr (CG == 2) tma_load_3d_pair(to, map, c0, c1, 0, map_to_rank(bar, 0));
                else tma_load_3d(to, map, c0, c1, 0, bar);
            };
            uint32_t fill = 0;
            bool ok = true;
            for (int u = first; ok && u < units; u += step) {
                const int split = JOIN ? share : u / g.tiles, t = JOIN ? u : u - split * g.tiles;
                const int mt = t / g.tiles_n, nt = t - mt * g.tiles_n;
                const int end = split_begin(g, split + 1);
                const int row_a = mt * kTile + static_cast<int>(rank) * 128, row_b = nt * kTile + static_cast<int>(rank) * 128;
                for (int kb = split_begin(g, split); kb < end; ++kb, ++fill) {
                    const uint32_t s = fill % kStages;
                    if (fill >= kStages) ok = mbar_wait(empty + s, (fill / kStages - 1) & 1, g.status);
                    if (!ok) break;
                    uint8_t* sa = smem + s * 2 * kOperand;
                    uint8_t* sb = sa + kOperand;
                    if (rank == 0) mbar_arrive_expect_tx(full + s, 2 * kOperand * CG);
                    if constexpr (A_MN) {
#pragma unroll
                        for (int c = 0; c < 2; ++c) load(sa + c * kOperand / 2, &g.a, row_a + c * 64, kb * kTileK, full + s);
                    } else {
                        load(sa, &g.a, kb * kTileK, row_a, full + s);
                    }
                    if constexpr (B_MN) {
#pragma unroll
                        for (int c = 0; c < 2; ++c) load(sb + c * kOperand / 2, &g.b, row_b + c * 64, kb * kTileK, full + s);
                    } else {
                        load(sb, &g.b, kb * kTileK, row_b, full + s);
                    }
                }
            }
            // no copy may still be landing when the CTAs end
            if (rank == 0)
                for (uint32_t f = fill > kStages ? fill - kStages : 0; f < fill; ++f)
                    mbar_wait(full + f % kStages, (f / kStages) & 1, g.status);
        }
    } else if (warp == 1) {
        if (rank == 0) {
            constexpr uint32_t idesc = idesc_bf16_f32(kTile, kTile, B_MN, A_MN);
            const bool leader = elect_one();
            const uint32_t base = smem_u32(smem);
            const uint64_t da0 = A_MN ? desc_mnmajor_sw128(base, 0, kOperand / 2) : desc_kmajor_sw128(base, 0);
            const uint64_t db0 = B_MN ? desc_mnmajor_sw128(base + kOperand, 0, kOperand / 2)
                                      : desc_kmajor_sw128(base + kOperand, 0);
            constexpr uint64_t kStepA = A_MN ? 128 : 2, kStepB = B_MN ? 128 : 2;  // 16 of k, in 16-byte units
            uint32_t fill = 0, n_tile = 0;
            bool ok = true;
            auto commit = [&](uint64_t* bar) {
                if (leader) {
                    if constexpr (CG == 2) tc_commit_pair(bar);
                    else tc_commit(bar);
                }
            };
            for (int u = first; ok && u < units; u += step, ++n_tile) {
                const int split = JOIN ? share : u / g.tiles, begin = split_begin(g, split), end = split_begin(g, split + 1);
                const uint32_t buf = n_tile & 1;
                if (n_tile >= 2)
                    ok = __all_sync(0xFFFFFFFFu, mbar_wait(acc_empty + buf, (n_tile / 2 - 1) & 1, g.status));
                if (!ok) break;
                tc_fence_after();
                for (int kb = begin; kb < end; ++kb, ++fill) {
                    const uint32_t s = fill % kStages;
                    ok = __all_sync(0xFFFFFFFFu, mbar_wait(full + s, (fill / kStages) & 1, g.status));
                    if (!ok) break;
                    tc_fence_after();
                    if (leader) {
                        const uint64_t at = static_cast<uint64_t>(s) * (2 * kOperand >> 4);
#pragma unroll
                        for (int kk = 0; kk < kTileK / 16; ++kk) {
                            const uint32_t acc = kb > begin || kk > 0 ? 1u : 0u;
                            if constexpr (CG == 2)
                                umma_ss_pair(tmem + buf * kAccCols, da0 + at + kk * kStepA, db0 + at + kk * kStepB, idesc, acc);
                            else
                                umma_ss(tmem + buf * kAccCols, da0 + at + kk * kStepA, db0 + at + kk * kStepB, idesc, acc);
                        }
                    }
                    commit(empty + s);
                }
                if (ok) commit(acc_full + buf);
            }
        }
    } else if (warp >= 4) {
        const int quarter = warp & 3, side = (warp - 4) >> 2;
        const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
        uint8_t* pieces = smem + L::kPieces + (warp - 4) * 2 * kPiece;
        const Epilogue& e = g.e;
        const bool wide = e.out_dtype == BSS_DTYPE_F32, staged_pre = e.pre != nullptr && !wide, adds = e.residual != nullptr;
        const int width = wide ? 32 : 64, begin_c = side * (kTile / 2), end_c = begin_c + kTile / 2;
        if constexpr (JOIN) {
            // the sums of 32 rows and half of the columns, where the operands were: a row of
            // 512 bytes, its 16-byte units swizzled by the row
            if (__all_sync(0xFFFFFFFFu, mbar_wait(acc_full, 0, g.status))) {
                tc_fence_after();
                uint8_t* to = smem + (quarter * 32 + lane) * 512;
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    uint32_t x[32];
                    BSS_TMEM_LD32(tmem + lanes + side * 64 + 32 * c, x);
                    tmem_wait_ld();
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        *reinterpret_cast<uint4*>(to + ((side * 16 + c * 8 + (k ^ (lane & 7))) << 4)) =
                            make_uint4(x[4 * k], x[4 * k + 1], x[4 * k + 2], x[4 * k + 3]);
                }
            }
        } else {
        // Where a piece's columns lie; false past the tensor's ends.
        auto place = [&](int u, int c, int& col, int& row0) {
            const int t = u % g.tiles, mt = t / g.tiles_n;
            col = (t - mt * g.tiles_n) * kTile + c;
            row0 = mt * kTile + static_cast<int>(rank) * 128 + quarter * 32;
            return col < g.n && row0 < g.m;
        };
        uint32_t n_tile = 0, chunk = 0, taken[2] = {0, 0}, asked[2] = {0, 0};
        // out's pieces take turns; with pre it has the first one and out the second.  The
        // store that read a piece last must have done so before it is written again.
        auto piece_of = [&](uint32_t i) { return staged_pre ? 1u : i & 1; };
        auto free_piece = [&]() {
            if (lane == 0) {
                if (staged_pre) tma_store_wait_read<0>();
                else tma_store_wait_read<1>();
            }
            __syncwarp();
        };
        auto send = [&](const CUtensorMap* map, const uint8_t* from, int col, int row0, int plane) {
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                tma_store_3d(map, from, col, row0, plane);
                tma_store_commit();
            }
        };
        // The residual comes into the piece that its sum leaves from, a piece ahead.
        auto ask = [&](int u, int c) {
            int col, row0;
            while (u < units && (c >= end_c || !place(u, c, col, row0))) u += step, c = begin_c;
            if (u >= units) return;
            const uint32_t p = piece_of(chunk);
            if (lane == 0) {
                mbar_arrive_expect_tx(arrived + (warp - 4) * 2 + p, kPiece);
                tma_load_3d(pieces + p * kPiece, &g.residual, col, row0, 0, arrived + (warp - 4) * 2 + p);
            }
            if (p == 0) ++asked[0];
            else ++asked[1];
        };
        if (adds) ask(first, begin_c);
        bool ok = true;
        for (int u = first; ok && u < units; u += step, ++n_tile) {
            const uint32_t buf = n_tile & 1;
            int col0, row0;
            place(u, begin_c, col0, row0);
            const int split = u / g.tiles, row = row0 + lane;
            const int64_t group = e.gate != nullptr && row < g.m ? e.by_rows.div(row) : 0;
            if (!(ok = __all_sync(0xFFFFFFFFu, mbar_wait(acc_full + buf, (n_tile / 2) & 1, g.status)))) break;
            tc_fence_after();
#pragma unroll 1
            for (int c = begin_c; c < end_c; c += width) {
                if (!place(u, c, col0, row0)) break;
                const uint32_t p = piece_of(chunk);
                uint8_t* to = pieces + p * kPiece + lane * 128;
                if (adds) {
                    const uint32_t n = p == 0 ? taken[0]++ : taken[1]++;
                    if (!(ok = __all_sync(0xFFFFFFFFu, mbar_wait(arrived + (warp - 4) * 2 + p, n & 1, g.status)))) break;
                } else {
                    free_piece();
                }
                ++chunk;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if (h == 1 && wide) break;
                    const int col = col0 + 32 * h;
                    // Everything is loaded before anything is computed, without a branch in
                    // between (with one for every 8 columns a tile's epilogue took 20,000
                    // cycles).  Columns past the end take the last ones' parameters; the
                    // stores clip them.
                    float2 bias[16], gate[16];
                    if constexpr (!kPlain) {
                        load_params32(e.bias, 0, col, g.n, e.param_dtype, 0.0f, bias);
                        load_params32(e.gate, group * e.gate_stride, col, g.n, e.param_dtype, 1.0f, gate);
                    }
                    uint32_t x[32];
                    BSS_TMEM_LD32(tmem + lanes + buf * kAccCols + c + 32 * h, x);
                    tmem_wait_ld();
                    float2 v[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        v[i] = make_float2(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1]));
                        if constexpr (!kPlain) v[i] = __fadd2_rn(v[i], bias[i]);
                    }
                    if constexpr (!kPlain) {
                        if (e.pre != nullptr) {
                            if (staged_pre) {
                                put32(pieces + lane * 128, 4 * h, v);
                            } else if (row < g.m) {
#pragma unroll
                                for (int k = 0; k < 4; ++k)
                                    if (col + 8 * k < g.n)
                                        *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(e.pre) + row * e.pre_stride + col + 8 * k) =
                                            make_uint4(pack2(v[4 * k].x, v[4 * k].y), pack2(v[4 * k + 1].x, v[4 * k + 1].y),
                                                       pack2(v[4 * k + 2].x, v[4 * k + 2].y), pack2(v[4 * k + 3].x, v[4 * k + 3].y));
                            }
                        }
#pragma unroll
                        for (int i = 0; i < 16; ++i) v[i] = __fmul2_rn(activate<ACT>(v[i]), gate[i]);
                        if (adds) {
                            float2 r[16];
                            if (wide) get32_float(to, r);
                            else get32(to, 4 * h, r);
#pragma unroll
                            for (int i = 0; i < 16; ++i) v[i] = __ffma2_rn(r[i], f2(e.residual_scale), v[i]);
                        }
                    }
                    if (wide) put32_float(to, v);
                    else put32(to, 4 * h, v);
                }
                send(&g.out, to - lane * 128, col0, row0, split);
                if (staged_pre) send(&g.pre, pieces, col0, row0, 0);
                if (adds) {
                    free_piece();
                    ask(u, c + width);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if constexpr (CG == 2) mbar_arrive_cluster(map_to_rank(acc_empty + buf, 0));
                else mbar_arrive(acc_empty + buf);
            }
        }
        if (lane == 0) {
            // no copy may still be landing, the pieces are read before the CTA ends
            for (int p = 0; p < 2; ++p)
                if (asked[p] > taken[p]) mbar_wait(arrived + (warp - 4) * 2 + p, (asked[p] - 1) & 1, g.status);
            tma_store_wait_read_all();
        }
        }
    }

    tc_fence_before();
    __syncwarp();
    if constexpr (JOIN) {
        cluster_sync();
        if (warp >= 4) {
            // 16 threads a row, 8 columns each; all shares' loads at once, added in their order
            const int t = first, mt = t / g.tiles_n, end = 128 * (share + 1) / g.splits;
            const int unit = (threadIdx.x & 15) * 2, col = (t - mt * g.tiles_n) * kTile + unit * 4;
            for (int r = 128 * share / g.splits + (static_cast<int>(threadIdx.x) - 128) / 16; r < end; r += 16) {
                const int row = mt * kTile + r;
                if (row >= g.m || col >= g.n) continue;
                const uint32_t at = static_cast<uint32_t>(r) * 512 + ((unit & ~7) << 4);
                const uint32_t first_unit = at + (((unit & 7) ^ (r & 7)) << 4), second_unit = at + ((((unit & 7) + 1) ^ (r & 7)) << 4);
                float4 x[kMostJoined], y[kMostJoined];
#pragma unroll
                for (int s = 0; s < kMostJoined; ++s) {
                    if (s < g.splits) {
                        const uint32_t from = map_to_rank(smem, s);
                        x[s] = lds_cluster(from + first_unit);
                        y[s] = lds_cluster(from + second_unit);
                    }
                }
                float v[8] = {x[0].x, x[0].y, x[0].z, x[0].w, y[0].x, y[0].y, y[0].z, y[0].w}, w[8];
#pragma unroll
                for (int s = 1; s < kMostJoined; ++s) {
                    if (s < g.splits) {
                        v[0] += x[s].x, v[1] += x[s].y, v[2] += x[s].z, v[3] += x[s].w;
                        v[4] += y[s].x, v[5] += y[s].y, v[6] += y[s].z, v[7] += y[s].w;
                    }
                }
                end_row8<ACT>(g.e, row, col, v, w);
            }
        }
        __syncwarp();
        cluster_sync();  // the others have read
    } else if constexpr (CG == 2) {
        cluster_sync();
    } else {
        __syncthreads();
    }
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        if constexpr (CG == 2) tmem_dealloc_pair(tmem, 2 * kAccCols);
        else tmem_dealloc(tmem, 2 * kAccCols);
    }
}

// Sums of the splits, then the epilogue: 8 columns a thread.
struct FinishArgs {
    const float* sums;  // [splits][m][n]
    int32_t m, n, splits;
    FastDiv by_vectors;
    Epilogue e;
};

template <int ACT>
__global__ void __launch_bounds__(256) finish_kernel(const __grid_constant__ FinishArgs a) {
    cudaGridDependencySynchronize();
    const int64_t plane = static_cast<int64_t>(a.m) * a.n;
    const uint32_t vectors = a.n / 8, all = a.m * vectors;  // below 2^31: the splits are of small results
    for (uint32_t i = blockIdx.x * 256 + threadIdx.x; i < all; i += gridDim.x * 256) {
        const int row = a.by_vectors.div(i), col = static_cast<int>(i - row * vectors) * 8;
        float v[8], w[8];
        load8(a.sums, row * static_cast<int64_t>(a.n) + col, BSS_DTYPE_F32, v);
#pragma unroll 8
        for (int s = 1; s < a.splits; ++s) {
            load8(a.sums, s * plane + row * static_cast<int64_t>(a.n) + col, BSS_DTYPE_F32, w);
#pragma unroll
            for (int x = 0; x < 8; ++x) v[x] += w[x];
        }
        end_row8<ACT>(a.e, row, col, v, w);
    }
}

// ---------------------------------------------------------------- few rows
// The weights' bytes are the work: every warp streams its share of them straight into
// the operand of a small matrix product (16 output channels a block; lane 4 g + c loads
// 16 bytes of rows g and g + 8: channels that follow one another, the same ones of x's
// rows), 8 warps share the contraction, and their sums meet in shared memory.  1,280 ->
// 7,680: one row 4.7 us with the 19.7 MB of weights in L2 (9.0 from memory), 16 rows 6.8; by
// tiles 17 rows 9.5.
constexpr int kFewRows = 16;
constexpr int kFewWarps = 8;

struct FewArgs {
    const __nv_bfloat16 *x, *weight;
    int64_t x_stride, weight_stride;
    int32_t rows, inner, outer;
    Epilogue e;
};

__device__ __forceinline__ void few_product(float (&d)[4], const uint4& w0, const uint4& w1, const uint4& x) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(w0.x), "r"(w1.x), "r"(w0.y), "r"(w1.y), "r"(x.x), "r"(x.y));
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(w0.z), "r"(w1.z), "r"(w0.w), "r"(w1.w), "r"(x.z), "r"(x.w));
}

template <int NT, int ACT>  // NT: tiles of 8 rows
__global__ void __launch_bounds__(32 * kFewWarps) few_rows_kernel(const __grid_constant__ FewArgs a) {
    __shared__ float sums[kFewWarps][8 * NT][17];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = (lane & 3) * 8;
    const int o0 = blockIdx.x * 16;
    const uint4 none = make_uint4(0, 0, 0, 0);
    // (output channels come in eights: the second eight may not exist)
    const __nv_bfloat16* w0 = a.weight + (o0 + g) * a.weight_stride + c;
    const __nv_bfloat16* w1 = w0 + 8 * a.weight_stride;
    const bool both = o0 + 8 < a.outer;
    cudaGridDependencySynchronize();
    float d[NT][4] = {};
    constexpr int kBatch = NT == 1 ? 8 : 4;  // blocks of 32 channels in flight
    const int blocks = (a.inner + 31) / 32, begin = blocks * warp / kFewWarps, end = blocks * (warp + 1) / kFewWarps;
    for (int b = begin; b < end; b += kBatch) {
        uint4 p[kBatch], q[kBatch], x[kBatch][NT];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int k = (b + i) * 32;
            const bool live = b + i < end && k + c < a.inner;
            p[i] = live ? ld_row(w0 + k) : none;
            q[i] = live && both ? ld_row(w1 + k) : none;
#pragma unroll
            for (int t = 0; t < NT; ++t)
                x[i][t] = live && 8 * t + g < a.rows
                              ? __ldg(reinterpret_cast<const uint4*>(a.x + (8 * t + g) * a.x_stride + k + c)) : none;
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
#pragma unroll
            for (int t = 0; t < NT; ++t) few_product(d[t], p[i], q[i], x[i][t]);
    }
    // d: channels g and g + 8 of rows 2 (lane % 4) and the next
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const int r = 8 * t + (lane & 3) * 2;
        sums[warp][r][g] = d[t][0];
        sums[warp][r + 1][g] = d[t][1];
        sums[warp][r][g + 8] = d[t][2];
        sums[warp][r + 1][g + 8] = d[t][3];
    }
    __syncthreads();
    const Epilogue& e = a.e;
    for (int i = threadIdx.x; i < 8 * NT * 16; i += 32 * kFewWarps) {
        const int row = i >> 4, o = o0 + (i & 15);
        if (row >= a.rows || o >= a.outer) continue;
        float z = 0.0f;
#pragma unroll
        for (int w = 0; w < kFewWarps; ++w) z += sums[w][row][i & 15];
        if (e.bias != nullptr) z += load_param(e.bias, o, e.param_dtype);
        if (e.pre != nullptr) static_cast<__nv_bfloat16*>(e.pre)[row * e.pre_stride + o] = __float2bfloat16(z);
        float v = activate<ACT>(z);
        if (e.gate != nullptr) v *= load_param(e.gate, e.by_rows.div(row) * e.gate_stride + o, e.param_dtype);
        if (e.out_dtype == BSS_DTYPE_F32) {
            if (e.residual != nullptr) v = fmaf(e.residual_scale, static_cast<const float*>(e.residual)[row * e.residual_stride + o], v);
            static_cast<float*>(e.out)[row * e.out_stride + o] = v;
        } else {
            if (e.residual != nullptr)
                v = fmaf(e.residual_scale, __bfloat162float(static_cast<const __nv_bfloat16*>(e.residual)[row * e.residual_stride + o]), v);
            static_cast<__nv_bfloat16*>(e.out)[row * e.out_stride + o] = __float2bfloat16(v);
        }
    }
}

// ---------------------------------------------------------------- dz and its sums over rows
// A thread has 8 channels, a warp walks over rows; a block covers `units` rows that
// share a gate, or (small groups) whole groups, one a warp at a time.  dz is rounded to
// bf16, the type of the other operand of both products that read it (the tensor cores take
// both in one); dbias and dgate are summed from the 32-bit values.  Bound by DRAM:
// 37,800 x 5,120 with GELU's slope and the bias sums 184 us, 6,310 GB/s (95% of a copy).
struct DzArgs {
    const void* dout;
    const __nv_bfloat16* pre;
    const void* gate;
    __nv_bfloat16* dz;  // NULL: only the sums are wanted
    float *dbias, *dgate;  // partial sums, or (small groups) dgate itself
    int64_t rows, group_rows, dout_stride, pre_stride, gate_stride;
    int64_t units;      // rows of a block's chunk; of small groups: groups of a block
    int32_t chunks;     // blocks a group; 0: small groups
    int32_t n, dout_dtype, param_dtype;
};

constexpr int kDzWarps = 8;

template <int ACT, bool WIDE, bool GATED>  // WIDE: dout is float
__global__ void __launch_bounds__(32 * kDzWarps) dz_kernel(const __grid_constant__ DzArgs a) {
    __shared__ float sums[kDzWarps][2][32 * 9];  // a lane's 8 values 9 apart
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int c = (blockIdx.x * 32 + lane) * 8;
    const bool live = c < a.n;
    const bool small = a.chunks == 0;
    int64_t group, begin, end;
    if (small) {
        group = blockIdx.y * a.units + warp;
        begin = end = 0;
    } else {
        group = blockIdx.y / a.chunks;
        begin = group * a.group_rows + (blockIdx.y - group * a.chunks) * a.units;
        end = begin + a.units;
        const int64_t group_end = (group + 1) * a.group_rows;
        if (end > group_end) end = group_end;
        if (end > a.rows) end = a.rows;
    }
    const int64_t last_group = (blockIdx.y + 1) * a.units;  // small groups
    cudaGridDependencySynchronize();
    float db[8] = {}, dg[8] = {}, gate[8];
    while (true) {
        if (small) {
            begin = group * a.group_rows;
            end = begin + a.group_rows;
            if (end > a.rows) end = a.rows;
            if (group >= last_group || begin >= a.rows) break;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) gate[i] = 1.0f;
        if (a.gate != nullptr && live) load_param8(a.gate, group * a.gate_stride + c, a.param_dtype, gate);
        // several rows' loads at once: two of 16 bytes alone leave the memory idle
        constexpr int kRows = WIDE ? 2 : 4;
        const int64_t every = small ? 1 : kDzWarps;
        for (int64_t row = begin + (small ? 0 : warp); live && row < end; row += kRows * every) {
            float d[kRows][8], z[kRows][8];
#pragma unroll
            for (int k = 0; k < kRows; ++k) {
                const int64_t at = row + k * every < end ? row + k * every : row;
                load8(a.dout, at * a.dout_stride + c, WIDE ? BSS_DTYPE_F32 : BSS_DTYPE_BF16, d[k]);
                if (a.pre != nullptr) load8(a.pre, at * a.pre_stride + c, BSS_DTYPE_BF16, z[k]);
                else z[k][0] = z[k][1] = z[k][2] = z[k][3] = z[k][4] = z[k][5] = z[k][6] = z[k][7] = 0.0f;
            }
#pragma unroll
            for (int k = 0; k < kRows; ++k) {
                if (row + k * every >= end) break;
#pragma unroll
                for (int i = 0; i < 8; i += 2) {
                    float2 x = make_float2(d[k][i], d[k][i + 1]), share = f2(1.0f), slope = f2(1.0f);
                    const float2 at = make_float2(z[k][i], z[k][i + 1]);
                    if constexpr (ACT != BSS_ACT_NONE) share_and_slope<ACT>(at, share, slope);
                    if constexpr (GATED) {
                        const float2 v = __fmul2_rn(at, share);
                        const float2 s = __ffma2_rn(x, v, make_float2(dg[i], dg[i + 1]));
                        dg[i] = s.x, dg[i + 1] = s.y;
                        x = __fmul2_rn(x, make_float2(gate[i], gate[i + 1]));
                    }
                    if constexpr (ACT != BSS_ACT_NONE) x = __fmul2_rn(x, slope);
                    db[i] += x.x, db[i + 1] += x.y;
                    d[k][i] = x.x, d[k][i + 1] = x.y;
                }
                if (a.dz != nullptr) store8(a.dz, (row + k * every) * a.n + c, BSS_DTYPE_BF16, d[k]);
            }
        }
        if (!small) break;
        if (a.dgate != nullptr && live) store8(a.dgate, group * a.n + c, BSS_DTYPE_F32, dg);
#pragma unroll
        for (int i = 0; i < 8; ++i) dg[i] = 0.0f;
        group += kDzWarps;
    }
    const bool want_gate = a.dgate != nullptr && !small;
    if (a.dbias == nullptr && !want_gate) return;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        sums[warp][0][lane * 9 + i] = db[i];
        sums[warp][1][lane * 9 + i] = dg[i];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 256; i += 32 * kDzWarps) {
        const int col = blockIdx.x * 256 + i, at = (i >> 3) * 9 + (i & 7);
        if (col >= a.n) continue;
        float b = 0.0f, g = 0.0f;
#pragma unroll
        for (int w = 0; w < kDzWarps; ++w) {
            b += sums[w][0][at];
            g += sums[w][1][at];
        }
        if (a.dbias != nullptr) a.dbias[static_cast<int64_t>(blockIdx.y) * a.n + col] = b;
        if (want_gate) a.dgate[static_cast<int64_t>(blockIdx.y) * a.n + col] = g;
    }
}

// Sums of parts in a fixed order, a block's eight warps taking every eighth part each:
// row 0 of the grid has dbias, of all blocks' parts, the others a group's dgate each.
struct SumArgs {
    const float *bias_parts, *gate_parts;  // NULL: not wanted
    float *dbias, *dgate;
    int64_t blocks;
    int32_t chunks, n;
};

__global__ void __launch_bounds__(256) sum_parts_kernel(const __grid_constant__ SumArgs a) {
    __shared__ float sums[8][32];
    cudaGridDependencySynchronize();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int c = blockIdx.x * 32 + lane;
    const bool bias = blockIdx.y == 0 && a.bias_parts != nullptr;
    const int64_t group = a.bias_parts != nullptr ? blockIdx.y - 1ll : blockIdx.y, parts = bias ? a.blocks : a.chunks;
    const float* from = bias ? a.bias_parts : a.gate_parts + group * a.chunks * a.n;
    float s = 0.0f;
    if (c < a.n)
#pragma unroll 8
        for (int64_t i = warp; i < parts; i += 8) s += from[i * a.n + c];
    sums[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && c < a.n) {
#pragma unroll
        for (int w = 1; w < 8; ++w) s += sums[w][lane];
        (bias ? a.dbias : a.dgate + group * a.n)[c] = s;
    }
}

// ---------------------------------------------------------------- host side
// Operand [rows][width] whose k (K-major) or m / n (MN-major) is its width.
bss_status operand_map(CUtensorMap* map, const void* p, int64_t rows, int64_t stride, int64_t width, bool mn_major) {
    const uint64_t bytes = static_cast<uint64_t>(rows > 1 ? stride : (width + 7) / 8 * 8) * 2;
    return encode_tmap_3d(map, p, width, rows, 1, bytes, bytes, 64, mn_major ? kTileK : 128);
}

// How a product is cut: by pairs of CTAs or single ones, and its contraction into splits,
// whose sums a second kernel adds.  The least of a simple estimate in microseconds:
// rounds of the tiles times a block of 64 of the contraction (pairs 0.38, single 0.25,
// measured at 75,600 x 5,120 x 1,280), plus 4 for the second kernel and its bytes at
// 5 TB/s.  (1,280 x 5,120 of 75,600: 752 us with one split, 100 tiles for 76 pairs.)  Up to 64
// splits: the gradients of 75,600 x 64 -> 64 without a bias 38 -> 29 us against at most 16.
// Where the tiles leave CTAs over, a cluster of them shares a tile and nothing goes
// through memory (512 x 4,096 -> 1,280: 11.7 us, with a second kernel 11.2, but calls
// one after another 12.8 instead of 20.4: no workspace, one launch).
struct Cut {
    bool pair;
    int splits;
    bool join;  // the splits are a cluster's
};

Cut cut_of(int64_t m, int64_t n, int64_t k) {
    const int64_t blocks = (k + kTileK - 1) / kTileK;
    Cut best = {false, 1, false};
    double least = 1e30;
    for (int pair = 1; pair >= 0; --pair) {
        const int64_t tile = pair ? 256 : 128, units = num_sms() / (pair ? 2 : 1);
        const int64_t tiles = ((m + tile - 1) / tile) * ((n + tile - 1) / tile);
        for (int s = 1; s <= 64 && (s == 1 || s * 4 <= blocks); ++s) {
            if (s > 1 && m * n > (int64_t(1) << 28)) break;
            const double rounds = static_cast<double>((tiles * s + units - 1) / units);
            double t = rounds * static_cast<double>((blocks + s - 1) / s) * (pair ? 0.38 : 0.25);
            if (s > 1) t += 4.0 + 8.0 * s * m * n / 5e6;
            if (t < least) least = t, best = {pair != 0, s, false};
        }
        for (int s = 2; !pair && s <= kMostJoined && tiles * s <= units && s * 2 <= blocks; ++s) {
            const double t = static_cast<double>((blocks + s - 1) / s) * 0.25 + 1.5;
            if (t < least) least = t, best = {false, s, true};
        }
    }
    return best;
}

int64_t cut_bytes(const Cut& c, int64_t m, int64_t n) { return c.splits > 1 && !c.join ? 4 * c.splits * m * n : 0; }

template <int CG, bool A_MN, bool B_MN, int ACT, bool JOIN = false>
bss_status launch_gemm(GemmArgs& g, cudaStream_t stream) {
    constexpr int kTile = 128 * CG;
    const int64_t tiles_m = (static_cast<int64_t>(g.m) + kTile - 1) / kTile;
    g.tiles_n = (g.n + kTile - 1) / kTile;
    if (tiles_m * g.tiles_n * g.splits > 0x7FFFFFFF - 4096) return set_error(BSS_ERR_UNSUPPORTED, "too many tiles");
    g.tiles = static_cast<int32_t>(tiles_m * g.tiles_n);
    auto kernel = gemm_kernel<CG, A_MN, B_MN, ACT, JOIN>;
    int blocks;
    const bss_status st = resident_blocks(reinterpret_cast<const void*>(kernel), kThreads, GemmSmem::kAlloc, &blocks);
    if (st != BSS_OK) return st;
    int units = num_sms() / CG;
    if (JOIN || units > g.tiles * g.splits) units = g.tiles * g.splits;
    return launch_behind_with(kernel, dim3(static_cast<unsigned>(units * CG)), kThreads, GemmSmem::kAlloc, JOIN ? g.splits : CG,
                              stream, "matrix product launch", g);
}

template <bool A_MN, bool B_MN, int ACT>
bss_status launch_cut(GemmArgs& g, const Cut& cut, cudaStream_t stream) {
    if (cut.join) return launch_gemm<1, A_MN, B_MN, ACT, true>(g, stream);
    return cut.pair ? launch_gemm<2, A_MN, B_MN, ACT>(g, stream) : launch_gemm<1, A_MN, B_MN, ACT>(g, stream);
}

// The kernel of an activation.
template <typename F>
bss_status by_activation(int activation, F&& f) {
    switch (activation) {
        case BSS_ACT_GELU_TANH: return f(std::integral_constant<int, BSS_ACT_GELU_TANH>());
        case BSS_ACT_GELU: return f(std::integral_constant<int, BSS_ACT_GELU>());
        case BSS_ACT_SILU: return f(std::integral_constant<int, BSS_ACT_SILU>());
        default: return f(std::integral_constant<int, BSS_ACT_NONE>());
    }
}

// D[m][n] = A B^T of k, then the epilogue; with splits through `sums`.
template <bool A_MN, bool B_MN>
bss_status gemm(const void* a, int64_t a_stride, const void* b, int64_t b_stride, int64_t m, int64_t n, int64_t k,
                const Cut& cut, float* sums, const Epilogue& e, cudaStream_t stream) {
    GemmArgs g;
    memset(&g, 0, sizeof(g));
    g.status = device_status_ptr();
    if (g.status == nullptr) return set_error(BSS_ERR_CUDA, "cannot resolve the device status word");
    bss_status st = A_MN ? operand_map(&g.a, a, k, a_stride, m, true) : operand_map(&g.a, a, m, a_stride, k, false);
    if (st != BSS_OK) return st;
    st = B_MN ? operand_map(&g.b, b, k, b_stride, n, true) : operand_map(&g.b, b, n, b_stride, k, false);
    if (st != BSS_OK) return st;
    g.m = static_cast<int32_t>(m);
    g.n = static_cast<int32_t>(n);
    g.kblocks = static_cast<int32_t>((k + kTileK - 1) / kTileK);
    g.splits = cut.splits;
    const bool through_memory = cut.splits > 1 && !cut.join;
    if (cut.join) {
        g.e = e;
    } else if (through_memory) {
        g.e.out_dtype = BSS_DTYPE_F32;
        st = encode_tmap_rows(&g.out, sums, BSS_DTYPE_F32, n, m, n * 4, 32, cut.splits, m * n * 4);
    } else {
        g.e = e;
        st = encode_tmap_rows(&g.out, e.out, e.out_dtype, n, m, e.out_stride * element_size(e.out_dtype), 32);
        if (st == BSS_OK && e.residual != nullptr)
            st = encode_tmap_rows(&g.residual, e.residual, e.out_dtype, n, m, e.residual_stride * element_size(e.out_dtype), 32);
        if (st == BSS_OK && e.pre != nullptr && e.out_dtype == BSS_DTYPE_BF16) st = encode_tmap_rows(&g.pre, e.pre, BSS_DTYPE_BF16, n, m, e.pre_stride * 2, 32);
    }
    if (st != BSS_OK) return st;
    if constexpr (A_MN || B_MN)
        st = launch_cut<A_MN, B_MN, BSS_ACT_NONE>(g, cut, stream);
    else
        st = by_activation(g.e.activation, [&](auto act) { return launch_cut<false, false, decltype(act)::value>(g, cut, stream); });
    if (st != BSS_OK || !through_memory) return st;
    FinishArgs f;
    f.sums = sums, f.m = g.m, f.n = g.n, f.splits = cut.splits, f.by_vectors = FastDiv(static_cast<uint32_t>(n / 8)), f.e = e;
    int64_t blocks = (m * (n / 8) + 255) / 256;
    if (blocks > 8ll * num_sms()) blocks = 8ll * num_sms();
    return by_activation(e.activation, [&](auto act) {
        return launch_behind(finish_kernel<decltype(act)::value>, dim3(static_cast<unsigned>(blocks)), 256, stream, "split sums launch", f);
    });
}

template <int ACT>
bss_status launch_few(const FewArgs& f, cudaStream_t stream) {
    const unsigned blocks = static_cast<unsigned>((f.outer + 15) / 16);
    return launch_behind(f.rows <= 8 ? few_rows_kernel<1, ACT> : few_rows_kernel<2, ACT>, dim3(blocks), 32 * kFewWarps, stream,
                         "few rows launch", f);
}

bss_status check_sizes(int64_t rows, int64_t* rows_per_group, int32_t in, int32_t out, int32_t activation) {
    if (rows <= 0 || *rows_per_group <= 0) return set_error(BSS_ERR_INVALID_ARG, "rows and rows_per_group must be positive");
    if (rows > 0x7FFFFFFF) return set_error(BSS_ERR_UNSUPPORTED, "rows must be below 2^31");
    if (in <= 0 || out <= 0 || in % 8 != 0 || out % 8 != 0)
        return set_error(BSS_ERR_INVALID_ARG, "channels must be positive multiples of 8 (got %d, %d)", in, out);
    if (in > kMaxWidth || out > kMaxWidth) return set_error(BSS_ERR_UNSUPPORTED, "more than %d channels", kMaxWidth);
    if (activation < BSS_ACT_NONE || activation > BSS_ACT_SILU) return set_error(BSS_ERR_INVALID_ARG, "unknown activation %d", activation);
    if (*rows_per_group > rows) *rows_per_group = rows;
    return BSS_OK;
}

bss_status check_linear(bss_linear_args& a) {
    bss_status st = check_sizes(a.rows, &a.rows_per_group, a.in_channels, a.out_channels, a.activation);
    if (st != BSS_OK) return st;
    if (!known_dtype(a.out_dtype) || !known_dtype(a.param_dtype)) return set_error(BSS_ERR_INVALID_ARG, "unknown dtype");
    if (a.x == nullptr || a.weight == nullptr || a.out == nullptr) return set_error(BSS_ERR_INVALID_ARG, "x, weight or out is NULL");
    if (!std::isfinite(a.residual_scale)) return set_error(BSS_ERR_INVALID_ARG, "residual_scale must be finite");
    if (a.residual == nullptr && a.residual_scale != 1.0f)
        return set_error(BSS_ERR_INVALID_ARG, "residual_scale is given without a residual");
    return BSS_OK;
}

bool takes_few(const bss_linear_args& a) { return a.rows <= kFewRows; }

int64_t linear_need(const bss_linear_args& a) {
    return takes_few(a) ? 0 : cut_bytes(cut_of(a.rows, a.out_channels, a.in_channels), a.rows, a.out_channels);
}

int64_t groups_of(int64_t rows, int64_t per) { return (rows + per - 1) / per; }

// How the rows are dealt to blocks for dz and its sums, and the workspace.
struct GradPlan {
    bool makes_dz, sums;
    int64_t groups, units, blocks;
    int32_t chunks;
    int64_t dz_at, dbias_at, dgate_at, sums_at, bytes;
    Cut dx, dweight;  // both products' split sums take turns in one place
};

int64_t aligned_up(int64_t v) { return (v + 255) / 256 * 256; }

GradPlan plan_of(const bss_linear_grads& a) {
    GradPlan p = {};
    const int64_t n = a.out_channels;
    p.makes_dz = a.activation != BSS_ACT_NONE || a.gate != nullptr || a.dout_dtype == BSS_DTYPE_F32;
    p.makes_dz = p.makes_dz && (a.dx != nullptr || a.dweight != nullptr);
    p.sums = a.dbias != nullptr || a.dgate != nullptr;
    // without a gate all rows are one group here
    const int64_t per = a.gate != nullptr ? a.rows_per_group : a.rows;
    p.groups = groups_of(a.rows, per);
    // about 16 blocks an SM over all columns, 4 of a column (every one leaves a row of sums
    // to be added: with 16 of a column dbias of 75,600 x 64 took 28 us instead of 8), of 32
    // rows at least
    const int64_t columns = (n + 255) / 256;
    int64_t want = (columns > 4 ? 16ll : 4 * columns) * num_sms() / columns;
    if (want < 1) want = 1;
    int64_t rows = (a.rows + want - 1) / want;
    if (rows < 32) rows = 32;
    if (per >= rows || p.groups == 1) {
        int64_t chunks = (per + rows - 1) / rows;
        if (chunks > 32768) chunks = 32768;
        p.units = (per + chunks - 1) / chunks;
        p.chunks = static_cast<int32_t>((per + p.units - 1) / p.units);
        p.blocks = p.groups * p.chunks;
    } else {
        p.units = (rows + per - 1) / per;
        p.chunks = 0;
        p.blocks = (p.groups + p.units - 1) / p.units;
    }
    p.bytes = 0;
    if (p.makes_dz) {
        p.dz_at = 0;
        p.bytes = aligned_up(a.rows * n * 2);
    }
    if (a.dbias != nullptr) {
        p.dbias_at = p.bytes;
        p.bytes += aligned_up(p.blocks * n * 4);
    }
    if (a.dgate != nullptr && p.chunks > 0) {
        p.dgate_at = p.bytes;
        p.bytes += aligned_up(p.blocks * n * 4);
    }
    int64_t sums = 0;
    if (a.dx != nullptr) {
        p.dx = cut_of(a.rows, a.in_channels, n);
        sums = cut_bytes(p.dx, a.rows, a.in_channels);
    }
    if (a.dweight != nullptr) {
        p.dweight = cut_of(n, a.in_channels, a.rows);
        const int64_t b = cut_bytes(p.dweight, n, a.in_channels);
        if (b > sums) sums = b;
    }
    p.sums_at = p.bytes;
    p.bytes += sums;
    return p;
}

bss_status check_grads(bss_linear_grads& a) {
    bss_status st = check_sizes(a.rows, &a.rows_per_group, a.in_channels, a.out_channels, a.activation);
    if (st != BSS_OK) return st;
    if (!known_dtype(a.dout_dtype) || !known_dtype(a.param_dtype) || !known_dtype(a.dweight_dtype))
        return set_error(BSS_ERR_INVALID_ARG, "unknown dtype");
    if (a.dout == nullptr) return set_error(BSS_ERR_INVALID_ARG, "dout is NULL");
    if (a.dx == nullptr && a.dweight == nullptr && a.dbias == nullptr && a.dgate == nullptr)
        return set_error(BSS_ERR_INVALID_ARG, "no gradient is wanted");
    if (a.dx != nullptr && a.weight == nullptr) return set_error(BSS_ERR_INVALID_ARG, "dx needs weight");
    if (a.dweight != nullptr && a.x == nullptr) return set_error(BSS_ERR_INVALID_ARG, "dweight needs x");
    if (a.dgate != nullptr && a.gate == nullptr) return set_error(BSS_ERR_INVALID_ARG, "dgate needs gate");
    if ((a.dgate != nullptr || a.activation != BSS_ACT_NONE) && a.pre == nullptr)
        return set_error(BSS_ERR_INVALID_ARG, "an activation's slope and dgate need pre");
    return BSS_OK;
}

template <int ACT>
bss_status launch_dz(const DzArgs& d, int64_t blocks, cudaStream_t stream) {
    const unsigned columns = static_cast<unsigned>((d.n + 255) / 256);
    const dim3 grid(columns, static_cast<unsigned>(blocks));
    const bool wide = d.dout_dtype == BSS_DTYPE_F32;
    auto kernel = d.gate != nullptr ? (wide ? dz_kernel<ACT, true, true> : dz_kernel<ACT, false, true>)
                                    : (wide ? dz_kernel<ACT, true, false> : dz_kernel<ACT, false, false>);
    return launch_behind(kernel, grid, 32 * kDzWarps, stream, "dz launch", d);
}

}  // namespace
}  // namespace bss

extern "C" {

bss_status bss_linear_workspace(const bss_linear_args* args, int64_t* bytes) {
    using namespace bss;
    clear_error();
    if (bytes == nullptr) return set_error(BSS_ERR_INVALID_ARG, "bytes is NULL");
    *bytes = 0;
    if (args == nullptr) return set_error(BSS_ERR_INVALID_ARG, "args is NULL");
    bss_linear_args a = *args;
    const bss_status st = check_linear(a);
    if (st != BSS_OK) return st;
    *bytes = linear_need(a);
    return BSS_OK;
}

bss_status bss_linear(const bss_linear_args* args, cudaStream_t stream) {
    using namespace bss;
    clear_error();
    if (args == nullptr) return set_error(BSS_ERR_INVALID_ARG, "args is NULL");
    bss_linear_args a = *args;
    bss_status st = check_linear(a);
    if (st != BSS_OK) return st;
    const int64_t groups = groups_of(a.rows, a.rows_per_group), need = linear_need(a);
    Operand t[8];
    if ((st = check_matrix(&t[0], a.x, "x", a.rows, a.x_stride, a.in_channels, BSS_DTYPE_BF16, false)) != BSS_OK ||
        (st = check_matrix(&t[1], a.weight, "weight", a.out_channels, a.weight_stride, a.in_channels, BSS_DTYPE_BF16, false)) != BSS_OK ||
        (st = check_matrix(&t[2], a.bias, "bias", 1, 0, a.out_channels, a.param_dtype, false)) != BSS_OK ||
        (st = check_matrix(&t[3], a.gate, "gate", groups, a.gate_stride, a.out_channels, a.param_dtype, false)) != BSS_OK ||
        (st = check_matrix(&t[4], a.residual, "residual", a.rows, a.residual_stride, a.out_channels, a.out_dtype, false)) != BSS_OK ||
        (st = check_matrix(&t[5], a.out, "out", a.rows, a.out_stride, a.out_channels, a.out_dtype, true)) != BSS_OK ||
        (st = check_matrix(&t[6], a.pre, "pre", a.rows, a.pre_stride, a.out_channels, BSS_DTYPE_BF16, true)) != BSS_OK ||
        (st = check_run(&t[7], need > 0 ? a.workspace : nullptr, "workspace", need, 16, true)) != BSS_OK ||
        (st = check_workspace(a.workspace, a.workspace_bytes, need)) != BSS_OK)
        return st;
    t[5].over = 4;
    if ((st = check_outputs(t, 8)) != BSS_OK) return st;
    Epilogue e = {};
    e.bias = a.bias, e.gate = a.gate, e.residual = a.residual, e.out = a.out, e.pre = a.pre;
    e.gate_stride = a.gate_stride, e.residual_stride = a.residual_stride;
    e.out_stride = a.out_stride, e.pre_stride = a.pre_stride;
    e.param_dtype = a.param_dtype, e.out_dtype = a.out_dtype, e.activation = a.activation;
    e.residual_scale = a.residual_scale;
    e.by_rows = FastDiv(static_cast<uint32_t>(a.rows_per_group));
    if (takes_few(a)) {
        FewArgs f;
        f.x = static_cast<const __nv_bfloat16*>(a.x), f.weight = static_cast<const __nv_bfloat16*>(a.weight);
        f.x_stride = a.x_stride, f.weight_stride = a.weight_stride;
        f.rows = static_cast<int32_t>(a.rows), f.inner = a.in_channels, f.outer = a.out_channels, f.e = e;
        return by_activation(a.activation, [&](auto act) { return launch_few<decltype(act)::value>(f, stream); });
    }
    return gemm<false, false>(a.x, a.x_stride, a.weight, a.weight_stride, a.rows, a.out_channels, a.in_channels,
                              cut_of(a.rows, a.out_channels, a.in_channels), static_cast<float*>(a.workspace), e, stream);
}

bss_status bss_linear_backward_workspace(const bss_linear_grads* args, int64_t* bytes) {
    using namespace bss;
    clear_error();
    if (bytes == nullptr) return set_error(BSS_ERR_INVALID_ARG, "bytes is NULL");
    *bytes = 0;
    if (args == nullptr) return set_error(BSS_ERR_INVALID_ARG, "args is NULL");
    bss_linear_grads a = *args;
    const bss_status st = check_grads(a);
    if (st != BSS_OK) return st;
    *bytes = plan_of(a).bytes;
    return BSS_OK;
}

bss_status bss_linear_backward(const bss_linear_grads* args, cudaStream_t stream) {
    using namespace bss;
    clear_error();
    if (args == nullptr) return set_error(BSS_ERR_INVALID_ARG, "args is NULL");
    bss_linear_grads a = *args;
    bss_status st = check_grads(a);
    if (st != BSS_OK) return st;
    const GradPlan p = plan_of(a);
    // what is not read is not looked at
    if (a.dx == nullptr) a.weight = nullptr;
    if (a.dweight == nullptr) a.x = nullptr;
    if (a.activation == BSS_ACT_NONE && a.dgate == nullptr) a.pre = nullptr;
    const int64_t n = a.out_channels, k = a.in_channels;
    Operand t[10];
    if ((st = check_matrix(&t[0], a.dout, "dout", a.rows, a.dout_stride, n, a.dout_dtype, false)) != BSS_OK ||
        (st = check_matrix(&t[1], a.x, "x", a.rows, a.x_stride, k, BSS_DTYPE_BF16, false)) != BSS_OK ||
        (st = check_matrix(&t[2], a.weight, "weight", n, a.weight_stride, k, BSS_DTYPE_BF16, false)) != BSS_OK ||
        (st = check_matrix(&t[3], a.pre, "pre", a.rows, a.pre_stride, n, BSS_DTYPE_BF16, false)) != BSS_OK ||
        (st = check_matrix(&t[4], a.gate, "gate", groups_of(a.rows, a.rows_per_group), a.gate_stride, n, a.param_dtype, false)) != BSS_OK ||
        (st = check_matrix(&t[5], a.dx, "dx", a.rows, a.dx_stride, k, BSS_DTYPE_BF16, true)) != BSS_OK ||
        (st = check_matrix(&t[6], a.dweight, "dweight", n, a.dweight_stride, k, a.dweight_dtype, true)) != BSS_OK ||
        (st = check_run(&t[7], a.dbias, "dbias", 4 * n, 16, true)) != BSS_OK ||
        (st = check_run(&t[8], a.dgate, "dgate", 4 * n * p.groups, 16, true)) != BSS_OK ||
        (st = check_run(&t[9], p.bytes > 0 ? a.workspace : nullptr, "workspace", p.bytes, 16, true)) != BSS_OK ||
        (st = check_workspace(a.workspace, a.workspace_bytes, p.bytes)) != BSS_OK ||
        (st = check_outputs(t, 10)) != BSS_OK)
        return st;
    char* ws = static_cast<char*>(a.workspace);
    float* sums = reinterpret_cast<float*>(ws + p.sums_at);
    const void* dz = a.dout;
    int64_t dz_stride = a.dout_stride;
    if (p.makes_dz || p.sums) {
        DzArgs d = {};
        d.dout = a.dout, d.gate = a.gate, d.pre = static_cast<const __nv_bfloat16*>(a.pre);
        if (p.makes_dz) {
            d.dz = reinterpret_cast<__nv_bfloat16*>(ws + p.dz_at);
            dz = d.dz, dz_stride = n;
        }
        if (a.dbias != nullptr) d.dbias = reinterpret_cast<float*>(ws + p.dbias_at);
        if (a.dgate != nullptr) d.dgate = p.chunks > 0 ? reinterpret_cast<float*>(ws + p.dgate_at) : a.dgate;
        d.rows = a.rows, d.group_rows = a.gate != nullptr ? a.rows_per_group : a.rows;
        d.dout_stride = a.dout_stride, d.pre_stride = a.pre_stride, d.gate_stride = a.gate_stride;
        d.units = p.units, d.chunks = p.chunks;
        d.n = a.out_channels, d.dout_dtype = a.dout_dtype, d.param_dtype = a.param_dtype;
        st = by_activation(a.activation, [&](auto act) { return launch_dz<decltype(act)::value>(d, p.blocks, stream); });
        if (st != BSS_OK) return st;
        const unsigned columns = static_cast<unsigned>((n + 31) / 32);
        SumArgs sum = {d.dbias, p.chunks > 0 ? d.dgate : nullptr, a.dbias, a.dgate, p.blocks, p.chunks, a.out_channels};
        const int64_t sum_rows = (sum.bias_parts != nullptr) + (sum.gate_parts != nullptr ? p.groups : 0);
        if (sum_rows > 0)
            st = launch_behind(sum_parts_kernel, dim3(columns, static_cast<unsigned>(sum_rows)), 256, stream,
                               "bias and gate gradient launch", sum);
        if (st != BSS_OK) return st;
    }
    Epilogue e = {};
    if (a.dx != nullptr) {
        e.out = a.dx, e.out_stride = a.dx_stride, e.out_dtype = BSS_DTYPE_BF16;
        st = gemm<false, true>(dz, dz_stride, a.weight, a.weight_stride, a.rows, k, n, p.dx, sums, e, stream);
        if (st != BSS_OK) return st;
    }
    if (a.dweight != nullptr) {
        e.out = a.dweight, e.out_stride = a.dweight_stride, e.out_dtype = a.dweight_dtype;
        st = gemm<true, true>(dz, dz_stride, a.x, a.x_stride, n, k, a.rows, p.dweight, sums, e, stream);
    }
    return st;
}

}  // extern "C"
