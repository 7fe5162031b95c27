// bss_cross.cuh -- what the two passes of the cross attention share: the call's
// geometry, its checks and the tensor maps.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <cmath>

#include "bss_args.h"
#include "bss_rows.cuh"

namespace bss {

constexpr int64_t kMaxStateStride = int64_t(1) << 38;
constexpr int kKeyTile = 128;  // keys of a tile
constexpr int kHalfRows = 128; // query rows of an MMA

// What the kernels of both passes know of a call.
struct CrossShape {
    int32_t rows, group_rows, groups, heads, kv_heads, share, keys;
    int32_t shared_states;  // 1: one set of states for all groups
    const int32_t* lengths;
    float scale_log2;  // softmax_scale log2(e)
    FastDiv by_heads, by_share;

    // valid keys of a group
    __device__ __forceinline__ int valid(int g) const {
        if (lengths == nullptr) return keys;
        const int n = __ldg(lengths + g);
        return n < 0 ? 0 : (n > keys ? keys : n);
    }
    __device__ __forceinline__ int rows_of(int g) const {
        const int left = rows - g * group_rows;
        return left < group_rows ? left : group_rows;
    }
};

// Rows of a tile that hold nothing valid, up to the next multiple of 16 (as far as an
// MMA reads): zeroed, because a zero weight times what they hold may be NaN.  By one
// warp, whose lanes meet at a barrier of their own (32 arrivals; a bounded wait, unlike
// a warp's, in case one of them gave up elsewhere), before the MMAs it issues then.
template <int D>
__device__ __forceinline__ bool clear_rows(uint8_t* tile, int first, uint64_t* bar, uint32_t& uses, int* status) {
    const int lane = threadIdx.x & 31, end = (first + 15) & ~15;
    for (int i = lane; i < (end - first) * (D / 8); i += 32) {
        const int row = first + i / (D / 8), unit = i % (D / 8);
        *reinterpret_cast<uint4*>(tile + (unit >> 3) * kChunkBytesSw128 + row * 128 + (unit & 7) * 16) = make_uint4(0, 0, 0, 0);
    }
    fence_proxy_async_smem();
    mbar_arrive(bar);
    return mbar_wait(bar, uses++ & 1, status);
}

// Groups of N lanes hold a row each, N 16-byte units of it a lane; afterwards lane i of
// a group has unit i of its N rows.
template <int N>
__device__ __forceinline__ void transpose_units(uint4 (&u)[N]) {
#pragma unroll
    for (int o = N / 2; o > 0; o >>= 1) {
        const bool upper = (threadIdx.x & o) != 0;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if (i & o) continue;
            const uint4 send = upper ? u[i] : u[i | o];
            uint4 got;
            got.x = __shfl_xor_sync(0xFFFFFFFFu, send.x, o);
            got.y = __shfl_xor_sync(0xFFFFFFFFu, send.y, o);
            got.z = __shfl_xor_sync(0xFFFFFFFFu, send.z, o);
            got.w = __shfl_xor_sync(0xFFFFFFFFu, send.w, o);
            if (upper) u[i] = got;
            else u[i | o] = got;
        }
    }
}

// COLS accumulator columns of the warp's 32 rows (a lane of TMEM each) times a factor
// a row, as bf16: 16-byte units of a lane's own row.
template <int COLS>
__device__ __forceinline__ void read_rows(uint4 (&u)[COLS / 8], uint32_t at, float factor) {
#pragma unroll
    for (int c = 0; c < COLS / 32; ++c) {
        uint32_t o[32];
        BSS_TMEM_LD32(at + 32 * c, o);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t w[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const float2 y = __fmul2_rn(make_float2(__uint_as_float(o[8 * i + 2 * x]), __uint_as_float(o[8 * i + 2 * x + 1])), f2(factor));
                w[x] = pack_bf16x2(y.x, y.y);
            }
            u[4 * c + i] = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
}

// They -> memory; `to`: the first row's first column, `rows` of the 32 exist.  A lane
// alone would write 16 bytes of 32 rows at a time (a cycle of the memory pipe each);
// transposed, 8 lanes write 128 bytes of one row together.
template <int UNITS>
__device__ __forceinline__ void write_rows(const uint4 (&v)[UNITS], uint16_t* to, int64_t row_stride, int rows) {
    constexpr int N = UNITS < 8 ? UNITS : 8;
    const int lane = threadIdx.x & 31, unit = lane % N, first = lane - unit;
#pragma unroll
    for (int c = 0; c < UNITS; c += N) {
        uint4 u[N];
#pragma unroll
        for (int i = 0; i < N; ++i) u[i] = v[c + i];
        transpose_units<N>(u);
        uint16_t* p = to + (c + unit) * 8 + first * row_stride;
#pragma unroll
        for (int k = 0; k < N; ++k, p += row_stride)
            if (first + k < rows) *reinterpret_cast<uint4*>(p) = u[k];
        __syncwarp();
    }
}

// Both; a lane whose row is not live writes zeros.
template <int COLS>
__device__ __forceinline__ void store_rows(uint32_t at, uint16_t* to, int64_t row_stride, int rows, float factor, bool live) {
#pragma unroll
    for (int c = 0; c < COLS; c += 64) {  // 128 bytes a row at a time
        constexpr int kCols = COLS < 64 ? COLS : 64;
        uint4 u[kCols / 8];
        read_rows<kCols>(u, at + c, factor);
#pragma unroll
        for (int i = 0; i < kCols / 8; ++i)
            if (!live) u[i] = make_uint4(0, 0, 0, 0);
        write_rows<kCols / 8>(u, to + c, row_stride, rows);
    }
}

// ---------------------------------------------------------------- few rows
// A key to eight lanes, each with d / 8 of its channels.  16 warps a block: one row x 10 x
// 128 over 2,048 states 14.8 us forward and 16.3 backward, with 8 warps 21.9 and 23.9, with 32
// (which spill) 18.2 and 31.6.
constexpr int kFewThreads = 512, kFewWarps = kFewThreads / 32;

// A lane's channels of a row: 16-byte units 8 apart.
template <int N>
__device__ __forceinline__ void load_part(const uint16_t* row, int unit, float (&x)[8 * N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const uint4 u = *reinterpret_cast<const uint4*>(row + 8 * (unit + 8 * i));
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            x[8 * i + 2 * j] = __uint_as_float(w[j] << 16);
            x[8 * i + 2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
        }
    }
}

template <int N>
__device__ __forceinline__ void store_part(uint16_t* row, int unit, const float (&x)[8 * N], float scale) {
#pragma unroll
    for (int i = 0; i < N; ++i)
        *reinterpret_cast<uint4*>(row + 8 * (unit + 8 * i)) =
            make_uint4(pack2(x[8 * i] * scale, x[8 * i + 1] * scale), pack2(x[8 * i + 2] * scale, x[8 * i + 3] * scale),
                       pack2(x[8 * i + 4] * scale, x[8 * i + 5] * scale), pack2(x[8 * i + 6] * scale, x[8 * i + 7] * scale));
}

// The eight lanes' sum of products.
template <int N>
__device__ __forceinline__ float dot_part(const float (&x)[8 * N], const float (&y)[8 * N]) {
    float a = 0.0f, b = 0.0f;
#pragma unroll
    for (int i = 0; i < 8 * N; i += 2) a = fmaf(x[i], y[i], a), b = fmaf(x[i + 1], y[i + 1], b);
    a += b;
#pragma unroll
    for (int m = 1; m < 8; m *= 2) a += __shfl_xor_sync(0xFFFFFFFFu, a, m);
    return a;
}

// ---------------------------------------------------------------- host side
bss_status check_cross_sizes(int64_t rows, int64_t* rows_per_group, int32_t heads, int32_t kv_heads, int32_t head_dim,
                             int32_t keys, float softmax_scale, const int32_t* lengths);

// [rows][heads][d]
bss_status check_row_heads(Operand* o, const bss_token_tensor& t, const char* name, int64_t rows, int32_t heads, int32_t d,
                           bool output);
// [groups][keys][heads][d]
bss_status check_states(Operand* o, const bss_state_tensor& t, const char* name, int64_t groups, int64_t keys, int32_t heads,
                        int32_t d, bool output);

CrossShape cross_shape(int64_t rows, int64_t rows_per_group, int32_t heads, int32_t kv_heads, int32_t head_dim, int32_t keys,
                       float softmax_scale, const int32_t* lengths, int64_t group_stride);

// Tiles of 64 channels x `box` rows: coordinates (channel, row, head) and (channel, key, head, group).
bss_status row_heads_map(CUtensorMap* map, const bss_token_tensor& t, int64_t rows, int32_t heads, int32_t d, int box);
bss_status states_map(CUtensorMap* map, const bss_state_tensor& t, int64_t groups, int64_t keys, int32_t heads, int32_t d,
                      int box);

}  // namespace bss
