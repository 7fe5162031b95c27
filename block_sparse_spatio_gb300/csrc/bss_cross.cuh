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

// Rows of a key tile that hold no valid state up to the next multiple of 16 (as far
// as an MMA reads): zeroed, because a zero weight times what they hold may be NaN.
// By one warp; ordered before the MMAs that it issues afterwards.
template <int D>
__device__ __forceinline__ void clear_rows(uint8_t* tile, uint32_t chunk_bytes, int first) {
    const int lane = threadIdx.x & 31, end = (first + 15) & ~15;
    for (int i = lane; i < (end - first) * (D / 8); i += 32) {
        const int row = first + i / (D / 8), unit = i % (D / 8);
        *reinterpret_cast<uint4*>(tile + (unit >> 3) * chunk_bytes + row * 128 + (unit & 7) * 16) = make_uint4(0, 0, 0, 0);
    }
    fence_proxy_async_smem();
    __syncwarp();
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
