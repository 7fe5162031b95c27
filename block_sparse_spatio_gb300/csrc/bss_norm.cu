// bss_norm.cu -- the residual update of a block fused with the norm in front of
// the next one, forward and backward.
//
// Forward, per row (token):
//   r = a x + gate * y_norm(y) * y_weight
//   h = (norm(r) * weight + bias) * (1 + scale) + shift
// Backward, with xh = (r - mean) rstd, yh = y_norm(y), t = dh (1 + scale) weight:
//   u  = dr + rstd (t - mean(t) - xh mean(t xh))        (RMS: without mean(t))
//   dx = a u,   z = u gate y_weight
//   dy = z, or rstd_y (z - mean(z) - yh mean(z yh))
//   A = sum dh xh, B = sum dh, C = sum u yh over the rows of a group, and from
//   them every parameter's gradient: dscale = weight A + bias B, dshift = B,
//   dgate = y_weight C, dweight = sum over groups of (1 + scale) A,
//   dbias = sum of (1 + scale) B, dy_weight = sum of gate C.
//
// HBM-bound: each row's tensors are read once and written once (bf16: 8 bytes a
// channel forward, 12 backward), everything else stays on chip.  Statistics and
// sums are 32-bit; a variance is taken about the mean, not as a difference of
// squares.
#include <cstring>

#include "bss_rows.cuh"

namespace bss {
namespace {

constexpr int kMaxChannels = 8192;
constexpr int kMinChunkRows = 16;  // rows a block of the backward pass reduces at least

// Sum over the W warps that share a row (W = 1: the warp); every thread gets it.
// `buf` holds W floats and is used once between two barriers.
template <int W>
__device__ __forceinline__ float row_sum(float v, float* buf) {
    v = lane_sum<32>(v);
    if (W == 1) return v;
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.0f;
#pragma unroll
    for (int i = 0; i < W; ++i) v += buf[i];
    return v;
}

// ---------------------------------------------------------------- forward
// W warps share a row, each thread holding up to VPT vectors of it in registers.
// With W = 1 a block of 8 warps takes 8 rows; else one.
template <typename TS, typename TB, int W, int VPT>
__global__ void __launch_bounds__(W == 1 ? 256 : 32 * W) norm_forward_kernel(const __grid_constant__ bss_residual_norm_args a) {
    __shared__ float buf[4][W];
    constexpr int kRows = W == 1 ? 8 : 1;
    const int lane = W == 1 ? threadIdx.x & 31 : threadIdx.x;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * kRows + (W == 1 ? threadIdx.x >> 5 : 0);
    if (row >= a.rows) return;  // whole warps (W = 1) or never
    const int vecs = a.channels / 8;
    const float inv = 1.0f / a.channels;
    const int64_t group = row / a.rows_per_group;
    float r[VPT][8];
    {
        Raw8<TS> xr[VPT];
        Raw8<TB> yr[VPT];
        const TS* x = static_cast<const TS*>(a.x) + row * a.x_stride;
        const TB* y = static_cast<const TB*>(a.y) + row * a.y_stride;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int v = lane + i * 32 * W;
            xr[i] = zero_raw<TS>();
            yr[i] = zero_raw<TB>();
            if (v < vecs) xr[i] = load_raw(x + v * 8);
            if (v < vecs && a.y != nullptr) yr[i] = load_raw(y + v * 8);
        }
        float ym = 0.0f, yrstd = 1.0f;
        if (a.y != nullptr && a.y_norm != BSS_NORM_NONE) {
            float s = 0.0f;
            if (a.y_norm == BSS_NORM_LAYER) {
#pragma unroll
                for (int i = 0; i < VPT; ++i) {
                    float v[8];
                    unpack(yr[i], v);
#pragma unroll
                    for (int j = 0; j < 8; ++j) s += v[j];
                }
                ym = row_sum<W>(s, buf[0]) * inv;
            }
            s = 0.0f;
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                if (lane + i * 32 * W >= vecs) continue;
                float v[8];
                unpack(yr[i], v);
#pragma unroll
                for (int j = 0; j < 8; ++j) s = fmaf(v[j] - ym, v[j] - ym, s);
            }
            yrstd = rsqrtf(row_sum<W>(s, buf[1]) * inv + a.eps);
            if (a.y_stats != nullptr && lane == 0)
                *reinterpret_cast<float2*>(a.y_stats + 2 * row) = make_float2(ym, yrstd);
        }
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int v = lane + i * 32 * W;
            unpack(xr[i], r[i]);
            if (v >= vecs || a.y == nullptr) continue;
            float yv[8], p[8];
            unpack(yr[i], yv);
#pragma unroll
            for (int j = 0; j < 8; ++j) yv[j] = (yv[j] - ym) * yrstd;
            if (a.y_weight != nullptr) {
                load_param8(a.y_weight, v * 8, a.param_dtype, p);
#pragma unroll
                for (int j = 0; j < 8; ++j) yv[j] *= p[j];
            }
            if (a.gate != nullptr) {
                load_param8(a.gate, group * a.gate_stride + v * 8, a.param_dtype, p);
#pragma unroll
                for (int j = 0; j < 8; ++j) yv[j] *= p[j];
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) r[i][j] = fmaf(a.residual_scale, r[i][j], yv[j]);
            if (a.r != nullptr) store8(static_cast<TS*>(a.r) + row * a.r_stride + v * 8, r[i]);
        }
    }
    if (a.h == nullptr) return;
    float mean = 0.0f, rstd = 1.0f;
    if (a.norm != BSS_NORM_NONE) {
        float s = 0.0f;
        if (a.norm == BSS_NORM_LAYER) {
#pragma unroll
            for (int i = 0; i < VPT; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) s += r[i][j];  // vectors past the row hold zeros
            mean = row_sum<W>(s, buf[2]) * inv;
        }
        s = 0.0f;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            if (lane + i * 32 * W >= vecs) continue;
#pragma unroll
            for (int j = 0; j < 8; ++j) s = fmaf(r[i][j] - mean, r[i][j] - mean, s);
        }
        rstd = rsqrtf(row_sum<W>(s, buf[3]) * inv + a.eps);
        if (a.stats != nullptr && lane == 0) *reinterpret_cast<float2*>(a.stats + 2 * row) = make_float2(mean, rstd);
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int v = lane + i * 32 * W;
        if (v >= vecs) continue;
        float p[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) r[i][j] = (r[i][j] - mean) * rstd;
        if (a.weight != nullptr) {
            load_param8(a.weight, v * 8, a.param_dtype, p);
#pragma unroll
            for (int j = 0; j < 8; ++j) r[i][j] *= p[j];
        }
        if (a.bias != nullptr) {
            load_param8(a.bias, v * 8, a.param_dtype, p);
#pragma unroll
            for (int j = 0; j < 8; ++j) r[i][j] += p[j];
        }
        if (a.scale != nullptr) {
            load_param8(a.scale, group * a.scale_stride + v * 8, a.param_dtype, p);
#pragma unroll
            for (int j = 0; j < 8; ++j) r[i][j] = fmaf(r[i][j], p[j], r[i][j]);
        }
        if (a.shift != nullptr) {
            load_param8(a.shift, group * a.shift_stride + v * 8, a.param_dtype, p);
#pragma unroll
            for (int j = 0; j < 8; ++j) r[i][j] += p[j];
        }
        store8(static_cast<TB*>(a.h) + row * a.h_stride + v * 8, r[i]);
    }
}

// ---------------------------------------------------------------- backward
// A thread owns 8 channels and walks over rows, so the three column sums stay in
// its registers; `lanes` warps share a row, several rows go side by side in a
// block when a row is short.  A block covers one chunk of one group's rows.
struct GradShape {
    int warps;        // per row
    int side;         // rows side by side
    int threads;
    int64_t groups, chunks, chunk_rows;  // chunks per group
};

struct GradArgs {
    bss_residual_norm_grads a;
    GradShape s;
    float* partial;   // [groups][chunks][3][channels]
    int want_sums;
};

// Sums of N values over the row's warps.
template <int N>
__device__ __forceinline__ void shared_sums(float (&v)[N], int warps, int warp0, float* buf) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = lane_sum<32>(v[i]);
    if (warps == 1) return;
    if ((threadIdx.x & 31) == 0) {
#pragma unroll
        for (int i = 0; i < N; ++i) buf[(threadIdx.x >> 5) * N + i] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = 0.0f;
    for (int w = warp0; w < warp0 + warps; ++w) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += buf[w * N + i];
    }
}

template <typename TS, typename TB, int T>
__global__ void __launch_bounds__(T == 1 ? 1024 : 512) norm_backward_kernel(const __grid_constant__ GradArgs g) {
    extern __shared__ __align__(16) float shared[];  // sums of the row's warps; column sums of the rows side by side
    __shared__ float buf[4][32 * 2 * T];
    const bss_residual_norm_grads& a = g.a;
    const int per = g.s.warps * 32;
    const int side = threadIdx.x / per;
    const int v = threadIdx.x - side * per;
    const int warp0 = side * g.s.warps;
    const bool active = v * 8 < a.channels;
    const int c = active ? v * 8 : 0;
    const float inv = 1.0f / a.channels;
    const int64_t group = blockIdx.x / g.s.chunks, chunk = blockIdx.x - group * g.s.chunks;
    const int64_t first = group * a.rows_per_group + chunk * g.s.chunk_rows;
    int64_t last = first + g.s.chunk_rows;
    if (last > (group + 1) * a.rows_per_group) last = (group + 1) * a.rows_per_group;
    if (last > a.rows) last = a.rows;

    float m1[8], m2[8];  // (1 + scale) weight, gate y_weight
    {
        float p[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) m1[j] = m2[j] = 1.0f;
        if (a.scale != nullptr) {
            load_param8(a.scale, group * a.scale_stride + c, a.param_dtype, p);
#pragma unroll
            for (int j = 0; j < 8; ++j) m1[j] += p[j];
        }
        if (a.weight != nullptr) {
            load_param8(a.weight, c, a.param_dtype, p);
#pragma unroll
            for (int j = 0; j < 8; ++j) m1[j] *= p[j];
        }
        if (a.gate != nullptr) load_param8(a.gate, group * a.gate_stride + c, a.param_dtype, m2);
        if (a.y_weight != nullptr) {
            load_param8(a.y_weight, c, a.param_dtype, p);
#pragma unroll
            for (int j = 0; j < 8; ++j) m2[j] *= p[j];
        }
        if (!active) {  // lanes past the row: u there is -mean(t), keep it out of the sums over z
#pragma unroll
            for (int j = 0; j < 8; ++j) m2[j] = 0.0f;
        }
    }
    float sa[8], sb[8], sc[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) sa[j] = sb[j] = sc[j] = 0.0f;
    const bool stats = a.dh != nullptr && a.norm != BSS_NORM_NONE;
    const bool ystats = a.y != nullptr && a.y_norm != BSS_NORM_NONE;
    int turn = 0;
    for (int64_t row0 = first; row0 < last; row0 += g.s.side * T, turn ^= 2) {
        const int64_t mine = row0 + side * T;
        Raw8<TS> rr[T], drr[T];
        Raw8<TB> yr[T], dhr[T];
        float2 st[T], yst[T];
#pragma unroll
        for (int t = 0; t < T; ++t) {
            const int64_t row = mine + t;
            const bool live = active && row < last;
            rr[t] = zero_raw<TS>();
            drr[t] = zero_raw<TS>();
            yr[t] = zero_raw<TB>();
            dhr[t] = zero_raw<TB>();
            st[t] = yst[t] = make_float2(0.0f, 1.0f);
            if (!live) continue;
            if (a.dh != nullptr) {
                rr[t] = load_raw(static_cast<const TS*>(a.r) + row * a.r_stride + c);
                dhr[t] = load_raw(static_cast<const TB*>(a.dh) + row * a.dh_stride + c);
            }
            if (a.dr != nullptr) drr[t] = load_raw(static_cast<const TS*>(a.dr) + row * a.dr_stride + c);
            if (a.y != nullptr) yr[t] = load_raw(static_cast<const TB*>(a.y) + row * a.y_stride + c);
            if (stats) st[t] = __ldg(reinterpret_cast<const float2*>(a.stats) + row);
            if (ystats) yst[t] = __ldg(reinterpret_cast<const float2*>(a.y_stats) + row);
        }
        float sums[2 * T];
#pragma unroll
        for (int t = 0; t < T; ++t) {
            float rv[8], dhv[8], s1 = 0.0f, s2 = 0.0f;
            unpack(rr[t], rv);
            unpack(dhr[t], dhv);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float xh = (rv[j] - st[t].x) * st[t].y;
                const float tt = dhv[j] * m1[j];
                s1 += tt;
                s2 = fmaf(tt, xh, s2);
                sa[j] = fmaf(dhv[j], xh, sa[j]);
                sb[j] += dhv[j];
            }
            sums[2 * t] = s1;
            sums[2 * t + 1] = s2;
        }
        if (stats) shared_sums<2 * T>(sums, g.s.warps, warp0, buf[turn]);
        float u[T][8], zs[2 * T];
#pragma unroll
        for (int t = 0; t < T; ++t) {
            float rv[8], dhv[8], yv[8], out[8];
            unpack(rr[t], rv);
            unpack(dhr[t], dhv);
            unpack(drr[t], u[t]);
            unpack(yr[t], yv);
            const float mean1 = a.norm == BSS_NORM_LAYER ? sums[2 * t] * inv : 0.0f;
            const float mean2 = a.norm != BSS_NORM_NONE ? sums[2 * t + 1] * inv : 0.0f;
            float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float xh = (rv[j] - st[t].x) * st[t].y;
                const float tt = dhv[j] * m1[j];
                u[t][j] += st[t].y * (tt - mean1 - xh * mean2);
                out[j] = u[t][j] * a.residual_scale;
                const float yh = (yv[j] - yst[t].x) * yst[t].y;
                sc[j] = fmaf(u[t][j], yh, sc[j]);
                const float z = u[t][j] * m2[j];
                s1 += z;
                s2 = fmaf(z, yh, s2);
                u[t][j] = z;
            }
            zs[2 * t] = s1;
            zs[2 * t + 1] = s2;
            if (active && mine + t < last) store8(static_cast<TS*>(a.dx) + (mine + t) * a.dx_stride + c, out);
        }
        if (a.dy == nullptr) continue;
        if (ystats) shared_sums<2 * T>(zs, g.s.warps, warp0, buf[turn + 1]);
#pragma unroll
        for (int t = 0; t < T; ++t) {
            if (ystats) {
                float yv[8];
                unpack(yr[t], yv);
                const float mean1 = a.y_norm == BSS_NORM_LAYER ? zs[2 * t] * inv : 0.0f;
                const float mean2 = zs[2 * t + 1] * inv;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float yh = (yv[j] - yst[t].x) * yst[t].y;
                    u[t][j] = yst[t].y * (u[t][j] - mean1 - yh * mean2);
                }
            }
            if (active && mine + t < last) store8(static_cast<TB*>(a.dy) + (mine + t) * a.dy_stride + c, u[t]);
        }
    }
    if (!g.want_sums) return;
    // the rows side by side, in order
    const int C = a.channels;
    float* dst = g.partial + static_cast<int64_t>(blockIdx.x) * 3 * C;
    if (g.s.side > 1) {
        if (active) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                shared[(side * 3 + 0) * C + c + j] = sa[j];
                shared[(side * 3 + 1) * C + c + j] = sb[j];
                shared[(side * 3 + 2) * C + c + j] = sc[j];
            }
        }
        __syncthreads();
        for (int e = threadIdx.x; e < 3 * C; e += blockDim.x) {
            float s = 0.0f;
            for (int k = 0; k < g.s.side; ++k) s += shared[k * 3 * C + e];
            dst[e] = s;
        }
    } else if (active) {
#pragma unroll
        for (int j = 0; j < 8; j += 4) {
            *reinterpret_cast<float4*>(dst + c + j) = make_float4(sa[j], sa[j + 1], sa[j + 2], sa[j + 3]);
            *reinterpret_cast<float4*>(dst + C + c + j) = make_float4(sb[j], sb[j + 1], sb[j + 2], sb[j + 3]);
            *reinterpret_cast<float4*>(dst + 2 * C + c + j) = make_float4(sc[j], sc[j + 1], sc[j + 2], sc[j + 3]);
        }
    }
}

// One group's column sums over its chunks (in order within 8 lanes, then the
// lanes), the modulations' gradients, and the sums kept in the group's first
// chunk for the weights' gradients.
__global__ void __launch_bounds__(256) norm_groups_kernel(const __grid_constant__ GradArgs g) {
    __shared__ float part[3][8][33];
    const bss_residual_norm_grads& a = g.a;
    const int C = a.channels, col = threadIdx.x % 32, lane = threadIdx.x / 32;
    const int c = blockIdx.x * 32 + col;
    for (int64_t group = blockIdx.y; group < g.s.groups; group += gridDim.y) {
        float* base = g.partial + group * g.s.chunks * 3 * C;
        float s[3] = {0.0f, 0.0f, 0.0f};
        if (c < C)
            for (int64_t k = lane; k < g.s.chunks; k += 8)
#pragma unroll
                for (int q = 0; q < 3; ++q) s[q] += base[(k * 3 + q) * C + c];
#pragma unroll
        for (int q = 0; q < 3; ++q) part[q][lane][col] = s[q];
        __syncthreads();
        if (lane == 0 && c < C) {
#pragma unroll
            for (int q = 0; q < 3; ++q) {
                s[q] = 0.0f;
#pragma unroll
                for (int k = 0; k < 8; ++k) s[q] += part[q][k][col];
                base[q * C + c] = s[q];
            }
            const float w = a.weight != nullptr ? load_param(a.weight, c, a.param_dtype) : 1.0f;
            const float b = a.bias != nullptr ? load_param(a.bias, c, a.param_dtype) : 0.0f;
            const float wy = a.y_weight != nullptr ? load_param(a.y_weight, c, a.param_dtype) : 1.0f;
            if (a.dscale != nullptr) a.dscale[group * C + c] = fmaf(w, s[0], b * s[1]);
            if (a.dshift != nullptr) a.dshift[group * C + c] = s[1];
            if (a.dgate != nullptr) a.dgate[group * C + c] = wy * s[2];
        }
        __syncthreads();
    }
}

// The weights' gradients: over the groups, in order within 8 lanes.
__global__ void __launch_bounds__(256) norm_weights_kernel(const __grid_constant__ GradArgs g) {
    __shared__ float part[3][8][33];
    const bss_residual_norm_grads& a = g.a;
    const int C = a.channels, col = threadIdx.x % 32, lane = threadIdx.x / 32;
    const int c = blockIdx.x * 32 + col;
    float s[3] = {0.0f, 0.0f, 0.0f};
    if (c < C)
        for (int64_t group = lane; group < g.s.groups; group += 8) {
            const float* base = g.partial + group * g.s.chunks * 3 * C;
            const float m = a.scale != nullptr ? 1.0f + load_param(a.scale, group * a.scale_stride + c, a.param_dtype) : 1.0f;
            const float gt = a.gate != nullptr ? load_param(a.gate, group * a.gate_stride + c, a.param_dtype) : 1.0f;
            s[0] = fmaf(m, base[c], s[0]);
            s[1] = fmaf(m, base[C + c], s[1]);
            s[2] = fmaf(gt, base[2 * C + c], s[2]);
        }
#pragma unroll
    for (int q = 0; q < 3; ++q) part[q][lane][col] = s[q];
    __syncthreads();
    if (lane != 0 || c >= C) return;
    float* out[3] = {a.dweight, a.dbias, a.dy_weight};
#pragma unroll
    for (int q = 0; q < 3; ++q) {
        float t = 0.0f;
#pragma unroll
        for (int k = 0; k < 8; ++k) t += part[q][k][col];
        if (out[q] != nullptr) out[q][c] = t;
    }
}

// ---------------------------------------------------------------- host side

int esize(int32_t dtype) { return dtype == BSS_DTYPE_F32 ? 4 : 2; }

bss_status check_common(int64_t rows, int64_t rows_per_group, int32_t channels, int32_t sd, int32_t bd, int32_t pd,
                        int32_t norm, int32_t y_norm, float residual_scale) {
    if (rows <= 0 || rows_per_group <= 0) return set_error(BSS_ERR_INVALID_ARG, "rows and rows_per_group must be positive");
    if (rows > (int64_t(1) << 31) - 1) return set_error(BSS_ERR_UNSUPPORTED, "too many rows");
    if (channels < 8 || channels % 8 != 0)
        return set_error(BSS_ERR_INVALID_ARG, "channels must be a positive multiple of 8 (got %d)", channels);
    if (channels > kMaxChannels) return set_error(BSS_ERR_UNSUPPORTED, "at most %d channels (got %d)", kMaxChannels, channels);
    for (int32_t t : {sd, bd, pd})
        if (t != BSS_DTYPE_BF16 && t != BSS_DTYPE_F32)
            return set_error(BSS_ERR_INVALID_ARG, "element types must be 0 (bf16) or 1 (float)");
    if (sd == BSS_DTYPE_BF16 && bd == BSS_DTYPE_F32)
        return set_error(BSS_ERR_UNSUPPORTED, "a float branch on a bf16 stream is not supported");
    for (int32_t n : {norm, y_norm})
        if (n < BSS_NORM_NONE || n > BSS_NORM_RMS) return set_error(BSS_ERR_INVALID_ARG, "norm must be 0 (none), 1 (layer) or 2 (RMS)");
    if (!(residual_scale >= -3.0e38f && residual_scale <= 3.0e38f))
        return set_error(BSS_ERR_INVALID_ARG, "residual_scale is not finite");
    return BSS_OK;
}

// One row tensor (NULL passes): alignment, stride, the bytes it touches.
bss_status check_rows(const void* p, const char* name, int64_t rows, int64_t stride, int32_t channels, int32_t dtype,
                      bool output, Region* r) {
    if (p == nullptr) return BSS_OK;
    if (!is_aligned(p, 16)) return set_error(BSS_ERR_INVALID_ARG, "%s must be 16-byte aligned", name);
    if (rows > 1 && (stride % 8 != 0 || stride < 0 || stride > (int64_t(1) << 31)))
        return set_error(BSS_ERR_INVALID_ARG, "%s: the row stride must be a multiple of 8 elements, 0 .. 2^31", name);
    *r = region_2d(p, rows, stride, channels, esize(dtype));
    if (output && r->self_overlap) return set_error(BSS_ERR_INVALID_ARG, "%s: rows overlap", name);
    return BSS_OK;
}

bss_status check_param(const void* p, const char* name, int64_t groups, int64_t stride, int32_t channels, int32_t dtype,
                       Region* r) {
    return check_rows(p, name, groups, stride, channels, dtype, false, r);
}

// Inputs may be named twice; an output must share no byte with any other tensor,
// but for the pairs that may be the same tensor.
struct Named {
    const void* p;
    Region r;
    bool output;
    const void* same;  // the input this output may equal
};

bss_status check_overlaps(const Named* t, int n) {
    for (int i = 0; i < n; ++i) {
        if (t[i].p == nullptr || !t[i].output) continue;
        for (int j = 0; j < n; ++j) {
            if (j == i || t[j].p == nullptr || (t[j].output && j < i)) continue;
            if (!t[j].output && t[i].same != nullptr && t[j].p == t[i].same && t[i].p == t[j].p &&
                t[i].r.stride == t[j].r.stride && t[i].r.extent == t[j].r.extent && !t[j].r.self_overlap)
                continue;
            if (!disjoint(t[i].r, t[j].r)) return set_error(BSS_ERR_INVALID_ARG, "an output overlaps another tensor");
        }
    }
    return BSS_OK;
}

template <typename TS, typename TB, int W, int VPT>
bss_status launch_forward(const bss_residual_norm_args& a, cudaStream_t stream) {
    const int64_t blocks = W == 1 ? (a.rows + 7) / 8 : a.rows;
    norm_forward_kernel<TS, TB, W, VPT><<<static_cast<unsigned>(blocks), W == 1 ? 256 : 32 * W, 0, stream>>>(a);
    return cuda_check(cudaGetLastError(), "residual norm launch");
}

// Warps per row by the row's vectors: a warp alone needs no barrier and holds up
// to 5 vectors a lane (1280 channels); longer rows take 8 warps.
template <typename TS, typename TB>
bss_status forward_of(const bss_residual_norm_args& a, cudaStream_t stream) {
    const int vecs = a.channels / 8;
    if (vecs <= 32) return launch_forward<TS, TB, 1, 1>(a, stream);
    if (vecs <= 64) return launch_forward<TS, TB, 1, 2>(a, stream);
    if (vecs <= 160) return launch_forward<TS, TB, 1, 5>(a, stream);
    if (vecs <= 512) return launch_forward<TS, TB, 8, 2>(a, stream);
    return launch_forward<TS, TB, 8, 4>(a, stream);
}

bool wants_sums(const bss_residual_norm_grads& a) {
    return a.dgate || a.dscale || a.dshift || a.dweight || a.dbias || a.dy_weight;
}

// Whether rows of different groups differ at all (else one group holds them).
bool grouped(const bss_residual_norm_grads& a) {
    return a.gate || a.scale || a.dgate || a.dscale || a.dshift;
}

GradShape grad_shape(const bss_residual_norm_grads& a) {
    GradShape s;
    s.warps = (a.channels / 8 + 31) / 32;
    s.side = s.warps >= 4 ? 1 : 4 / s.warps;
    s.threads = s.warps * s.side * 32;
    const int64_t per_group = !grouped(a) || a.rows_per_group > a.rows ? a.rows : a.rows_per_group;
    s.groups = (a.rows + per_group - 1) / per_group;
    const int64_t per_sm = s.threads >= 512 ? 1 : 512 / s.threads;
    const int64_t most = (per_sm * num_sms() + s.groups - 1) / s.groups;
    s.chunks = (per_group + kMinChunkRows - 1) / kMinChunkRows;
    if (s.chunks > most) s.chunks = most;
    s.chunk_rows = (per_group + s.chunks - 1) / s.chunks;
    s.chunks = (per_group + s.chunk_rows - 1) / s.chunk_rows;
    return s;
}

int64_t grad_workspace(const bss_residual_norm_grads& a, const GradShape& s) {
    return wants_sums(a) ? s.groups * s.chunks * 3 * a.channels * 4 : 0;
}

template <typename TS, typename TB>
bss_status launch_backward(const GradArgs& g, cudaStream_t stream) {
    const int smem = g.s.side > 1 && g.want_sums ? g.s.side * 3 * g.a.channels * 4 : 0;
    const unsigned grid = static_cast<unsigned>(g.s.groups * g.s.chunks);
    if (g.s.threads <= 512)
        norm_backward_kernel<TS, TB, 2><<<grid, g.s.threads, smem, stream>>>(g);
    else
        norm_backward_kernel<TS, TB, 1><<<grid, g.s.threads, smem, stream>>>(g);
    return cuda_check(cudaGetLastError(), "residual norm backward launch");
}

bss_status check_grads(const bss_residual_norm_grads* args) {
    if (args == nullptr) return set_error(BSS_ERR_INVALID_ARG, "args is NULL");
    return check_common(args->rows, args->rows_per_group, args->channels, args->stream_dtype, args->branch_dtype,
                        args->param_dtype, args->norm, args->y_norm, args->residual_scale);
}

}  // namespace
}  // namespace bss

extern "C" {

bss_status bss_residual_norm(const bss_residual_norm_args* args, cudaStream_t stream) {
    using namespace bss;
    clear_error();
    if (args == nullptr) return set_error(BSS_ERR_INVALID_ARG, "args is NULL");
    bss_residual_norm_args a = *args;
    bss_status st = check_common(a.rows, a.rows_per_group, a.channels, a.stream_dtype, a.branch_dtype, a.param_dtype,
                                 a.norm, a.y_norm, a.residual_scale);
    if (st != BSS_OK) return st;
    if (!(a.eps >= 0.0f) || a.eps > 3.0e38f) return set_error(BSS_ERR_INVALID_ARG, "eps must be finite and not negative");
    if (a.x == nullptr) return set_error(BSS_ERR_INVALID_ARG, "x is NULL");
    if (a.r == nullptr && a.h == nullptr) return set_error(BSS_ERR_INVALID_ARG, "r and h are both NULL");
    if (a.y == nullptr &&
        (a.r != nullptr || a.gate != nullptr || a.y_weight != nullptr || a.y_stats != nullptr ||
         a.y_norm != BSS_NORM_NONE || a.residual_scale != 1.0f))
        return set_error(BSS_ERR_INVALID_ARG, "without y there is no r, gate, y_norm, y_weight, y_stats or residual_scale");
    if (a.h == nullptr && (a.scale != nullptr || a.shift != nullptr || a.weight != nullptr || a.bias != nullptr))
        return set_error(BSS_ERR_INVALID_ARG, "without h there is no scale, shift, weight or bias");
    if ((a.stats != nullptr && (a.h == nullptr || a.norm == BSS_NORM_NONE)) ||
        (a.y_stats != nullptr && a.y_norm == BSS_NORM_NONE))
        return set_error(BSS_ERR_INVALID_ARG, "statistics are only written by a norm");
    if (!is_aligned(a.stats, 8) || !is_aligned(a.y_stats, 8))
        return set_error(BSS_ERR_INVALID_ARG, "statistics must be 8-byte aligned");
    const int64_t groups = (a.rows + a.rows_per_group - 1) / a.rows_per_group;
    Named t[12] = {{a.x, {}, false, nullptr},     {a.y, {}, false, nullptr},        {a.gate, {}, false, nullptr},
                   {a.scale, {}, false, nullptr}, {a.shift, {}, false, nullptr},    {a.weight, {}, false, nullptr},
                   {a.bias, {}, false, nullptr},  {a.y_weight, {}, false, nullptr}, {a.r, {}, true, a.x},
                   {a.h, {}, true, a.y},          {a.stats, {}, true, nullptr},     {a.y_stats, {}, true, nullptr}};
    if ((st = check_rows(a.x, "x", a.rows, a.x_stride, a.channels, a.stream_dtype, false, &t[0].r)) != BSS_OK ||
        (st = check_rows(a.y, "y", a.rows, a.y_stride, a.channels, a.branch_dtype, false, &t[1].r)) != BSS_OK ||
        (st = check_param(a.gate, "gate", groups, a.gate_stride, a.channels, a.param_dtype, &t[2].r)) != BSS_OK ||
        (st = check_param(a.scale, "scale", groups, a.scale_stride, a.channels, a.param_dtype, &t[3].r)) != BSS_OK ||
        (st = check_param(a.shift, "shift", groups, a.shift_stride, a.channels, a.param_dtype, &t[4].r)) != BSS_OK ||
        (st = check_param(a.weight, "weight", 1, 0, a.channels, a.param_dtype, &t[5].r)) != BSS_OK ||
        (st = check_param(a.bias, "bias", 1, 0, a.channels, a.param_dtype, &t[6].r)) != BSS_OK ||
        (st = check_param(a.y_weight, "y_weight", 1, 0, a.channels, a.param_dtype, &t[7].r)) != BSS_OK ||
        (st = check_rows(a.r, "r", a.rows, a.r_stride, a.channels, a.stream_dtype, true, &t[8].r)) != BSS_OK ||
        (st = check_rows(a.h, "h", a.rows, a.h_stride, a.channels, a.branch_dtype, true, &t[9].r)) != BSS_OK)
        return st;
    t[10].r = region_2d(a.stats, 1, 0, 2 * a.rows, 4);
    t[11].r = region_2d(a.y_stats, 1, 0, 2 * a.rows, 4);
    if ((st = check_overlaps(t, 12)) != BSS_OK) return st;
    if (groups == 1) a.gate_stride = a.scale_stride = a.shift_stride = 0;
    if (a.stream_dtype == BSS_DTYPE_BF16) return forward_of<__nv_bfloat16, __nv_bfloat16>(a, stream);
    if (a.branch_dtype == BSS_DTYPE_BF16) return forward_of<float, __nv_bfloat16>(a, stream);
    return forward_of<float, float>(a, stream);
}

bss_status bss_residual_norm_backward_workspace(const bss_residual_norm_grads* args, int64_t* bytes) {
    using namespace bss;
    clear_error();
    if (bytes == nullptr) return set_error(BSS_ERR_INVALID_ARG, "bytes is NULL");
    *bytes = 0;
    const bss_status st = check_grads(args);
    if (st != BSS_OK) return st;
    *bytes = grad_workspace(*args, grad_shape(*args));
    return BSS_OK;
}

bss_status bss_residual_norm_backward(const bss_residual_norm_grads* args, cudaStream_t stream) {
    using namespace bss;
    clear_error();
    bss_status st = check_grads(args);
    if (st != BSS_OK) return st;
    GradArgs g;
    memset(&g, 0, sizeof(g));
    g.a = *args;
    bss_residual_norm_grads& a = g.a;
    if (a.dx == nullptr) return set_error(BSS_ERR_INVALID_ARG, "dx is NULL");
    if (a.dr == nullptr && a.dh == nullptr) return set_error(BSS_ERR_INVALID_ARG, "dr and dh are both NULL");
    if (a.dh != nullptr && a.r == nullptr) return set_error(BSS_ERR_INVALID_ARG, "the norm's gradient needs r");
    if (a.dh != nullptr && a.norm != BSS_NORM_NONE && a.stats == nullptr)
        return set_error(BSS_ERR_INVALID_ARG, "the norm's gradient needs stats");
    if ((a.y == nullptr) != (a.dy == nullptr)) return set_error(BSS_ERR_INVALID_ARG, "y and dy must be given together");
    if (a.y != nullptr && a.y_norm != BSS_NORM_NONE && a.y_stats == nullptr)
        return set_error(BSS_ERR_INVALID_ARG, "the gradient of y_norm needs y_stats");
    if (a.y == nullptr && (a.gate != nullptr || a.y_weight != nullptr || a.dgate != nullptr || a.dy_weight != nullptr ||
                           a.y_norm != BSS_NORM_NONE || a.residual_scale != 1.0f))
        return set_error(BSS_ERR_INVALID_ARG, "without y there is no gate, y_norm, y_weight or residual_scale");
    if (a.dh == nullptr && (a.dscale != nullptr || a.dshift != nullptr || a.dweight != nullptr || a.dbias != nullptr))
        return set_error(BSS_ERR_INVALID_ARG, "without dh there is no dscale, dshift, dweight or dbias");
    if (!is_aligned(a.stats, 8) || !is_aligned(a.y_stats, 8))
        return set_error(BSS_ERR_INVALID_ARG, "statistics must be 8-byte aligned");
    for (const float* p : {a.dgate, a.dscale, a.dshift, a.dweight, a.dbias, a.dy_weight})
        if (!is_aligned(p, 16)) return set_error(BSS_ERR_INVALID_ARG, "parameter gradients must be 16-byte aligned");
    const int64_t groups = (a.rows + a.rows_per_group - 1) / a.rows_per_group;
    g.s = grad_shape(a);
    const int64_t need = grad_workspace(a, g.s);
    if (need > 0 && (a.workspace == nullptr || !is_aligned(a.workspace, 16) || a.workspace_bytes < need))
        return set_error(BSS_ERR_INVALID_ARG, "the workspace must be 16-byte aligned and hold %lld bytes",
                         static_cast<long long>(need));
    // with dh NULL r is not read, without y_norm or norm neither are the statistics
    const void* r = a.dh != nullptr ? a.r : nullptr;
    const void* stats = a.dh != nullptr && a.norm != BSS_NORM_NONE ? a.stats : nullptr;
    const void* ystats = a.y_norm != BSS_NORM_NONE ? a.y_stats : nullptr;
    Named t[20] = {{r, {}, false, nullptr},          {a.y, {}, false, nullptr},      {a.dr, {}, false, nullptr},
                   {a.dh, {}, false, nullptr},       {a.gate, {}, false, nullptr},   {a.scale, {}, false, nullptr},
                   {a.weight, {}, false, nullptr},   {a.bias, {}, false, nullptr},   {a.y_weight, {}, false, nullptr},
                   {stats, {}, false, nullptr},      {ystats, {}, false, nullptr},   {a.dx, {}, true, a.dr},
                   {a.dy, {}, true, a.dh},           {a.dgate, {}, true, nullptr},   {a.dscale, {}, true, nullptr},
                   {a.dshift, {}, true, nullptr},    {a.dweight, {}, true, nullptr}, {a.dbias, {}, true, nullptr},
                   {a.dy_weight, {}, true, nullptr}, {need > 0 ? a.workspace : nullptr, {}, true, nullptr}};
    if ((st = check_rows(r, "r", a.rows, a.r_stride, a.channels, a.stream_dtype, false, &t[0].r)) != BSS_OK ||
        (st = check_rows(a.y, "y", a.rows, a.y_stride, a.channels, a.branch_dtype, false, &t[1].r)) != BSS_OK ||
        (st = check_rows(a.dr, "dr", a.rows, a.dr_stride, a.channels, a.stream_dtype, false, &t[2].r)) != BSS_OK ||
        (st = check_rows(a.dh, "dh", a.rows, a.dh_stride, a.channels, a.branch_dtype, false, &t[3].r)) != BSS_OK ||
        (st = check_param(a.gate, "gate", groups, a.gate_stride, a.channels, a.param_dtype, &t[4].r)) != BSS_OK ||
        (st = check_param(a.scale, "scale", groups, a.scale_stride, a.channels, a.param_dtype, &t[5].r)) != BSS_OK ||
        (st = check_param(a.weight, "weight", 1, 0, a.channels, a.param_dtype, &t[6].r)) != BSS_OK ||
        (st = check_param(a.bias, "bias", 1, 0, a.channels, a.param_dtype, &t[7].r)) != BSS_OK ||
        (st = check_param(a.y_weight, "y_weight", 1, 0, a.channels, a.param_dtype, &t[8].r)) != BSS_OK ||
        (st = check_rows(a.dx, "dx", a.rows, a.dx_stride, a.channels, a.stream_dtype, true, &t[11].r)) != BSS_OK ||
        (st = check_rows(a.dy, "dy", a.rows, a.dy_stride, a.channels, a.branch_dtype, true, &t[12].r)) != BSS_OK)
        return st;
    t[9].r = region_2d(stats, 1, 0, 2 * a.rows, 4);
    t[10].r = region_2d(ystats, 1, 0, 2 * a.rows, 4);
    for (int i = 13; i < 19; ++i) t[i].r = region_2d(t[i].p, 1, 0, (i < 16 ? groups : 1) * a.channels, 4);
    t[19].r = region_2d(a.workspace, 1, 0, need, 1);
    if ((st = check_overlaps(t, 20)) != BSS_OK) return st;
    if (groups == 1) a.gate_stride = a.scale_stride = 0;
    if (a.dh == nullptr) a.norm = BSS_NORM_NONE;
    a.rows_per_group = g.s.groups == 1 ? a.rows : a.rows_per_group;
    g.want_sums = wants_sums(a);
    g.partial = static_cast<float*>(a.workspace);
    if (a.stream_dtype == BSS_DTYPE_BF16) st = launch_backward<__nv_bfloat16, __nv_bfloat16>(g, stream);
    else if (a.branch_dtype == BSS_DTYPE_BF16) st = launch_backward<float, __nv_bfloat16>(g, stream);
    else st = launch_backward<float, float>(g, stream);
    if (st != BSS_OK || !g.want_sums) return st;
    const unsigned cols = (a.channels + 31) / 32;
    norm_groups_kernel<<<dim3(cols, static_cast<unsigned>(g.s.groups < 4096 ? g.s.groups : 4096)), 256, 0, stream>>>(g);
    if ((st = cuda_check(cudaGetLastError(), "modulation gradient launch")) != BSS_OK) return st;
    if (a.dweight == nullptr && a.dbias == nullptr && a.dy_weight == nullptr) return BSS_OK;
    norm_weights_kernel<<<cols, 256, 0, stream>>>(g);
    return cuda_check(cudaGetLastError(), "weight gradient launch");
}

}  // extern "C"
