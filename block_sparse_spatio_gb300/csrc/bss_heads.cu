// bss_heads.cu -- token-major Q, K, V <-> the attention calls' heads.
//
// Forward, for token n = (f, h, w) and head i:
//   norm      x^ = x * rsqrt(mean(x^2) + eps) * weight   (Q, K; over the head's
//             channels or over the whole token)
//   rotary    every pair of channels of x^ turned by its angle: the pair's axis
//             (time, height or width) picks the table, the token's position the
//             row (Q, K)
//   layout    row n of head i, or row s*F + f when the head is temporal (section
//             "Arrange tokens for efficient temporal access")
// Backward: the layout undone, the rotation by the opposite angle, then the
// norm's gradient
//   dx = r (g w - x r^2 mean(g w x)),   dweight = sum over rows of g x r.
//
// HBM-bound: forward reads and writes Q, K, V once (12 bytes an element of one
// tensor), backward reads dQ, dK, dV, Q, K and writes dq, dk, dv (16 bytes).
//
// A thread owns one 16-byte piece (8 channels) of one head and walks over
// tokens, so the weights and, in the backward pass, the weights' gradients stay
// in its registers.  d / 8 neighbouring lanes hold a head's row: global rows are
// read and written whole (128 or 256 bytes).  The angles of a block's tokens are
// gathered into shared memory once and used by all heads of Q and K.
#include <cstring>

#include "bss_rows.cuh"

namespace bss {
namespace {

constexpr int kMaxThreads = 1024;
constexpr int kMaxTokenWidth = 8192;  // H * head_dim of the norm over a token: one thread a piece

struct RotaryDev {
    const float2* table[3];
    int32_t first[4];   // first pair of each axis; [3] = all pairs
    int32_t pairs[3];
    int32_t offset[3];
};

struct HeadsArgs {
    const __nv_bfloat16* in[3];   // token-major q, k, v (forward), head-major dQh, dKh, dVh (backward)
    __nv_bfloat16* out[3];        // head-major (forward), token-major (backward)
    const __nv_bfloat16* x[2];    // backward: token-major q, k
    int64_t ts[3], hs[3];         // strides of the token-major tensors in / out
    int64_t xts[2], xhs[2];       // strides of x
    const void* weight[2];
    int32_t weight_dtype;
    float eps;
    RotaryDev rot;
    const uint8_t* flags;
    uint32_t N, F, S, Ws, H;
    int32_t heads_per_block;      // heads a block covers (all of them for the norm over a token)
    int32_t groups;               // tokens side by side in a block
    int32_t want_dweight;
    float* partial;               // backward: [blocks][2][width]
};

// Shared-memory layout of one buffer (two alternate between iterations).
struct Smem {
    int cs;       // float2 [tokens][d / 2]
    int sums;     // float [tensors x values][tokens][heads padded to 4]
    int bytes;    // of one buffer
    int hpad;
};

__host__ __device__ inline Smem smem_layout(int tokens, int pieces, int heads, int values, bool rotary, bool token_norm) {
    Smem s;
    s.hpad = (heads + 3) & ~3;
    s.cs = 0;
    s.sums = rotary ? tokens * pieces * 4 * 8 : 0;
    s.bytes = s.sums + (token_norm ? values * tokens * s.hpad * 4 : 0);
    s.bytes = (s.bytes + 15) & ~15;
    return s;
}

// (cos, sin) of the block's tokens, pair by pair; pairs past the rotated ones
// get the identity.
template <int P>
__device__ __forceinline__ void fill_angles(const HeadsArgs& a, float2* cs, uint32_t token0, int tokens) {
    constexpr int kPairs = P * 4;
    for (int e = threadIdx.x; e < tokens * kPairs; e += blockDim.x) {
        const uint32_t n = token0 + e / kPairs;
        const int p = e % kPairs;
        float2 v = make_float2(1.0f, 0.0f);
        if (n < a.N && p < a.rot.first[3]) {
            const uint32_t f = n / a.S, s = n - f * a.S;
            const uint32_t h = s / a.Ws, w = s - h * a.Ws;
            const int axis = p < a.rot.first[1] ? 0 : (p < a.rot.first[2] ? 1 : 2);
            const int64_t row = (axis == 0 ? f : axis == 1 ? h : w) + a.rot.offset[axis];
            v = __ldg(a.rot.table[axis] + row * a.rot.pairs[axis] + (p - a.rot.first[axis]));
        }
        cs[e] = v;
    }
}

// Turn 8 channels by their angles (sign = -1: back).  Interleaved pairs lie in
// the thread; the two halves' channels in lanes R/16 pieces apart.
template <int P, bool HALVES>
__device__ __forceinline__ void rotate8(float (&v)[8], const float2* cs, int piece, int rotated, float sign) {
    if (!HALVES) {
        const float4* c4 = reinterpret_cast<const float4*>(cs + piece * 4);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float4 c = c4[i];
            const float a0 = v[4 * i], b0 = v[4 * i + 1], a1 = v[4 * i + 2], b1 = v[4 * i + 3];
            v[4 * i] = a0 * c.x - sign * (b0 * c.y);
            v[4 * i + 1] = b0 * c.x + sign * (a0 * c.y);
            v[4 * i + 2] = a1 * c.z - sign * (b1 * c.w);
            v[4 * i + 3] = b1 * c.z + sign * (a1 * c.w);
        }
    } else {
        const int half = rotated / 16;  // pieces per half
        const bool lower = piece < half, in = piece < 2 * half;
        const int other = in ? (lower ? piece + half : piece - half) : piece;
        const int lane = (threadIdx.x & 31 & ~(P - 1)) | other;
        const float4* c4 = reinterpret_cast<const float4*>(cs + (lower ? piece : other) * 8);
        const float sg = lower ? -sign : sign;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float o0 = __shfl_sync(0xFFFFFFFFu, v[2 * i], lane);
            const float o1 = __shfl_sync(0xFFFFFFFFu, v[2 * i + 1], lane);
            if (in) {
                const float4 c = c4[i];
                v[2 * i] = v[2 * i] * c.x + sg * (o0 * c.y);
                v[2 * i + 1] = v[2 * i + 1] * c.z + sg * (o1 * c.w);
            }
        }
    }
}

__device__ __forceinline__ uint32_t head_row(const HeadsArgs& a, uint32_t n, bool temporal) {
    if (!temporal) return n;
    const uint32_t f = n / a.S;
    return (n - f * a.S) * a.F + f;
}

// Sum of a token's per-head values in shared memory (padding heads hold 0).
__device__ __forceinline__ float sum_heads(const float* p, int hpad) {
    const float4* q = reinterpret_cast<const float4*>(p);
    float s = 0.0f;
    for (int i = 0; i < hpad / 4; ++i) {
        const float4 v = q[i];
        s += (v.x + v.y) + (v.z + v.w);
    }
    return s;
}

// What a thread owns: a piece of a head, in one of the block's token groups.
struct Place {
    int piece, head_local, group;
    uint32_t head;
    bool active;
};

template <int P>
__device__ __forceinline__ Place place_of(const HeadsArgs& a) {
    Place p;
    const int per = a.heads_per_block * P;
    p.group = threadIdx.x / per;
    const int i = threadIdx.x - p.group * per;
    p.head_local = i / P;
    p.piece = i % P;
    p.head = blockIdx.y * a.heads_per_block + p.head_local;
    p.active = p.group < a.groups && p.head < a.H;
    return p;
}

// NORM: BSS_HEAD_NORM_*; T: tokens a thread handles together.
template <int P, bool HALVES, int NORM, int T>
__global__ void __launch_bounds__(T == 1 ? kMaxThreads : 512) heads_forward_kernel(const __grid_constant__ HeadsArgs a) {
    extern __shared__ __align__(16) unsigned char smem[];
    const bool rotary = a.rot.first[3] > 0;
    const Place me = place_of<P>(a);
    const int tokens = a.groups * T;
    const Smem lay = smem_layout(tokens, P, a.heads_per_block, 2, rotary, NORM == BSS_HEAD_NORM_TOKEN);
    float2* cs = reinterpret_cast<float2*>(smem + lay.cs);
    float* sums = reinterpret_cast<float*>(smem + lay.sums);
    const uint32_t token0 = blockIdx.x * tokens;
    const uint32_t n0 = token0 + me.group * T;
    const bool temporal = me.active && a.flags != nullptr && a.flags[me.head] != 0;
    const int64_t c0 = me.piece * 8;

    Raw8<__nv_bfloat16> raw[3][T];
#pragma unroll
    for (int i = 0; i < 3; ++i)
#pragma unroll
        for (int t = 0; t < T; ++t) {
            raw[i][t] = zero_raw<__nv_bfloat16>();
            if (a.in[i] != nullptr && me.active && n0 + t < a.N)
                raw[i][t] = load_raw(a.in[i] + static_cast<int64_t>(n0 + t) * a.ts[i] + me.head * a.hs[i] + c0);
        }
    if (rotary) fill_angles<P>(a, cs, token0, tokens);

    // sums of squares: over a head's lanes, and for the norm over a token over
    // the heads through shared memory
    float ssq[2][T];
    if (NORM != BSS_HEAD_NORM_NONE) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int t = 0; t < T; ++t) {
                float v[8], s = 0.0f;
                unpack(raw[i][t], v);
#pragma unroll
                for (int j = 0; j < 8; ++j) s = fmaf(v[j], v[j], s);
                ssq[i][t] = lane_sum<P>(s);
                if (NORM == BSS_HEAD_NORM_TOKEN && me.group < a.groups) {
                    float* row = sums + (i * tokens + me.group * T + t) * lay.hpad;
                    if (me.piece == 0) row[me.head_local] = ssq[i][t];
                    if (me.head_local == 0 && me.piece < lay.hpad - a.heads_per_block)
                        row[a.heads_per_block + me.piece] = 0.0f;
                }
            }
    }
    if (rotary || NORM == BSS_HEAD_NORM_TOKEN) __syncthreads();

#pragma unroll
    for (int i = 0; i < 3; ++i) {
        if (a.in[i] == nullptr) continue;
        float w[8];
        const bool weighted = i < 2 && NORM != BSS_HEAD_NORM_NONE && a.weight[i < 2 ? i : 0] != nullptr;
        if (weighted && me.active)
            load_param8(a.weight[i < 2 ? i : 0], NORM == BSS_HEAD_NORM_TOKEN ? me.head * (P * 8) + c0 : c0,
                        a.weight_dtype, w);
        __nv_bfloat16* dst = a.out[i] + static_cast<int64_t>(me.active ? me.head : 0) * a.N * (P * 8) + c0;
#pragma unroll
        for (int t = 0; t < T; ++t) {
            const uint32_t n = n0 + t;
            const bool live = me.active && n < a.N;
            if (i == 2) {
                if (live) st_row(dst + static_cast<int64_t>(head_row(a, n, temporal)) * (P * 8), raw[i][t].q[0]);
                continue;
            }
            float v[8];
            unpack(raw[i][t], v);
            if (NORM != BSS_HEAD_NORM_NONE) {
                float s = ssq[i < 2 ? i : 0][t], width = P * 8;
                if (NORM == BSS_HEAD_NORM_TOKEN && me.group < a.groups) {
                    s = sum_heads(sums + (i * tokens + me.group * T + t) * lay.hpad, lay.hpad);
                    width *= a.H;
                }
                const float r = rsqrtf(s / width + a.eps);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = weighted ? v[j] * r * w[j] : v[j] * r;
            }
            if (rotary) {
                const int tok = me.group < a.groups ? me.group * T + t : 0;
                rotate8<P, HALVES>(v, cs + tok * (P * 4), me.piece, 2 * a.rot.first[3], 1.0f);
            }
            if (live) store8(dst + static_cast<int64_t>(head_row(a, n, temporal)) * (P * 8), v);
        }
    }
}

template <int P, bool HALVES, int NORM, int T>
__global__ void __launch_bounds__(T == 1 ? kMaxThreads : 512) heads_backward_kernel(const __grid_constant__ HeadsArgs a) {
    extern __shared__ __align__(16) unsigned char smem[];
    const bool rotary = a.rot.first[3] > 0;
    const Place me = place_of<P>(a);
    const int tokens = a.groups * T;
    const Smem lay = smem_layout(tokens, P, a.heads_per_block, 4, rotary, NORM == BSS_HEAD_NORM_TOKEN);
    const bool temporal = me.active && a.flags != nullptr && a.flags[me.head] != 0;
    const int64_t c0 = me.piece * 8;
    float w[2][8], dw[2][8];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int j = 0; j < 8; ++j) w[i][j] = 1.0f, dw[i][j] = 0.0f;
        if (NORM != BSS_HEAD_NORM_NONE && me.active && a.weight[i] != nullptr)
            load_param8(a.weight[i], NORM == BSS_HEAD_NORM_TOKEN ? me.head * (P * 8) + c0 : c0, a.weight_dtype, w[i]);
    }
    const uint32_t blocks = (a.N + tokens - 1) / tokens;
    int buffer = 0;
    for (uint32_t b = blockIdx.x; b < blocks; b += gridDim.x, buffer ^= 1) {
        float2* cs = reinterpret_cast<float2*>(smem + buffer * lay.bytes + lay.cs);
        float* sums = reinterpret_cast<float*>(smem + buffer * lay.bytes + lay.sums);
        const uint32_t token0 = b * tokens;
        const uint32_t n0 = token0 + me.group * T;
        Raw8<__nv_bfloat16> g[3][T], x[2][T];
#pragma unroll
        for (int i = 0; i < 3; ++i)
#pragma unroll
            for (int t = 0; t < T; ++t) {
                const uint32_t n = n0 + t;
                g[i][t] = zero_raw<__nv_bfloat16>();
                if (i < 2) x[i < 2 ? i : 0][t] = zero_raw<__nv_bfloat16>();
                if (a.in[i] == nullptr || !me.active || n >= a.N) continue;
                g[i][t] = load_raw(a.in[i] + (static_cast<int64_t>(me.head) * a.N + head_row(a, n, temporal)) * (P * 8) + c0);
                if (NORM != BSS_HEAD_NORM_NONE && i < 2)
                    x[i < 2 ? i : 0][t] = load_raw(a.x[i < 2 ? i : 0] + static_cast<int64_t>(n) * a.xts[i < 2 ? i : 0] +
                                                   me.head * a.xhs[i < 2 ? i : 0] + c0);
            }
        if (rotary) {
            fill_angles<P>(a, cs, token0, tokens);
            __syncthreads();
        }
        float gr[2][T][8], ssq[2][T], gx[2][T];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int t = 0; t < T; ++t) {
                unpack(g[i][t], gr[i][t]);
                if (rotary) {
                    const int tok = me.group < a.groups ? me.group * T + t : 0;
                    rotate8<P, HALVES>(gr[i][t], cs + tok * (P * 4), me.piece, 2 * a.rot.first[3], -1.0f);
                }
                if (NORM == BSS_HEAD_NORM_NONE) continue;
                float v[8], s = 0.0f, q = 0.0f;
                unpack(x[i][t], v);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    s = fmaf(v[j], v[j], s);
                    q = fmaf(gr[i][t][j] * w[i][j], v[j], q);
                }
                ssq[i][t] = lane_sum<P>(s);
                gx[i][t] = lane_sum<P>(q);
                if (NORM == BSS_HEAD_NORM_TOKEN && me.group < a.groups) {
                    float* row = sums + (2 * i * tokens + me.group * T + t) * lay.hpad;
                    float* row2 = row + tokens * lay.hpad;
                    if (me.piece == 0) row[me.head_local] = ssq[i][t], row2[me.head_local] = gx[i][t];
                    if (me.head_local == 0 && me.piece < lay.hpad - a.heads_per_block)
                        row[a.heads_per_block + me.piece] = row2[a.heads_per_block + me.piece] = 0.0f;
                }
            }
        if (NORM == BSS_HEAD_NORM_TOKEN) __syncthreads();
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            if (a.in[i] == nullptr) continue;
#pragma unroll
            for (int t = 0; t < T; ++t) {
                const uint32_t n = n0 + t;
                if (!me.active || n >= a.N) continue;
                __nv_bfloat16* dst = a.out[i] + static_cast<int64_t>(n) * a.ts[i] + me.head * a.hs[i] + c0;
                if (i == 2) {
                    st_row(dst, g[i][t].q[0]);
                    continue;
                }
                constexpr int kTwo = 1;
                const int k = i < 2 ? i : kTwo;
                float v[8];
                if (NORM != BSS_HEAD_NORM_NONE) {
                    float s = ssq[k][t], q = gx[k][t], width = P * 8;
                    if (NORM == BSS_HEAD_NORM_TOKEN) {
                        const float* row = sums + (2 * k * tokens + me.group * T + t) * lay.hpad;
                        s = sum_heads(row, lay.hpad);
                        q = sum_heads(row + tokens * lay.hpad, lay.hpad);
                        width *= a.H;
                    }
                    const float r = rsqrtf(s / width + a.eps);
                    const float m = r * r * (q / width);
                    unpack(x[k][t], v);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        dw[k][j] = fmaf(gr[k][t][j], v[j] * r, dw[k][j]);
                        v[j] = r * (gr[k][t][j] * w[k][j] - v[j] * m);
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] = gr[k][t][j];
                }
                store8(dst, v);
            }
        }
    }
    if (NORM == BSS_HEAD_NORM_NONE || !a.want_dweight) return;
    // the block's share of the weight gradients: over its token groups, and for
    // the norm over a head over its heads, in a fixed order
    __syncthreads();
    float* acc = reinterpret_cast<float*>(smem);  // [2][threads][8]
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[(i * blockDim.x + threadIdx.x) * 8 + j] = dw[i][j];
    __syncthreads();
    const int per = a.heads_per_block * P;
    const int width = NORM == BSS_HEAD_NORM_TOKEN ? per * 8 : P * 8;
    const int sources = NORM == BSS_HEAD_NORM_TOKEN ? a.groups : a.groups * a.heads_per_block;
    float* dst = a.partial + static_cast<int64_t>(blockIdx.y * gridDim.x + blockIdx.x) * 2 * width;
    for (int e = threadIdx.x; e < 2 * width; e += blockDim.x) {
        const int i = e / width, c = e - i * width;
        float s = 0.0f;
        for (int k = 0; k < sources; ++k) s += acc[i * blockDim.x * 8 + k * width + c];
        dst[e] = s;
    }
}

// out[c] = sum over the blocks' partials [blocks][2][width], blocks in order
// within 8 lanes, the lanes' sums in order.
__global__ void __launch_bounds__(256) heads_reduce_kernel(const float* __restrict__ partial, int blocks, int width,
                                                           float* dq_weight, float* dk_weight) {
    __shared__ float part[8][33];
    const int c = blockIdx.x * 32 + threadIdx.x % 32, lane = threadIdx.x / 32;
    float s = 0.0f;
    if (c < 2 * width)
        for (int b = lane; b < blocks; b += 8) s += partial[static_cast<int64_t>(b) * 2 * width + c];
    part[lane][threadIdx.x % 32] = s;
    __syncthreads();
    if (lane != 0 || c >= 2 * width) return;
    s = 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) s += part[k][threadIdx.x % 32];
    if (c < width) {
        if (dq_weight != nullptr) dq_weight[c] = s;
    } else if (dk_weight != nullptr) {
        dk_weight[c - width] = s;
    }
}

__global__ void rotary_table_kernel(const double* positions, int32_t length, int32_t pairs, int32_t dim, double base,
                                    float2* out) {
    const int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
    if (i >= static_cast<int64_t>(length) * pairs) return;
    const int64_t row = i / pairs;
    const int64_t j = i - row * pairs;
    const double pos = positions != nullptr ? positions[row] : static_cast<double>(row);
    const double angle = pos * pow(base, -2.0 * static_cast<double>(j) / dim);
    double sn, cn;
    sincos(angle, &sn, &cn);
    out[i] = make_float2(static_cast<float>(cn), static_cast<float>(sn));
}

// ---------------------------------------------------------------- host side

// How the heads are dealt to blocks: for the norm over a token one block holds
// them all; otherwise up to 256 threads' worth, several tokens side by side when
// the heads are few.
struct Shape {
    int heads_per_block, groups, threads, T, tokens;
    uint32_t grid_y;
};

Shape shape_of(int32_t H, int pieces, int32_t norm, int T) {
    Shape s;
    s.heads_per_block = norm == BSS_HEAD_NORM_TOKEN ? H : (H * pieces <= 256 ? H : 256 / pieces);
    const int per = s.heads_per_block * pieces;
    s.groups = per >= 128 ? 1 : 128 / per;
    s.threads = (per * s.groups + 31) / 32 * 32;
    s.T = s.threads > 512 ? 1 : T;
    s.tokens = s.groups * s.T;
    s.grid_y = static_cast<uint32_t>((H + s.heads_per_block - 1) / s.heads_per_block);
    return s;
}

constexpr int kForwardTokens = 4, kBackwardTokens = 2;

// Blocks of the backward pass: enough to fill the GPU, each walking over tokens
// so that a block leaves one partial sum of the weight gradients.
uint32_t backward_grid(const Shape& s, uint32_t N) {
    const uint32_t blocks = (N + s.tokens - 1) / s.tokens;
    const uint32_t per_sm = 1024 / s.threads > 0 ? 1024 / s.threads : 1;
    uint32_t most = per_sm * static_cast<uint32_t>(num_sms()) / s.grid_y;
    if (most < 1) most = 1;
    return blocks < most ? blocks : most;
}

bss_status check_geometry(const bss_mask_params* params, int32_t H) {
    const bss_status st = check_mask_params(params);
    if (st != BSS_OK) return st;
    if (H <= 0) return set_error(BSS_ERR_INVALID_ARG, "H must be positive");
    if (H > 65535) return set_error(BSS_ERR_UNSUPPORTED, "too many heads (at most 65535)");
    return BSS_OK;
}

bss_status check_norm(int32_t norm, int32_t H, int32_t d) {
    if (norm < BSS_HEAD_NORM_NONE || norm > BSS_HEAD_NORM_TOKEN)
        return set_error(BSS_ERR_INVALID_ARG, "norm must be 0 (none), 1 (head) or 2 (token)");
    if (norm == BSS_HEAD_NORM_TOKEN && static_cast<int64_t>(H) * d > kMaxTokenWidth)
        return set_error(BSS_ERR_UNSUPPORTED, "the norm over a token takes at most %d channels (got %lld)",
                         kMaxTokenWidth, static_cast<long long>(H) * d);
    return BSS_OK;
}

bool span_ok(int64_t n, int64_t stride) { return stride >= 0 && (n <= 1 || stride <= (int64_t(1) << 56) / n); }

// One token-major tensor: alignment and strides.
bss_status check_tokens(const bss_token_tensor* t, const char* name, uint32_t N, int32_t H, int32_t d, Region* r) {
    if (!is_aligned(t->data, 16)) return set_error(BSS_ERR_INVALID_ARG, "%s must be 16-byte aligned", name);
    const int64_t ts = N > 1 ? t->token_stride : 0, hs = H > 1 ? t->head_stride : 0;
    if (!span_ok(N, ts) || !span_ok(H, hs) || ts % 8 != 0 || hs % 8 != 0)
        return set_error(BSS_ERR_INVALID_ARG, "%s: strides must be multiples of 8 elements, not negative", name);
    *r = region_3d(t->data, N, ts, H, hs, d, 2);
    return BSS_OK;
}

// Options and the rotary tables' ranges -> kernel arguments.
bss_status set_options(const bss_heads_options* o, const bss_mask_params* p, int32_t H, HeadsArgs* a, int* pairing) {
    if (o == nullptr) return set_error(BSS_ERR_INVALID_ARG, "options is NULL");
    const bss_status st = check_norm(o->norm, H, p->head_dim);
    if (st != BSS_OK) return st;
    *pairing = BSS_PAIR_INTERLEAVED;
    if (o->norm != BSS_HEAD_NORM_NONE) {
        if (!(o->eps >= 0.0f) || o->eps > 3.0e38f) return set_error(BSS_ERR_INVALID_ARG, "eps must be finite and not negative");
        if (o->weight_dtype != BSS_DTYPE_BF16 && o->weight_dtype != BSS_DTYPE_F32)
            return set_error(BSS_ERR_INVALID_ARG, "weight_dtype must be 0 (bf16) or 1 (float)");
        if (!is_aligned(o->q_weight, 16) || !is_aligned(o->k_weight, 16))
            return set_error(BSS_ERR_INVALID_ARG, "weights must be 16-byte aligned");
        a->weight[0] = o->q_weight;
        a->weight[1] = o->k_weight;
        a->weight_dtype = o->weight_dtype;
        a->eps = o->eps;
    }
    if (o->rotary == nullptr) return BSS_OK;
    const bss_rotary& r = *o->rotary;
    if (r.pairing != BSS_PAIR_INTERLEAVED && r.pairing != BSS_PAIR_HALVES)
        return set_error(BSS_ERR_INVALID_ARG, "pairing must be 0 (interleaved) or 1 (halves)");
    const int32_t size[3] = {p->F, p->Hs, p->Ws};
    int64_t total = 0;
    for (int i = 0; i < 3; ++i) {
        if (r.pairs[i] < 0) return set_error(BSS_ERR_INVALID_ARG, "rotary pairs must not be negative");
        if (r.pairs[i] > 0) {
            if (r.table[i] == nullptr || !is_aligned(r.table[i], 16))
                return set_error(BSS_ERR_INVALID_ARG, "rotary table %d must be given, 16-byte aligned", i);
            if (r.offset[i] < 0 || static_cast<int64_t>(r.offset[i]) + size[i] > r.length[i])
                return set_error(BSS_ERR_INVALID_ARG, "rotary axis %d: positions %d .. %lld of a table of %d", i,
                                 r.offset[i], static_cast<long long>(r.offset[i]) + size[i] - 1, r.length[i]);
        }
        a->rot.table[i] = reinterpret_cast<const float2*>(r.table[i]);
        a->rot.pairs[i] = r.pairs[i];
        a->rot.offset[i] = r.offset[i];
        a->rot.first[i] = static_cast<int32_t>(total);
        total += r.pairs[i];
        if (2 * total > p->head_dim)
            return set_error(BSS_ERR_INVALID_ARG, "rotary pairs cover more than head_dim = %d channels", p->head_dim);
    }
    a->rot.first[3] = static_cast<int32_t>(total);
    if (r.pairing == BSS_PAIR_HALVES && (2 * total) % 16 != 0)
        return set_error(BSS_ERR_UNSUPPORTED, "paired halves need a multiple of 16 rotated channels (got %lld)",
                         static_cast<long long>(2 * total));
    *pairing = r.pairing;
    return BSS_OK;
}

using Kernel = void (*)(const HeadsArgs);

template <int P, bool HALVES, int T>
Kernel pick_forward(int32_t norm) {
    if (norm == BSS_HEAD_NORM_HEAD) return heads_forward_kernel<P, HALVES, BSS_HEAD_NORM_HEAD, T>;
    if (norm == BSS_HEAD_NORM_TOKEN) return heads_forward_kernel<P, HALVES, BSS_HEAD_NORM_TOKEN, T>;
    return heads_forward_kernel<P, HALVES, BSS_HEAD_NORM_NONE, T>;
}

template <int P, bool HALVES, int T>
Kernel pick_backward(int32_t norm) {
    if (norm == BSS_HEAD_NORM_HEAD) return heads_backward_kernel<P, HALVES, BSS_HEAD_NORM_HEAD, T>;
    if (norm == BSS_HEAD_NORM_TOKEN) return heads_backward_kernel<P, HALVES, BSS_HEAD_NORM_TOKEN, T>;
    return heads_backward_kernel<P, HALVES, BSS_HEAD_NORM_NONE, T>;
}

template <int P, bool HALVES>
Kernel pick_tokens(bool backward, int32_t norm, int T) {
    if (backward) return T == 1 ? pick_backward<P, HALVES, 1>(norm) : pick_backward<P, HALVES, kBackwardTokens>(norm);
    return T == 1 ? pick_forward<P, HALVES, 1>(norm) : pick_forward<P, HALVES, kForwardTokens>(norm);
}

Kernel pick(bool backward, int pieces, int pairing, int32_t norm, int T) {
    const bool halves = pairing == BSS_PAIR_HALVES;
    if (pieces == 16)
        return halves ? pick_tokens<16, true>(backward, norm, T) : pick_tokens<16, false>(backward, norm, T);
    return halves ? pick_tokens<8, true>(backward, norm, T) : pick_tokens<8, false>(backward, norm, T);
}

bss_status launch(Kernel k, const HeadsArgs& a, dim3 grid, int threads, int smem, cudaStream_t stream,
                  const char* what) {
    if (smem > 48 * 1024) {
        const bss_status st = cuda_check(
            cudaFuncSetAttribute(reinterpret_cast<const void*>(k), cudaFuncAttributeMaxDynamicSharedMemorySize, smem),
            "shared memory size");
        if (st != BSS_OK) return st;
    }
    k<<<grid, threads, smem, stream>>>(a);
    return cuda_check(cudaGetLastError(), what);
}

void set_geometry(const bss_mask_params* p, int32_t H, const uint8_t* flags, HeadsArgs* a) {
    a->F = p->F;
    a->S = static_cast<uint32_t>(p->Hs) * p->Ws;
    a->Ws = p->Ws;
    a->N = a->S * a->F;
    a->H = H;
    a->flags = flags;
}

}  // namespace
}  // namespace bss

extern "C" {

bss_status bss_rotary_table(const double* positions, int32_t length, int32_t pairs, int32_t dim, double base,
                            float* out, cudaStream_t stream) {
    using namespace bss;
    clear_error();
    if (length <= 0 || pairs <= 0 || dim <= 0) return set_error(BSS_ERR_INVALID_ARG, "length, pairs and dim must be positive");
    if (!(base > 0.0) || base > 1.0e300) return set_error(BSS_ERR_INVALID_ARG, "base must be positive and finite");
    if (out == nullptr || !is_aligned(out, 16) || !is_aligned(positions, 8))
        return set_error(BSS_ERR_INVALID_ARG, "out must be given, 16-byte aligned, positions 8-byte aligned");
    const int64_t n = static_cast<int64_t>(length) * pairs;
    if (n >= (int64_t(1) << 31)) return set_error(BSS_ERR_UNSUPPORTED, "rotary table of %lld entries is too large", (long long)n);
    rotary_table_kernel<<<static_cast<unsigned>((n + 127) / 128), 128, 0, stream>>>(positions, length, pairs, dim, base,
                                                                                 reinterpret_cast<float2*>(out));
    return cuda_check(cudaGetLastError(), "rotary table launch");
}

bss_status bss_heads_from_tokens(const bss_token_tensor* q, const bss_token_tensor* k, const bss_token_tensor* v,
                                 void* Qh, void* Kh, void* Vh, const uint8_t* head_is_temporal, int32_t H,
                                 const bss_mask_params* params, const bss_heads_options* options,
                                 cudaStream_t stream) {
    using namespace bss;
    clear_error();
    bss_status st = check_geometry(params, H);
    if (st != BSS_OK) return st;
    HeadsArgs a;
    memset(&a, 0, sizeof(a));
    int pairing = 0;
    if ((st = set_options(options, params, H, &a, &pairing)) != BSS_OK) return st;
    set_geometry(params, H, head_is_temporal, &a);
    const int d = params->head_dim;
    const bss_token_tensor* in[3] = {q, k, v};
    void* out[3] = {Qh, Kh, Vh};
    const char* names[3] = {"q", "k", "v"};
    Region rin[3], rout[3];
    int given = 0;
    for (int i = 0; i < 3; ++i) {
        const bool has = in[i] != nullptr && in[i]->data != nullptr;
        if (has != (out[i] != nullptr))
            return set_error(BSS_ERR_INVALID_ARG, "%s and its output must be given together", names[i]);
        if (!has) continue;
        ++given;
        if ((st = check_tokens(in[i], names[i], a.N, H, d, &rin[i])) != BSS_OK) return st;
        if (!is_aligned(out[i], 16)) return set_error(BSS_ERR_INVALID_ARG, "outputs must be 16-byte aligned");
        rout[i] = region_2d(out[i], 1, 0, static_cast<int64_t>(H) * a.N * d, 2);
        a.in[i] = static_cast<const __nv_bfloat16*>(in[i]->data);
        a.out[i] = static_cast<__nv_bfloat16*>(out[i]);
        a.ts[i] = a.N > 1 ? in[i]->token_stride : 0;
        a.hs[i] = H > 1 ? in[i]->head_stride : 0;
    }
    if (given == 0) return set_error(BSS_ERR_INVALID_ARG, "no tensor given");
    for (int i = 0; i < 3; ++i)
        for (int j = 0; j < 3; ++j) {
            if (a.out[i] != nullptr && a.in[j] != nullptr && !disjoint(rout[i], rin[j]))
                return set_error(BSS_ERR_INVALID_ARG, "an output overlaps an input");
            if (j < i && a.out[i] != nullptr && a.out[j] != nullptr && !disjoint(rout[i], rout[j]))
                return set_error(BSS_ERR_INVALID_ARG, "outputs overlap");
        }
    const int pieces = d / 8;
    const Shape s = shape_of(H, pieces, options->norm, kForwardTokens);
    const bool token_norm = options->norm == BSS_HEAD_NORM_TOKEN;
    const Smem lay = smem_layout(s.tokens, pieces, s.heads_per_block, 2, a.rot.first[3] > 0, token_norm);
    a.heads_per_block = s.heads_per_block;
    a.groups = s.groups;
    return launch(pick(false, pieces, pairing, options->norm, s.T), a, dim3((a.N + s.tokens - 1) / s.tokens, s.grid_y),
                  s.threads, lay.bytes, stream, "heads launch");
}

bss_status bss_heads_from_tokens_backward_workspace(int32_t H, const bss_mask_params* params, int32_t norm,
                                                    int64_t* bytes) {
    using namespace bss;
    clear_error();
    if (bytes == nullptr) return set_error(BSS_ERR_INVALID_ARG, "bytes is NULL");
    *bytes = 0;
    bss_status st = check_geometry(params, H);
    if (st != BSS_OK) return st;
    if ((st = check_norm(norm, H, params->head_dim)) != BSS_OK) return st;
    if (norm == BSS_HEAD_NORM_NONE) return BSS_OK;
    const Shape s = shape_of(H, params->head_dim / 8, norm, kBackwardTokens);
    const int64_t width = norm == BSS_HEAD_NORM_TOKEN ? static_cast<int64_t>(H) * params->head_dim : params->head_dim;
    *bytes = static_cast<int64_t>(backward_grid(s, static_cast<uint32_t>(params->F) * params->Hs * params->Ws)) *
             s.grid_y * 2 * width * 4;
    return BSS_OK;
}

bss_status bss_heads_from_tokens_backward(const void* dQh, const void* dKh, const void* dVh,
                                          const bss_token_tensor* q, const bss_token_tensor* k,
                                          const bss_token_tensor* dq, const bss_token_tensor* dk,
                                          const bss_token_tensor* dv, float* dq_weight, float* dk_weight,
                                          const uint8_t* head_is_temporal, int32_t H, const bss_mask_params* params,
                                          const bss_heads_options* options, void* workspace,
                                          int64_t workspace_bytes, cudaStream_t stream) {
    using namespace bss;
    clear_error();
    bss_status st = check_geometry(params, H);
    if (st != BSS_OK) return st;
    HeadsArgs a;
    memset(&a, 0, sizeof(a));
    int pairing = 0;
    if ((st = set_options(options, params, H, &a, &pairing)) != BSS_OK) return st;
    set_geometry(params, H, head_is_temporal, &a);
    const int d = params->head_dim;
    const int32_t norm = options->norm;
    const void* grad[3] = {dQh, dKh, dVh};
    const bss_token_tensor* x[2] = {q, k};
    const bss_token_tensor* out[3] = {dq, dk, dv};
    float* dweight[2] = {dq_weight, dk_weight};
    const char* names[3] = {"dq", "dk", "dv"};
    const char* xnames[2] = {"q", "k"};
    Region rin[5], rout[3];
    bool has_x[2] = {false, false};
    int given = 0;
    for (int i = 0; i < 3; ++i) {
        const bool has = grad[i] != nullptr;
        if (has != (out[i] != nullptr && out[i]->data != nullptr))
            return set_error(BSS_ERR_INVALID_ARG, "%s and its gradient must be given together", names[i]);
        if (i < 2 && dweight[i] != nullptr && (!has || norm == BSS_HEAD_NORM_NONE))
            return set_error(BSS_ERR_INVALID_ARG, "a weight gradient needs a norm and the tensor's gradient");
        if (!has) continue;
        ++given;
        if (!is_aligned(grad[i], 16)) return set_error(BSS_ERR_INVALID_ARG, "gradients must be 16-byte aligned");
        rin[i] = region_2d(grad[i], 1, 0, static_cast<int64_t>(H) * a.N * d, 2);
        if ((st = check_tokens(out[i], names[i], a.N, H, d, &rout[i])) != BSS_OK) return st;
        if (rout[i].self_overlap) return set_error(BSS_ERR_INVALID_ARG, "%s overlaps itself", names[i]);
        a.in[i] = static_cast<const __nv_bfloat16*>(grad[i]);
        a.out[i] = static_cast<__nv_bfloat16*>(out[i]->data);
        a.ts[i] = a.N > 1 ? out[i]->token_stride : 0;
        a.hs[i] = H > 1 ? out[i]->head_stride : 0;
        if (i == 2 || norm == BSS_HEAD_NORM_NONE) continue;
        if (x[i] == nullptr || x[i]->data == nullptr)
            return set_error(BSS_ERR_INVALID_ARG, "the norm's gradient needs %s", xnames[i]);
        if ((st = check_tokens(x[i], xnames[i], a.N, H, d, &rin[3 + i])) != BSS_OK) return st;
        has_x[i] = true;
        a.x[i] = static_cast<const __nv_bfloat16*>(x[i]->data);
        a.xts[i] = a.N > 1 ? x[i]->token_stride : 0;
        a.xhs[i] = H > 1 ? x[i]->head_stride : 0;
    }
    if (given == 0) return set_error(BSS_ERR_INVALID_ARG, "no tensor given");
    for (int i = 0; i < 3; ++i) {
        if (a.out[i] == nullptr) continue;
        for (int j = 0; j < 5; ++j)
            if ((j < 3 ? a.in[j] != nullptr : has_x[j - 3]) && !disjoint(rout[i], rin[j]))
                return set_error(BSS_ERR_INVALID_ARG, "an output overlaps an input");
        for (int j = 0; j < i; ++j)
            if (a.out[j] != nullptr && !disjoint(rout[i], rout[j]))
                return set_error(BSS_ERR_INVALID_ARG, "outputs overlap");
    }
    const int pieces = d / 8;
    const Shape s = shape_of(H, pieces, norm, kBackwardTokens);
    const bool token_norm = norm == BSS_HEAD_NORM_TOKEN;
    const Smem lay = smem_layout(s.tokens, pieces, s.heads_per_block, 4, a.rot.first[3] > 0, token_norm);
    a.heads_per_block = s.heads_per_block;
    a.groups = s.groups;
    a.want_dweight = dq_weight != nullptr || dk_weight != nullptr;
    const uint32_t grid_x = backward_grid(s, a.N);
    const int width = token_norm ? H * d : d;
    int smem = 2 * lay.bytes;
    if (a.want_dweight) {
        if (!is_aligned(dq_weight, 16) || !is_aligned(dk_weight, 16))
            return set_error(BSS_ERR_INVALID_ARG, "weight gradients must be 16-byte aligned");
        const int64_t need = static_cast<int64_t>(grid_x) * s.grid_y * 2 * width * 4;
        if (workspace == nullptr || !is_aligned(workspace, 16) || workspace_bytes < need)
            return set_error(BSS_ERR_INVALID_ARG, "the workspace must be 16-byte aligned and hold %lld bytes",
                             static_cast<long long>(need));
        a.partial = static_cast<float*>(workspace);
        if (smem < 2 * s.threads * 32) smem = 2 * s.threads * 32;
    }
    st = launch(pick(true, pieces, pairing, norm, s.T), a, dim3(grid_x, s.grid_y), s.threads, smem, stream,
                "heads backward launch");
    if (st != BSS_OK || !a.want_dweight) return st;
    heads_reduce_kernel<<<(2 * width + 31) / 32, 256, 0, stream>>>(a.partial, static_cast<int>(grid_x * s.grid_y), width,
                                                                  dq_weight, dk_weight);
    return cuda_check(cudaGetLastError(), "weight gradient launch");
}

bss_status bss_attention_step_tokens(const bss_token_tensor* q, const bss_token_tensor* k,
                                     const bss_token_tensor* v, void* O, float* lse, bss_tile_map map,
                                     const uint8_t* head_is_temporal, int32_t H, const bss_heads_options* options,
                                     void* Qh, void* Kh, void* Vh, cudaStream_t stream) {
    using namespace bss;
    clear_error();
    if (!tile_map_is_live(map)) return set_error(BSS_ERR_INVALID_ARG, "invalid or destroyed tile map");
    if (O == nullptr || Qh == nullptr || Kh == nullptr || Vh == nullptr)
        return set_error(BSS_ERR_INVALID_ARG, "NULL tensor");
    const uint8_t* permuted = map->p.temporal_permuted ? head_is_temporal : nullptr;
    const bss_status st = bss_heads_from_tokens(q, k, v, Qh, Kh, Vh, permuted, H, &map->p, options, stream);
    if (st != BSS_OK) return st;
    if (permuted == nullptr)
        return bss_sparse_attention(Qh, Kh, Vh, O, lse, map, head_is_temporal, H, 0.0f, stream);
    return bss_sparse_attention_split(Qh, Kh, Vh, O, Qh, Kh, Vh, nullptr, lse, map, head_is_temporal, H, 0.0f, stream);
}

}  // extern "C"
