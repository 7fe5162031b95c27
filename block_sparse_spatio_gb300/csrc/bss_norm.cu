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
// squares.  Every thread copies its own vectors of the next rows into its own
// slots of shared memory (cp.async) while it works on this one, so loads stay in
// flight without holding registers.
//
// Measured (75,600 x 1,280, GB300, share of the measured copy bandwidth): forward
// bf16 128 us (89%; 302,400 rows 92 to 93%), float stream with both norms 181 us (95%);
// backward bf16 182 us (94%), 302,400 rows with both norms RMS 713 us (96%).
#include <cstring>
#include <type_traits>

#include "bss_rows.cuh"

namespace bss {
namespace {

constexpr int kMaxChannels = 8192;
constexpr int64_t kMaxStride = int64_t(1) << 28;  // elements between rows: a row's offset is one 32 x 32 bit product
// A group's rows are shared by at most one block for every so many of them (5 rows: two
// blocks of 3 and 2; groups of fewer rows: a block each).
constexpr int kRowsPerChunk = 4;

// ---------------------------------------------------------------- shared memory
__device__ __forceinline__ uint4 lds128(uint32_t at) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at));
    return v;
}

__device__ __forceinline__ void sts128(uint32_t at, const uint4& v) {
    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

__device__ __forceinline__ uint2 lds64(uint32_t at) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(at));
    return v;
}

__device__ __forceinline__ V8 floats_of(const uint4& a, const uint4& b) {
    V8 v;
    v.p[0] = make_float2(__uint_as_float(a.x), __uint_as_float(a.y));
    v.p[1] = make_float2(__uint_as_float(a.z), __uint_as_float(a.w));
    v.p[2] = make_float2(__uint_as_float(b.x), __uint_as_float(b.y));
    v.p[3] = make_float2(__uint_as_float(b.z), __uint_as_float(b.w));
    return v;
}

__device__ __forceinline__ uint4 bits_of(const float2& a, const float2& b) {
    return make_uint4(__float_as_uint(a.x), __float_as_uint(a.y), __float_as_uint(b.x), __float_as_uint(b.y));
}

// The 8 channels of a thread's vector.  Rows of bf16 alone: 8 neighbouring
// channels, 16 bytes.  With a float stream (SPLIT): two runs of 4, 128 channels
// apart, so that 32 lanes read and write whole sectors of every tensor: 16 bytes
// a lane of float, 8 of bf16 (8 neighbouring float channels would be two loads of
// 16 bytes at a stride of 32, each sector asked for twice).
template <bool SPLIT>
__device__ __forceinline__ int channel_at(int warp_of_row, int half) {
    const int lane = threadIdx.x & 31;
    return SPLIT ? warp_of_row * 256 + half * 128 + lane * 4 : (warp_of_row * 32 + lane) * 8 + half * 4;
}

// A vector in shared memory: `lanes` threads' pieces side by side, a piece of
// 16 (or 8) bytes of thread `idx` at region + idx * size, its second half after
// all the first ones.
template <typename T, bool SPLIT>
__device__ __forceinline__ void fetch_vector(uint32_t region, int idx, int lanes, const T* from, bool live0, bool live1) {
    if constexpr (!SPLIT) {
        if (live0) cp_async_16(region + idx * 16, from);
    } else if constexpr (sizeof(T) == 4) {
        if (live0) cp_async_16(region + idx * 16, from);
        if (live1) cp_async_16(region + (lanes + idx) * 16, from + 128);
    } else {
        if (live0)
            asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(region + idx * 8), "l"(from) : "memory");
        if (live1)
            asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(region + (lanes + idx) * 8), "l"(from + 128)
                         : "memory");
    }
}

template <typename T, bool SPLIT>
__device__ __forceinline__ V8 lds_vector(uint32_t region, int idx, int lanes) {
    if constexpr (!SPLIT) {
        return unpack_bf16<false>(lds128(region + idx * 16));
    } else if constexpr (sizeof(T) == 4) {
        return floats_of(lds128(region + idx * 16), lds128(region + (lanes + idx) * 16));
    } else {
        const uint2 a = lds64(region + idx * 8), b = lds64(region + (lanes + idx) * 8);
        return unpack_bf16<false>(make_uint4(a.x, a.y, b.x, b.y));
    }
}

__device__ __forceinline__ void st_row8(void* p, uint32_t a, uint32_t b) {
    asm volatile("st.global.cs.v2.u32 [%0], {%1,%2};" ::"l"(p), "r"(a), "r"(b) : "memory");
}

template <typename T, bool SPLIT>
__device__ __forceinline__ void store_vector(T* to, const V8& v, bool live0, bool live1) {
    if constexpr (!SPLIT) {
        if (live0) st_row(to, pack_bf16<false>(v));
    } else if constexpr (sizeof(T) == 4) {
        if (live0) st_row(to, bits_of(v.p[0], v.p[1]));
        if (live1) st_row(to + 128, bits_of(v.p[2], v.p[3]));
    } else {
        if (live0) st_row8(to, pack2(v.p[0].x, v.p[0].y), pack2(v.p[1].x, v.p[1].y));
        if (live1) st_row8(to + 128, pack2(v.p[2].x, v.p[2].y), pack2(v.p[3].x, v.p[3].y));
    }
}

template <typename T>
__device__ __forceinline__ T* at_row(T* base, uint32_t row, uint32_t stride_bytes) {
    using Byte = std::conditional_t<std::is_const_v<T>, const char, char>;
    return reinterpret_cast<T*>(reinterpret_cast<Byte*>(base) + static_cast<uint64_t>(row) * stride_bytes);
}

template <typename T>
__device__ __forceinline__ uint32_t bytes_of(int64_t stride) {
    return static_cast<uint32_t>(stride * static_cast<int64_t>(sizeof(T)));
}

__device__ __forceinline__ V8 zeros() { return floats_of(make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)); }

// Zeros in the half that lies past the row.
__device__ __forceinline__ void keep_live(V8& v, bool live0, bool live1) {
    if (!live0) v.p[0] = v.p[1] = f2(0.0f);
    if (!live1) v.p[2] = v.p[3] = f2(0.0f);
}

// Four parameters.
__device__ __forceinline__ void param4(const void* p, int64_t at, int dtype, float2& a, float2& b) {
    if (dtype == BSS_DTYPE_F32) {
        const float4 v = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(p) + at));
        a = make_float2(v.x, v.y), b = make_float2(v.z, v.w);
    } else {
        const uint2 v = __ldg(reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(p) + at));
        a = make_float2(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xFFFF0000u));
        b = make_float2(__uint_as_float(v.y << 16), __uint_as_float(v.y & 0xFFFF0000u));
    }
}

// Those of the channels c0 .. c0 + 3 and c1 .. c1 + 3.
__device__ __forceinline__ V8 param_vector(const void* p, int64_t row, int c0, int c1, int dtype) {
    V8 v;
    param4(p, row + c0, dtype, v.p[0], v.p[1]);
    param4(p, row + c1, dtype, v.p[2], v.p[3]);
    return v;
}

__device__ __forceinline__ V8 add8(const V8& a, const V8& b) {
    V8 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r.p[i] = __fadd2_rn(a.p[i], b.p[i]);
    return r;
}

__device__ __forceinline__ V8 add8(const V8& a, float b) {
    V8 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r.p[i] = __fadd2_rn(a.p[i], f2(b));
    return r;
}

__device__ __forceinline__ float sum8(const V8& a) {
    const float2 s = __fadd2_rn(__fadd2_rn(a.p[0], a.p[1]), __fadd2_rn(a.p[2], a.p[3]));
    return s.x + s.y;
}

// ---------------------------------------------------------------- forward
// What multiplies and is added to the normed values of a group, folded:
//   0  gate * y_weight      1  weight * (1 + scale)      2  bias * (1 + scale) + shift
struct Folded {
    bool has[3];
};

struct ForwardArgs {
    bss_residual_norm_args a;
    Folded folded;
    int32_t folds;          // how many of them there are
    int64_t groups;         // of rows that share them
    int64_t chunks, chunk_rows;
    FastDiv by_rows;        // rows of a group
};

__device__ __forceinline__ V8 fold(const bss_residual_norm_args& a, int which, int64_t group, int c0, int c1) {
    V8 v = zeros();
    const int dt = a.param_dtype;
    if (which == 0) {
        v = a.gate != nullptr ? param_vector(a.gate, group * a.gate_stride, c0, c1, dt) : add8(v, 1.0f);
        if (a.y_weight != nullptr) v = mul(v, param_vector(a.y_weight, 0, c0, c1, dt));
        return v;
    }
    V8 m = add8(v, 1.0f);
    if (a.scale != nullptr) m = add8(param_vector(a.scale, group * a.scale_stride, c0, c1, dt), 1.0f);
    if (which == 1) return a.weight != nullptr ? mul(m, param_vector(a.weight, 0, c0, c1, dt)) : m;
    if (a.bias != nullptr) v = mul(m, param_vector(a.bias, 0, c0, c1, dt));
    return a.shift != nullptr ? add8(v, param_vector(a.shift, group * a.shift_stride, c0, c1, dt)) : v;
}

// Sum over the W warps that share a row; every thread gets it.  Each use between
// two barriers has W floats of its own.
template <int W>
__device__ __forceinline__ float row_sum(float v, float* buf) {
    v = lane_sum<32>(v);
    if (W == 1) return v;
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
    __syncthreads();
    v = buf[0];
#pragma unroll
    for (int i = 1; i < W; ++i) v += buf[i];
    return v;
}

template <typename TS, typename TB>
__host__ __device__ constexpr uint32_t forward_stage(int vpt) {
    return vpt * (sizeof(TS) + sizeof(TB)) * 8 * 32;
}

// W warps share a row, each thread holding up to VPT vectors of it in registers;
// with W = 1 a block takes 4 rows side by side.  A block covers one chunk of one
// group's rows, whose folded parameters it keeps in shared memory (STAGED); with
// few rows a group it reads them row by row.
template <typename TS, typename TB, int W, int VPT, bool STAGED>
__global__ void __launch_bounds__(W > 4 ? 32 * W : 128) norm_forward_kernel(const __grid_constant__ ForwardArgs g) {
    extern __shared__ __align__(16) float4 folded[];
    __shared__ float buf[2][4][W];
    const bss_residual_norm_args& a = g.a;
    constexpr bool kSplit = sizeof(TS) == 4;
    constexpr int kWarps = W > 4 ? W : 4, kRows = kWarps / W;
    constexpr uint32_t kStage = forward_stage<TS, TB>(VPT), kY = VPT * sizeof(TS) * 256;
    const int lane = threadIdx.x & 31, warp = W == 1 ? 0 : threadIdx.x >> 5;
    const int C = a.channels;
    const float inv = 1.0f / C;
    const int64_t first_group = blockIdx.x / static_cast<uint32_t>(g.chunks), chunk = blockIdx.x - first_group * g.chunks;
    const int64_t group_rows = STAGED ? a.rows_per_group : a.rows;
    const int64_t begin = first_group * group_rows + chunk * g.chunk_rows;
    int64_t end = begin + g.chunk_rows;
    if (end > (first_group + 1) * group_rows) end = (first_group + 1) * group_rows;
    if (end > a.rows) end = a.rows;
    const uint32_t last = static_cast<uint32_t>(end);
    uint32_t row = static_cast<uint32_t>(begin) + threadIdx.x / 32 / W;
    const uint32_t r_bytes = bytes_of<TS>(a.r_stride), h_bytes = bytes_of<TB>(a.h_stride);

    // channels of vector i: c0 + i * 256 W and c1 + i * 256 W, four each
    const int c0 = channel_at<kSplit>(warp, 0), c1 = channel_at<kSplit>(warp, 1);
    auto live0 = [&](int i) { return c0 + i * 256 * W < C; };
    auto live1 = [&](int i) { return (kSplit ? c1 : c0) + i * 256 * W < C; };
    const uint32_t base = smem_u32(folded);
    const uint32_t slots = base + (STAGED ? g.folds * C * 4 : 0) + (threadIdx.x >> 5) * 2 * kStage;
    const TS* x = at_row(static_cast<const TS*>(a.x), row, bytes_of<TS>(a.x_stride)) + c0;
    const TB* y = at_row(static_cast<const TB*>(a.y), row, bytes_of<TB>(a.y_stride)) + c0;
    auto fetch = [&](bool exists, uint32_t to) {
        if (exists) {
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                fetch_vector<TS, kSplit>(to + i * sizeof(TS) * 256, lane, 32, x + i * 256 * W, live0(i), live1(i));
                if (a.y != nullptr)
                    fetch_vector<TB, kSplit>(to + kY + i * sizeof(TB) * 256, lane, 32, y + i * 256 * W, live0(i), live1(i));
            }
            x += kRows * a.x_stride;
            y += kRows * a.y_stride;
        }
        cp_async_commit();
    };
    fetch(row < last, slots);
    // folded parameters: by channel, or for neighbouring channels in two planes, so
    // that lanes read them without bank conflicts
    const uint32_t fold1 = base + (g.folded.has[0] ? C * 4 : 0);
    const uint32_t fold2 = fold1 + (g.folded.has[1] ? C * 4 : 0);
    auto fold_at = [&](int which, int c) -> uint32_t {
        const uint32_t at = which == 0 ? base : which == 1 ? fold1 : fold2;
        return kSplit ? at + c * 4 : at + (c & 4) * (C / 2) + (c >> 3) * 16;
    };
    if (STAGED && g.folds > 0) {
#pragma unroll
        for (int which = 0; which < 3; ++which) {
            if (!g.folded.has[which]) continue;
#pragma unroll 2
            for (int c = threadIdx.x * 8; c < C; c += blockDim.x * 8) {
                const V8 f = fold(a, which, first_group, c, c + 4);
                sts128(fold_at(which, c), bits_of(f.p[0], f.p[1]));
                sts128(fold_at(which, c + 4), bits_of(f.p[2], f.p[3]));
            }
        }
        __syncthreads();
    }
    // those of vector i; only called where it is live, a dead half takes the other's
    auto folded_of = [&](int which, int64_t group, int i) {
        const int lo = c0 + i * 256 * W, hi = live1(i) ? c1 + i * 256 * W : lo;
        if (!STAGED) return fold(a, which, group, lo, hi);
        return floats_of(lds128(fold_at(which, lo)), lds128(fold_at(which, hi)));
    };
    uint32_t now = slots, other = slots + kStage;
    int parity = 0;
    for (; row < last; row += kRows, parity ^= 1) {
        fetch(last - row > kRows, other);
        cp_async_wait_group<1>();
        const int64_t group = STAGED ? first_group : g.by_rows.div(row);
        V8 r[VPT];
        float ym = 0.0f, yrstd = 1.0f;
        if (a.y != nullptr && a.y_norm != BSS_NORM_NONE) {
            float s = 0.0f;
            if (a.y_norm == BSS_NORM_LAYER) {
#pragma unroll
                for (int i = 0; i < VPT; ++i)
                    if (live0(i)) {
                        V8 v = lds_vector<TB, kSplit>(now + kY + i * sizeof(TB) * 256, lane, 32);
                        keep_live(v, true, live1(i));
                        s += sum8(v);
                    }
                ym = row_sum<W>(s, buf[parity][0]) * inv;
            }
            s = 0.0f;
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                if (!live0(i)) continue;
                V8 v = add8(lds_vector<TB, kSplit>(now + kY + i * sizeof(TB) * 256, lane, 32), -ym);
                keep_live(v, true, live1(i));
                s += dot(v, v);
            }
            yrstd = rsqrtf(row_sum<W>(s, buf[parity][1]) * inv + a.eps);
            if (a.y_stats != nullptr && lane == 0 && warp == 0)
                *reinterpret_cast<float2*>(a.y_stats + 2 * static_cast<int64_t>(row)) = make_float2(ym, yrstd);
        }
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            r[i] = zeros();
            if (!live0(i)) continue;
            r[i] = lds_vector<TS, kSplit>(now + i * sizeof(TS) * 256, lane, 32);
            if (a.y != nullptr) {
                V8 t = lds_vector<TB, kSplit>(now + kY + i * sizeof(TB) * 256, lane, 32);
                if (a.y_norm != BSS_NORM_NONE) t = mul(add8(t, -ym), yrstd);
                if (g.folded.has[0]) t = mul(t, folded_of(0, group, i));
                r[i] = fma8(r[i], a.residual_scale, t);
                if (a.r != nullptr)
                    store_vector<TS, kSplit>(at_row(static_cast<TS*>(a.r), row, r_bytes) + c0 + i * 256 * W, r[i], true, live1(i));
            }
            keep_live(r[i], true, live1(i));
            s += sum8(r[i]);
        }
        const uint32_t t = now;
        now = other, other = t;
        if (a.h == nullptr) continue;
        float mean = 0.0f, rstd = 1.0f;
        if (a.norm != BSS_NORM_NONE) {
            if (a.norm == BSS_NORM_LAYER) mean = row_sum<W>(s, buf[parity][2]) * inv;
            s = 0.0f;
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                if (!live0(i)) continue;
                r[i] = add8(r[i], -mean);
                keep_live(r[i], true, live1(i));
                s += dot(r[i], r[i]);
            }
            rstd = rsqrtf(row_sum<W>(s, buf[parity][3]) * inv + a.eps);
            if (a.stats != nullptr && lane == 0 && warp == 0)
                *reinterpret_cast<float2*>(a.stats + 2 * static_cast<int64_t>(row)) = make_float2(mean, rstd);
        }
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            if (!live0(i)) continue;
            V8 n = mul(r[i], rstd);
            if (g.folded.has[1]) n = mul(n, folded_of(1, group, i));
            if (g.folded.has[2]) n = add8(n, folded_of(2, group, i));
            store_vector<TB, kSplit>(at_row(static_cast<TB*>(a.h), row, h_bytes) + c0 + i * 256 * W, n, true, live1(i));
        }
    }
    cp_async_wait_group<0>();
}

// ---------------------------------------------------------------- backward
// A thread owns 8 channels and walks over rows, T at a time, so the three column
// sums stay in its registers; `warps` warps share a row, several rows go side by
// side in a block when a row is short.  A block covers one chunk of one group's
// rows.
struct GradShape {
    int warps;        // per row
    int side;         // rows side by side
    int threads, T, stages, smem;
    int64_t groups, chunks, chunk_rows;  // chunks per group
};

struct GradArgs {
    bss_residual_norm_grads a;
    GradShape s;
    float* partial;   // [groups][chunks][3][channels]
    int want_sums;
};

// Shared memory of one stage: T rows of r, dr, dh, y, a column of 16-byte pieces a
// thread, and the rows' statistics, 16 bytes a row: a copy a thread, or with a norm
// of y, where shared memory is busier, a copy a warp (302,400 x 1,280 RMS both
// sides: 713 us against 848; without a norm of y 711 against 686).
__host__ __device__ constexpr uint32_t grad_stage(int T, int stream_size, int branch_size, int threads, bool plain) {
    return static_cast<uint32_t>(T * (stream_size + branch_size) * threads * 16 + T * (plain ? threads : threads / 32) * 16);
}

// What is behind the two gradients:
//   PLAIN  no norm of y, one round of sums (mean t, mean t xh)
//   RMS2   both norms RMS: one round too, since z = u f with f = gate y_weight is
//          linear in mean(t xh):
//            sum z yh = sum f yh (dr + rstd t) - rstd mean(t xh) sum f yh xh
//   BOTH   any other norm of y: a second round for z
enum { PLAIN = 0, RMS2 = 1, BOTH = 2 };

// Sums of NV values over the row's warps; `buf` holds NV floats a warp of the block.
template <int NV>
__device__ __forceinline__ void shared_sums(float (&v)[NV], int warps, int warp0, float* buf) {
    const float s = scatter_sum<NV, 32>(v);
    if (scattered_writer<NV, 32>()) buf[(threadIdx.x >> 5) * NV + scattered_index<NV, 32>()] = s;
    if (warps == 1)
        __syncwarp();
    else
        __syncthreads();
#pragma unroll
    for (int i = 0; i < NV; ++i) v[i] = buf[warp0 * NV + i];
    for (int w = warp0 + 1; w < warp0 + warps; ++w) {
#pragma unroll
        for (int i = 0; i < NV; ++i) v[i] += buf[w * NV + i];
    }
}

template <typename TS, typename TB, int MODE, int T, int THREADS>
__global__ void __launch_bounds__(THREADS) norm_backward_kernel(const __grid_constant__ GradArgs g) {
    extern __shared__ __align__(16) float shared[];  // slots; at the end the column sums of the rows side by side
    __shared__ __align__(16) float buf[4][32 * (MODE == RMS2 ? 4 : 2) * T];
    const bss_residual_norm_grads& a = g.a;
    constexpr bool kSplit = sizeof(TS) == 4;
    constexpr int kS = sizeof(TS) / 2, kB = sizeof(TB) / 2, kPieces = 2 * (kS + kB);  // of a row
    const int side = (threadIdx.x >> 5) / g.s.warps;
    const int warp0 = side * g.s.warps;
    const int warp = (threadIdx.x >> 5) - warp0;
    const bool active = channel_at<kSplit>(warp, 0) < a.channels;
    const bool whole = kSplit ? channel_at<kSplit>(warp, 1) < a.channels : active;  // the second half too
    const int c = active ? channel_at<kSplit>(warp, 0) : 0;
    const int c1 = whole ? channel_at<kSplit>(warp, 1) : c;
    const int idx = threadIdx.x, lanes = blockDim.x;
    const float inv = 1.0f / a.channels;
    const int64_t group = blockIdx.x / static_cast<uint32_t>(g.s.chunks), chunk = blockIdx.x - group * g.s.chunks;
    const int64_t begin = group * a.rows_per_group + chunk * g.s.chunk_rows;
    int64_t end = begin + g.s.chunk_rows;
    if (end > (group + 1) * a.rows_per_group) end = (group + 1) * a.rows_per_group;
    if (end > a.rows) end = a.rows;
    // a chunk past its group's rows is empty
    const uint32_t first = static_cast<uint32_t>(begin < end ? begin : end), last = static_cast<uint32_t>(end);
    const uint32_t r_bytes = bytes_of<TS>(a.r_stride), dr_bytes = bytes_of<TS>(a.dr_stride);
    const uint32_t dh_bytes = bytes_of<TB>(a.dh_stride), y_bytes = bytes_of<TB>(a.y_stride);
    const uint32_t dx_bytes = bytes_of<TS>(a.dx_stride), dy_bytes = bytes_of<TB>(a.dy_stride);
    const bool stats = a.dh != nullptr && a.norm != BSS_NORM_NONE;
    constexpr bool ystats = MODE != PLAIN;

    // slot of piece k: a column of `threads` 16-byte pieces
    const uint32_t apart = blockDim.x * 16, stage_bytes = grad_stage(T, sizeof(TS), sizeof(TB), blockDim.x, MODE == PLAIN);
    const uint32_t slots = smem_u32(shared);
    const uint32_t stats_at = T * kPieces * apart + (MODE == PLAIN ? threadIdx.x : threadIdx.x >> 5) * (T * 16);
    const TS* r_in = static_cast<const TS*>(a.r) + c;
    const TS* dr_in = static_cast<const TS*>(a.dr) + c;
    const TB* dh_in = static_cast<const TB*>(a.dh) + c;
    const TB* y_in = static_cast<const TB*>(a.y) + c;
    auto fetch = [&](uint32_t row0, uint32_t to) {
#pragma unroll
        for (int t = 0; t < T; ++t) {
            const uint32_t row = row0 + t;
            if (!active || row >= last) continue;
            const uint32_t at = to + t * kPieces * apart;
            if (a.dh != nullptr) {
                fetch_vector<TS, kSplit>(at, idx, lanes, at_row(r_in, row, r_bytes), true, whole);
                fetch_vector<TB, kSplit>(at + (2 * kS) * apart, idx, lanes, at_row(dh_in, row, dh_bytes), true, whole);
            }
            if (a.dr != nullptr)
                fetch_vector<TS, kSplit>(at + kS * apart, idx, lanes, at_row(dr_in, row, dr_bytes), true, whole);
            if (a.y != nullptr)
                fetch_vector<TB, kSplit>(at + (2 * kS + kB) * apart, idx, lanes, at_row(y_in, row, y_bytes), true, whole);
        }
        if (MODE == PLAIN ? active : (threadIdx.x & 31) == 0) {
#pragma unroll
            for (int t = 0; t < T; ++t) {
                const uint32_t row = row0 + t, st = to + stats_at + t * 16;
                if (row >= last) continue;
                if (stats)
                    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(st), "l"(at_row(a.stats, row, 8)) : "memory");
                if (ystats)
                    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(st + 8), "l"(at_row(a.y_stats, row, 8))
                                 : "memory");
            }
        }
        cp_async_commit();
    };
    const uint32_t step = g.s.side * T;
    uint32_t mine = first + side * T;
    const bool ahead = g.s.stages > 1;  // the widest float rows have room for one stage only
    if (ahead) fetch(mine, slots);

    // (1 + scale) weight, gate y_weight; zeros past the row keep its lanes out of
    // the sums
    V8 m1 = zeros(), m2 = zeros();
    if (active) {
        m1 = add8(m1, 1.0f), m2 = add8(m2, 1.0f);
        const int dt = a.param_dtype;
        if (a.scale != nullptr) m1 = add8(m1, param_vector(a.scale, group * a.scale_stride, c, c1, dt));
        if (a.weight != nullptr) m1 = mul(m1, param_vector(a.weight, 0, c, c1, dt));
        if (a.gate != nullptr) m2 = param_vector(a.gate, group * a.gate_stride, c, c1, dt);
        if (a.y_weight != nullptr) m2 = mul(m2, param_vector(a.y_weight, 0, c, c1, dt));
        keep_live(m1, true, whole);
        keep_live(m2, true, whole);
    }
    V8 sa = zeros(), sb = zeros(), sc = zeros();
    int stage = 0, turn = 0;
    for (uint32_t row0 = first; row0 < last; row0 += step, mine += step, turn ^= 2) {
        if (MODE != PLAIN) __syncwarp();  // every lane has read the statistics in the slots to be filled
        if (ahead) {
            fetch(mine + step, slots + (stage ^ 1) * stage_bytes);
            cp_async_wait_group<1>();
        } else {
            fetch(mine, slots);
            cp_async_wait_group<0>();
        }
        if (MODE != PLAIN) __syncwarp();  // lane 0's copies of the statistics
        const uint32_t now = slots + stage * stage_bytes;
        stage ^= ahead ? 1 : 0;
        V8 xh[T], w[T];  // the normed stream; dr + rstd t
        float2 st[T], yst[T];
        constexpr int NV = MODE == RMS2 ? 4 : 2;
        float sums[NV * T];
#pragma unroll
        for (int t = 0; t < T; ++t) {
            const uint32_t at = now + t * kPieces * apart;
            const bool live = active && mine + t < last;
            xh[t] = w[t] = zeros();
            st[t] = yst[t] = make_float2(0.0f, 1.0f);
#pragma unroll
            for (int k = 0; k < NV; ++k) sums[NV * t + k] = 0.0f;
            if (!live) continue;
            const uint4 q = lds128(now + stats_at + t * 16);
            if (stats) st[t] = make_float2(__uint_as_float(q.x), __uint_as_float(q.y));
            if (ystats) yst[t] = make_float2(__uint_as_float(q.z), __uint_as_float(q.w));
            if (a.dr != nullptr) w[t] = lds_vector<TS, kSplit>(at + kS * apart, idx, lanes);
            if (a.dh != nullptr) {
                xh[t] = mul(add8(lds_vector<TS, kSplit>(at, idx, lanes), -st[t].x), st[t].y);
                V8 dh = lds_vector<TB, kSplit>(at + (2 * kS) * apart, idx, lanes);
                if (kSplit) keep_live(xh[t], true, whole), keep_live(dh, true, whole);
                const V8 tt = mul(dh, m1);
                sa = fma8(dh, xh[t], sa);
                sb = add8(sb, dh);
                w[t] = fma8(tt, st[t].y, w[t]);
                if (MODE != RMS2) sums[NV * t] = sum8(tt);
                sums[NV * t + 1] = dot(tt, xh[t]);
            }
            if (kSplit) keep_live(w[t], true, whole);
            if constexpr (MODE == RMS2) {
                V8 f = mul(mul(lds_vector<TB, kSplit>(at + (2 * kS + kB) * apart, idx, lanes), yst[t].y), m2);
                if (kSplit) keep_live(f, true, whole);
                sums[NV * t + 2] = dot(f, w[t]);
                sums[NV * t + 3] = dot(f, xh[t]);
            }
        }
        if (stats) shared_sums<NV * T>(sums, g.s.warps, warp0, buf[turn]);
        float zs[2 * T];
        V8 z[T];
#pragma unroll
        for (int t = 0; t < T; ++t) {
            const uint32_t at = now + t * kPieces * apart;
            const bool live = active && mine + t < last;
            const float mean1 = a.norm == BSS_NORM_LAYER ? sums[NV * t] * inv : 0.0f;
            const float mean2 = a.norm != BSS_NORM_NONE ? sums[NV * t + 1] * inv : 0.0f;
            V8 u = w[t];  // without a norm it is that: not 0 times an infinity of r more
            if (MODE == RMS2 || a.norm != BSS_NORM_NONE) u = fma8(xh[t], -st[t].y * mean2, u);
            if (a.norm == BSS_NORM_LAYER) u = add8(u, -st[t].y * mean1);
            if (live)
                store_vector<TS, kSplit>(at_row(static_cast<TS*>(a.dx) + c, mine + t, dx_bytes), mul(u, a.residual_scale), true,
                                         whole);
            z[t] = zeros();
            zs[2 * t] = zs[2 * t + 1] = 0.0f;
            if (a.dy == nullptr || !live) continue;
            V8 yh = mul(add8(lds_vector<TB, kSplit>(at + (2 * kS + kB) * apart, idx, lanes), -yst[t].x), yst[t].y);
            if (kSplit) keep_live(u, true, whole), keep_live(yh, true, whole);
            sc = fma8(u, yh, sc);
            z[t] = mul(u, m2);
            if constexpr (MODE == BOTH) {
                zs[2 * t] = sum8(z[t]);
                zs[2 * t + 1] = dot(z[t], yh);
            } else {
                if constexpr (MODE == RMS2)
                    z[t] = mul(fma8(yh, -inv * (sums[NV * t + 2] - st[t].y * mean2 * sums[NV * t + 3]), z[t]), yst[t].y);
                store_vector<TB, kSplit>(at_row(static_cast<TB*>(a.dy) + c, mine + t, dy_bytes), z[t], true, whole);
            }
        }
        if constexpr (MODE != BOTH) continue;
        if (MODE == BOTH) shared_sums<2 * T>(zs, g.s.warps, warp0, buf[turn + 1]);
#pragma unroll
        for (int t = 0; t < T; ++t) {
            if (!active || mine + t >= last) continue;
            {
                const uint32_t at = now + t * kPieces * apart;
                const float mean1 = a.y_norm == BSS_NORM_LAYER ? zs[2 * t] * inv : 0.0f;
                const V8 yh = mul(add8(lds_vector<TB, kSplit>(at + (2 * kS + kB) * apart, idx, lanes), -yst[t].x), yst[t].y);
                z[t] = mul(fma8(yh, -zs[2 * t + 1] * inv, add8(z[t], -mean1)), yst[t].y);
            }
            store_vector<TB, kSplit>(at_row(static_cast<TB*>(a.dy) + c, mine + t, dy_bytes), z[t], true, whole);
        }
    }
    cp_async_wait_group<0>();
    if (!g.want_sums) return;
    // the rows side by side, in order
    const int C = a.channels;
    float* dst = g.partial + static_cast<int64_t>(blockIdx.x) * 3 * C;
    const V8* sums3[3] = {&sa, &sb, &sc};
    if (g.s.side > 1) __syncthreads();
#pragma unroll
    for (int q = 0; q < 3; ++q) {
        if (!active) continue;
        float* at = g.s.side > 1 ? shared + (side * 3 + q) * C : dst + q * C;
        *reinterpret_cast<uint4*>(at + c) = bits_of(sums3[q]->p[0], sums3[q]->p[1]);
        if (whole) *reinterpret_cast<uint4*>(at + c1) = bits_of(sums3[q]->p[2], sums3[q]->p[3]);
    }
    if (g.s.side == 1) return;
    __syncthreads();
    for (int e = threadIdx.x; e < 3 * C; e += blockDim.x) {
        float s = 0.0f;
        for (int k = 0; k < g.s.side; ++k) s += shared[k * 3 * C + e];
        dst[e] = s;
    }
}

// One group's column sums over its chunks (in order within a lane, then the lanes
// in order; a block is 32 columns wide and has a lane per warp) and the
// modulations' gradients.  With one group the weights' gradients too; else the
// sums are kept in the group's first chunk for norm_weights_kernel.
__global__ void __launch_bounds__(1024) norm_groups_kernel(const __grid_constant__ GradArgs g) {
    __shared__ float part[3][32][33];
    const bss_residual_norm_grads& a = g.a;
    const int C = a.channels, col = threadIdx.x % 32, lane = threadIdx.x / 32, lanes = blockDim.x / 32;
    const int c = blockIdx.x * 32 + col;
    cudaGridDependencySynchronize();
    for (int64_t group = blockIdx.y; group < g.s.groups; group += gridDim.y) {
        float* base = g.partial + group * g.s.chunks * 3 * C;
        float s[3] = {0.0f, 0.0f, 0.0f};
        if (c < C) {
#pragma unroll 4
            for (int64_t k = lane; k < g.s.chunks; k += lanes)
#pragma unroll
                for (int q = 0; q < 3; ++q) s[q] += base[(k * 3 + q) * C + c];
        }
#pragma unroll
        for (int q = 0; q < 3; ++q) part[q][lane][col] = s[q];
        __syncthreads();
        if (lane == 0 && c < C) {
#pragma unroll
            for (int q = 0; q < 3; ++q) {
                s[q] = 0.0f;
                for (int k = 0; k < lanes; ++k) s[q] += part[q][k][col];
            }
            const float w = a.weight != nullptr ? load_param(a.weight, c, a.param_dtype) : 1.0f;
            const float b = a.bias != nullptr ? load_param(a.bias, c, a.param_dtype) : 0.0f;
            const float wy = a.y_weight != nullptr ? load_param(a.y_weight, c, a.param_dtype) : 1.0f;
            if (a.dscale != nullptr) a.dscale[group * C + c] = fmaf(w, s[0], b * s[1]);
            if (a.dshift != nullptr) a.dshift[group * C + c] = s[1];
            if (a.dgate != nullptr) a.dgate[group * C + c] = wy * s[2];
            if (g.s.groups > 1) {
#pragma unroll
                for (int q = 0; q < 3; ++q) base[q * C + c] = s[q];
            } else {
                const float m = a.scale != nullptr ? 1.0f + load_param(a.scale, c, a.param_dtype) : 1.0f;
                const float gt = a.gate != nullptr ? load_param(a.gate, c, a.param_dtype) : 1.0f;
                if (a.dweight != nullptr) a.dweight[c] = m * s[0];
                if (a.dbias != nullptr) a.dbias[c] = m * s[1];
                if (a.dy_weight != nullptr) a.dy_weight[c] = gt * s[2];
            }
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
    cudaGridDependencySynchronize();
    if (c < C) {
#pragma unroll 2
        for (int64_t group = lane; group < g.s.groups; group += 8) {
            const float* base = g.partial + group * g.s.chunks * 3 * C;
            const float m = a.scale != nullptr ? 1.0f + load_param(a.scale, group * a.scale_stride + c, a.param_dtype) : 1.0f;
            const float gt = a.gate != nullptr ? load_param(a.gate, group * a.gate_stride + c, a.param_dtype) : 1.0f;
            s[0] = fmaf(m, base[c], s[0]);
            s[1] = fmaf(m, base[C + c], s[1]);
            s[2] = fmaf(gt, base[2 * C + c], s[2]);
        }
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
    if (rows > 1 && (stride % 8 != 0 || stride < 0 || stride > kMaxStride))
        return set_error(BSS_ERR_INVALID_ARG, "%s: the row stride must be a multiple of 8 elements, 0 .. 2^28", name);
    *r = region_2d(p, rows, stride, channels, esize(dtype));
    if (output && r->self_overlap) return set_error(BSS_ERR_INVALID_ARG, "%s: rows overlap", name);
    return BSS_OK;
}

bss_status check_param(const void* p, const char* name, int64_t groups, int64_t stride, int32_t channels, int32_t dtype,
                       Region* r) {
    return check_rows(p, name, groups, stride, channels, dtype, false, r);
}

// Inputs may be named twice; an output must share no byte with any other tensor,
// but for the input that it may be written over (`over`, its place in the list; -1:
// none), and further row tensors that name the very same bytes as that one: a row is
// in its threads' hands before any of it is stored.  Parameters never are: other rows
// read them later.
struct Named {
    const void* p;
    Region r;
    bool output;
    int over;
};

// `rows`: the first so many are the call's row inputs.
bss_status check_overlaps(const Named* t, int n, int rows) {
    for (int i = 0; i < n; ++i) {
        if (t[i].p == nullptr || !t[i].output) continue;
        const Named* over = t[i].over < 0 ? nullptr : &t[t[i].over];
        const bool in_place = over != nullptr && over->p != nullptr && over->r.same_bytes(t[i].r) && !t[i].r.self_overlap;
        for (int j = 0; j < n; ++j) {
            if (j == i || t[j].p == nullptr || (t[j].output && j < i)) continue;
            if (in_place && j < rows && t[j].r.same_bytes(t[i].r) && !t[j].r.self_overlap) continue;
            if (!disjoint(t[i].r, t[j].r)) return set_error(BSS_ERR_INVALID_ARG, "an output overlaps another tensor");
        }
    }
    return BSS_OK;
}

// Rows a group must have for its folded parameters to be staged (75,600 x 1,280:
// groups of 8 rows 172 us staged, 286 read row by row; 302,400 x 256: groups of 4
// 200 and 181, of 16 111 and 139).
constexpr int64_t kStagedRows = 8;
// Waves of blocks (75,600 x 1,280, modulations a frame / RMS on both sides: one
// wave 142 / 197 us, two 131 / 189, four 128 / 182, eight 130 / 181).
constexpr int kForwardWaves = 4;

template <typename TS, typename TB, int W, int VPT, bool STAGED>
bss_status launch_forward(ForwardArgs g, cudaStream_t stream) {
    constexpr int kWarps = W > 4 ? W : 4, kRows = kWarps / W;
    const void* kernel = reinterpret_cast<const void*>(norm_forward_kernel<TS, TB, W, VPT, STAGED>);
    const int smem = (STAGED ? g.folds * g.a.channels * 4 : 0) +
                     kWarps * 2 * static_cast<int>(forward_stage<TS, TB>(VPT));
    int resident = 1;
    const bss_status st = resident_blocks(kernel, 32 * kWarps, smem, &resident);
    if (st != BSS_OK) return st;
    // a few waves of blocks, so that SMs that finish early take more; a block keeps
    // to one group
    const int64_t group_rows = STAGED ? g.a.rows_per_group : g.a.rows;
    g.groups = (g.a.rows + group_rows - 1) / group_rows;
    int64_t blocks = static_cast<int64_t>(kForwardWaves) * resident * num_sms() / g.groups;
    if (blocks < 1) blocks = 1;
    g.chunk_rows = (group_rows + blocks - 1) / blocks;
    g.chunk_rows = (g.chunk_rows + kRows - 1) / kRows * kRows;
    g.chunks = (group_rows + g.chunk_rows - 1) / g.chunk_rows;
    norm_forward_kernel<TS, TB, W, VPT, STAGED>
        <<<static_cast<unsigned>(g.groups * g.chunks), 32 * kWarps, smem, stream>>>(g);
    return cuda_check(cudaGetLastError(), "residual norm launch");
}

template <typename TS, typename TB, bool STAGED>
bss_status forward_width(const ForwardArgs& g, cudaStream_t stream) {
    // a warp alone needs no barrier and holds up to 5 vectors a lane (1280
    // channels); longer rows take 4 or 8 warps
    const int vecs = g.a.channels / 8;
    if (vecs <= 32) return launch_forward<TS, TB, 1, 1, STAGED>(g, stream);
    if (vecs <= 64) return launch_forward<TS, TB, 1, 2, STAGED>(g, stream);
    if (vecs <= 96) return launch_forward<TS, TB, 1, 3, STAGED>(g, stream);
    if (vecs <= 160) return launch_forward<TS, TB, 1, 5, STAGED>(g, stream);
    if (vecs <= 384) return launch_forward<TS, TB, 4, 3, STAGED>(g, stream);
    return launch_forward<TS, TB, 8, 4, STAGED>(g, stream);
}

template <typename TS, typename TB>
bss_status forward_of(const bss_residual_norm_args& a, cudaStream_t stream) {
    ForwardArgs g;
    memset(&g, 0, sizeof(g));
    g.a = a;
    // nothing that differs between groups: one group holds the rows
    if (a.gate == nullptr && a.scale == nullptr && a.shift == nullptr) g.a.rows_per_group = a.rows;
    g.by_rows = FastDiv(static_cast<uint32_t>(g.a.rows_per_group));
    g.folded.has[0] = a.gate != nullptr || a.y_weight != nullptr;
    g.folded.has[1] = a.scale != nullptr || a.weight != nullptr;
    g.folded.has[2] = a.shift != nullptr || a.bias != nullptr;
    for (bool has : g.folded.has) g.folds += has;
    return g.a.rows_per_group >= kStagedRows || g.a.rows_per_group == a.rows ? forward_width<TS, TB, true>(g, stream)
                                                                             : forward_width<TS, TB, false>(g, stream);
}

bool wants_sums(const bss_residual_norm_grads& a) {
    return a.dgate || a.dscale || a.dshift || a.dweight || a.dbias || a.dy_weight;
}

// Whether rows of different groups differ at all (else one group holds them).
bool grouped(const bss_residual_norm_grads& a) {
    return a.gate || a.scale || a.dgate || a.dscale || a.dshift;
}

bool norms_branch(const bss_residual_norm_grads& a) { return a.y != nullptr && a.y_norm != BSS_NORM_NONE; }

GradShape grad_shape(const bss_residual_norm_grads& a) {
    GradShape s;
    s.warps = (a.channels / 8 + 31) / 32;
    s.side = s.warps >= 4 ? 1 : 4 / s.warps;
    s.threads = s.warps * s.side * 32;
    s.T = s.threads <= 512 ? 2 : 1;
    const int stage = static_cast<int>(
        grad_stage(s.T, esize(a.stream_dtype), esize(a.branch_dtype), s.threads, !norms_branch(a)));
    s.stages = 2 * stage <= 224 * 1024 ? 2 : 1;
    s.smem = s.stages * stage;
    if (s.side > 1 && s.smem < s.side * 3 * a.channels * 4) s.smem = s.side * 3 * a.channels * 4;
    const int64_t per_group = !grouped(a) || a.rows_per_group > a.rows ? a.rows : a.rows_per_group;
    s.groups = (a.rows + per_group - 1) / per_group;
    // one wave of blocks: 16 warps an SM at 128 registers a thread, or what the
    // slots leave room for
    int per_sm = 512 / s.threads, by_smem = 224 * 1024 / (s.smem + 3 * 1024);
    per_sm = per_sm < by_smem ? per_sm : by_smem;
    int64_t most = (per_sm < 1 ? 1 : per_sm) * static_cast<int64_t>(num_sms()) / s.groups;
    if (most < 1) most = 1;
    s.chunks = (per_group + kRowsPerChunk - 1) / kRowsPerChunk;
    if (s.chunks > most) s.chunks = most;
    s.chunk_rows = (per_group + s.chunks - 1) / s.chunks;
    s.chunks = (per_group + s.chunk_rows - 1) / s.chunk_rows;
    return s;
}

int64_t grad_workspace(const bss_residual_norm_grads& a, const GradShape& s) {
    return wants_sums(a) ? s.groups * s.chunks * 3 * a.channels * 4 : 0;
}

template <typename TS, typename TB, int MODE, int T, int THREADS>
bss_status launch_backward_rows(const GradArgs& g, cudaStream_t stream) {
    int resident = 1;  // asked for the shared memory limit it sets
    const bss_status st = resident_blocks(reinterpret_cast<const void*>(norm_backward_kernel<TS, TB, MODE, T, THREADS>),
                                          g.s.threads, g.s.smem, &resident);
    if (st != BSS_OK) return st;
    norm_backward_kernel<TS, TB, MODE, T, THREADS>
        <<<static_cast<unsigned>(g.s.groups * g.s.chunks), g.s.threads, g.s.smem, stream>>>(g);
    return cuda_check(cudaGetLastError(), "residual norm backward launch");
}

template <typename TS, typename TB, int MODE>
bss_status launch_backward_mode(const GradArgs& g, cudaStream_t stream) {
    if (g.s.threads > 512) return launch_backward_rows<TS, TB, MODE, 1, 1024>(g, stream);
    return launch_backward_rows<TS, TB, MODE, 2, 512>(g, stream);
}

template <typename TS, typename TB>
bss_status launch_backward(const GradArgs& g, cudaStream_t stream) {
    if (!norms_branch(g.a)) return launch_backward_mode<TS, TB, PLAIN>(g, stream);
    if (g.a.dh != nullptr && g.a.norm == BSS_NORM_RMS && g.a.y_norm == BSS_NORM_RMS)
        return launch_backward_mode<TS, TB, RMS2>(g, stream);
    return launch_backward_mode<TS, TB, BOTH>(g, stream);
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
    if (a.rows_per_group > a.rows) a.rows_per_group = a.rows;
    const int64_t groups = (a.rows + a.rows_per_group - 1) / a.rows_per_group;
    Named t[12] = {{a.x, {}, false, -1},     {a.y, {}, false, -1},        {a.gate, {}, false, -1},
                   {a.scale, {}, false, -1}, {a.shift, {}, false, -1},    {a.weight, {}, false, -1},
                   {a.bias, {}, false, -1},  {a.y_weight, {}, false, -1}, {a.r, {}, true, 0},
                   {a.h, {}, true, 1},       {a.stats, {}, true, -1},     {a.y_stats, {}, true, -1}};
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
    if ((st = check_overlaps(t, 12, 2)) != BSS_OK) return st;
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
    if (a.rows_per_group > a.rows) a.rows_per_group = a.rows;
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
    Named t[20] = {{r, {}, false, -1},          {a.y, {}, false, -1},      {a.dr, {}, false, -1},
                   {a.dh, {}, false, -1},       {a.gate, {}, false, -1},   {a.scale, {}, false, -1},
                   {a.weight, {}, false, -1},   {a.bias, {}, false, -1},   {a.y_weight, {}, false, -1},
                   {stats, {}, false, -1},      {ystats, {}, false, -1},   {a.dx, {}, true, 2},
                   {a.dy, {}, true, 3},         {a.dgate, {}, true, -1},   {a.dscale, {}, true, -1},
                   {a.dshift, {}, true, -1},    {a.dweight, {}, true, -1}, {a.dbias, {}, true, -1},
                   {a.dy_weight, {}, true, -1}, {need > 0 ? a.workspace : nullptr, {}, true, -1}};
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
    if ((st = check_overlaps(t, 20, 4)) != BSS_OK) return st;
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
    const dim3 grid(cols, static_cast<unsigned>(g.s.groups < 4096 ? g.s.groups : 4096));
    st = launch_behind(norm_groups_kernel, grid, g.s.chunks > 64 ? 1024 : 256, stream, "modulation gradient launch", g);
    if (st != BSS_OK || g.s.groups == 1 || (a.dweight == nullptr && a.dbias == nullptr && a.dy_weight == nullptr)) return st;
    return launch_behind(norm_weights_kernel, dim3(cols), 256, stream, "weight gradient launch", g);
}

}  // extern "C"
