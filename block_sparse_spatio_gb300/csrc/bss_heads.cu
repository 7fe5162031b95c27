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
// A warp takes a whole token: lane l holds the 16-byte pieces (8 channels) l,
// l + 32, ... of its heads, so a piece's place in its head, and with it the angles
// of its rotary pairs, is the same for all the heads of Q and K that the lane
// holds, a token's coordinates are the same for the warp, and the norm's sums need
// no barrier.  Every lane copies its own pieces of the next token into its own
// slots of shared memory (cp.async) while it works on this one: loads stay in
// flight without holding registers.  Wide tokens are shared by several warps when
// the norm is over the token, else their heads go to several grid columns.
//
// Measured (75,600 tokens x 10 heads x 128, norm over the token, GB300): forward
// 188 us, backward 250 to 255 us, 91 and 89 to 91% of the measured copy bandwidth;
// what is left is mostly the ends of the launch (302,400 tokens: 92 to 93% and 94 to 96%).
#include <cstring>

#include "bss_rows.cuh"

namespace bss {
namespace {

constexpr int kMaxTokenWidth = 8192;  // H * head_dim of the norm over a token
constexpr int64_t kMaxTokenStride = int64_t(1) << 28;  // elements: a token's offset is one 32 x 32 bit product

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
    uint32_t ts[3], xts[2];       // bytes from token to token of the token-major tensors: in / out, x
    int64_t hs[3], xhs[2];        // elements from head to head
    const void* weight[2];
    int32_t weight_dtype;
    float eps, inv_width;         // 1 / channels of the norm's mean
    RotaryDev rot;
    const uint8_t* flags;
    FastDiv by_S, by_Ws;
    uint32_t N, F, S, H;
    int32_t pieces;               // 16-byte pieces of a head: 8 or 16
    int32_t heads_per_block;      // heads of a token that a block's grid column covers
    uint32_t span;                // tokens that a block walks over, one after the other
    float* partial;               // backward: [blocks][2][width], or NULL
};

// The pieces a lane holds: piece `piece` of the heads head0, head0 + step, ...
struct Lane {
    int piece, head0, step, count;  // count: how many of them exist
    uint32_t temporal;              // bit i: head i is permuted
};

// `warp`: which of the W warps of the token this is.
template <int W, int VPT>
__device__ __forceinline__ Lane lane_of(const HeadsArgs& a, int warp) {
    Lane l;
    const int lane = threadIdx.x & 31;
    const int per = 32 / a.pieces;  // heads side by side in a warp
    l.piece = lane & (a.pieces - 1);
    const int first = blockIdx.y * a.heads_per_block;
    const int last = min(static_cast<int>(a.H), first + a.heads_per_block);
    l.head0 = first + warp * per + lane / a.pieces;
    l.step = W * per;
    l.count = l.head0 < last ? min(VPT, (last - l.head0 + l.step - 1) / l.step) : 0;
    l.temporal = 0;
    return l;
}

template <int VPT>
__device__ __forceinline__ uint32_t temporal_heads(const HeadsArgs& a, const Lane& l) {
    uint32_t r = 0;
    if (a.flags != nullptr)
#pragma unroll
        for (int j = 0; j < VPT; ++j)
            if (j < l.count) r |= (a.flags[l.head0 + j * l.step] != 0 ? 1u : 0u) << j;
    return r;
}

struct Token {
    uint32_t f, h, w, temporal_row;
};

__device__ __forceinline__ Token token_of(const HeadsArgs& a, uint32_t n) {
    Token t;
    t.f = a.by_S.div(n);
    const uint32_t s = n - t.f * a.S;
    t.temporal_row = s * a.F + t.f;
    t.h = a.by_Ws.div(s);
    t.w = s - t.h * a.by_Ws.d;
    return t;
}

// Shared memory by 32-bit address, so that a piece's place is an offset in the
// instruction.
__device__ __forceinline__ uint4 lds128(uint32_t at) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at));
    return v;
}

__device__ __forceinline__ void sts128(uint32_t at, const uint4& v) {
    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// The angles of a token, one (cos, sin) a pair of a head, lie in the warp's slots:
// lane l copies those of pairs l and l + 32 (per pair the table entry of position
// 0, the table's row length and the axis), every lane reads those of its channels.
// Pairs past the rotated ones hold the identity throughout.
struct Angles {
    const float2* entry[2];
    uint32_t stride[2];
    uint32_t axes;   // 2 bits a pair; 3: not copied
};

__device__ __forceinline__ Angles angles_of(const HeadsArgs& a) {
    Angles r;
    r.axes = 0;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int p = (threadIdx.x & 31) + 32 * j;
        const int axis = p >= a.rot.first[3] ? 3 : p < a.rot.first[1] ? 0 : p < a.rot.first[2] ? 1 : 2;
        r.axes |= static_cast<uint32_t>(axis) << (2 * j);
        r.entry[j] = axis == 3 ? nullptr
                               : a.rot.table[axis] + static_cast<int64_t>(a.rot.offset[axis]) * a.rot.pairs[axis] +
                                     (p - a.rot.first[axis]);
        r.stride[j] = axis == 3 ? 0 : a.rot.pairs[axis] * 8;
    }
    return r;
}

constexpr uint32_t kAngleBytes = 64 * 8;  // of a warp's slots: 64 pairs at most

// `at`: the warp's angle slots, here and below.
__device__ __forceinline__ void clear_angles(const Angles& r, uint32_t at) {
#pragma unroll
    for (int j = 0; j < 2; ++j)
        if ((r.axes >> (2 * j) & 3u) == 3)
            asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(at + ((threadIdx.x & 31) + 32 * j) * 8), "f"(1.0f),
                         "f"(0.0f)
                         : "memory");
}

__device__ __forceinline__ void fetch_angles(const Angles& r, const Token& t, uint32_t at) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const uint32_t axis = r.axes >> (2 * j) & 3u;
        const uint32_t row = axis == 0 ? t.f : axis == 1 ? t.h : t.w;
        if (axis != 3)
            asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(at + ((threadIdx.x & 31) + 32 * j) * 8),
                         "l"(reinterpret_cast<const char*>(r.entry[j]) + static_cast<uint64_t>(row) * r.stride[j])
                         : "memory");
    }
}

// How a lane's channels pair up: 4 interleaved pairs, or for halves 8 pairs whose
// other channels lane `other` holds.
template <bool HALVES>
struct Pairs {
    uint32_t at;     // byte of the first one's angles
    int other;
    float sign;      // of the sine there
    uint32_t keep;   // bit j: pair j is not rotated (halves: none or all)
    bool partial;    // some channels of the head are not (the same for all lanes)
};

template <bool HALVES>
__device__ __forceinline__ Pairs<HALVES> pairs_of(const HeadsArgs& a, int piece) {
    Pairs<HALVES> r;
    r.partial = a.rot.first[3] < a.pieces * 4;
    r.sign = 1.0f;
    r.other = threadIdx.x & 31;
    r.keep = 0;
    if (HALVES) {
        const int half = a.rot.first[3] / 8;  // pieces per half
        const bool lower = piece < half, in = piece < 2 * half;
        const int other = in ? (lower ? piece + half : piece - half) : piece;
        r.other = (threadIdx.x & 31 & ~(a.pieces - 1)) | other;
        r.sign = lower ? -1.0f : 1.0f;
        r.at = in ? (lower ? piece : other) * 64 : 0;
        r.keep = in ? 0 : 0xFu;
    } else {
        r.at = piece * 32;
#pragma unroll
        for (int j = 0; j < 4; ++j) r.keep |= (piece * 4 + j >= a.rot.first[3] ? 1u : 0u) << j;
    }
    return r;
}

// One token's cosines and (signed, for halves and BACK) sines of a lane's pairs.
template <bool HALVES>
struct Turn {
    float2 c[HALVES ? 4 : 2], s[HALVES ? 4 : 2];
};

template <bool HALVES, bool BACK>
__device__ __forceinline__ Turn<HALVES> read_turn(const Pairs<HALVES>& pr, uint32_t at) {
    Turn<HALVES> r;
    const float sg = (HALVES ? pr.sign : 1.0f) * (BACK ? -1.0f : 1.0f);
#pragma unroll
    for (int j = 0; j < (HALVES ? 4 : 2); ++j) {
        const uint4 q = lds128(at + pr.at + 16 * j);
        r.c[j] = make_float2(__uint_as_float(q.x), __uint_as_float(q.z));
        r.s[j] = make_float2(__uint_as_float(q.y) * sg, __uint_as_float(q.w) * sg);
    }
    return r;
}

// Turn 8 channels by their angles.  Interleaved pairs lie in the thread (even
// channels apart from odd ones), those of halves in two lanes.  Channels that are
// not rotated keep their values (also next to an infinity, which the identity's
// zero sine would turn into NaN).
template <bool HALVES>
__device__ __forceinline__ void rotate8(V8& v, const Turn<HALVES>& t, const Pairs<HALVES>& pr) {
    const V8 old = v;
    if (!HALVES) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float2 a = v.p[2 * i], b = v.p[2 * i + 1];
            const float2 minus = make_float2(-t.s[i].x, -t.s[i].y);
            v.p[2 * i] = __ffma2_rn(b, minus, __fmul2_rn(a, t.c[i]));
            v.p[2 * i + 1] = __ffma2_rn(a, t.s[i], __fmul2_rn(b, t.c[i]));
        }
        if (pr.partial) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {  // pairs 2 (i / 2) and the next
                if (pr.keep >> (2 * (i / 2)) & 1u) v.p[i].x = old.p[i].x;
                if (pr.keep >> (2 * (i / 2) + 1) & 1u) v.p[i].y = old.p[i].y;
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 o = make_float2(__shfl_sync(0xFFFFFFFFu, v.p[i].x, pr.other),
                                         __shfl_sync(0xFFFFFFFFu, v.p[i].y, pr.other));
            v.p[i] = __ffma2_rn(o, t.s[i], __fmul2_rn(v.p[i], t.c[i]));
        }
        if (pr.partial && pr.keep != 0) v = old;
    }
}

// Sum over the lanes of a head (8 or 16).
__device__ __forceinline__ float head_sum(float v, int pieces) {
    v = lane_sum<8>(v);
    return pieces == 16 ? v + __shfl_xor_sync(0xFFFFFFFFu, v, 8) : v;
}

// Sums of NV values (2 or 4) over a token's W warps; every thread gets them.
// `buf` holds NV x W floats a use, used in turn with another, so the barrier of
// one use also ends the reads of the one before.  Tokens side by side in a block
// (`group`) wait apart from one another.
template <int NV, int W>
__device__ __forceinline__ void token_sum(float (&v)[NV], float* buf, int group, int warp) {
    const float s = scatter_sum<NV, 32>(v);
    if (scattered_writer<NV, 32>()) buf[warp * NV + scattered_index<NV, 32>()] = s;
    if (W == 1)
        __syncwarp();
    else
        asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "n"(32 * W) : "memory");
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        v[i] = buf[i];
#pragma unroll
        for (int k = 1; k < W; ++k) v[i] += buf[k * NV + i];
    }
}

// Eight floats a piece as two 16-byte planes `plane` bytes apart, pieces side by
// side: lanes read and write them without bank conflicts.
__device__ __forceinline__ V8 planes_load(uint32_t at, uint32_t plane) {
    const uint4 a = lds128(at), b = lds128(at + plane);
    V8 v;
    v.p[0] = make_float2(__uint_as_float(a.x), __uint_as_float(a.y));
    v.p[1] = make_float2(__uint_as_float(a.z), __uint_as_float(a.w));
    v.p[2] = make_float2(__uint_as_float(b.x), __uint_as_float(b.y));
    v.p[3] = make_float2(__uint_as_float(b.z), __uint_as_float(b.w));
    return v;
}

__device__ __forceinline__ void planes_store(uint32_t at, uint32_t plane, const V8& v) {
    sts128(at, make_uint4(__float_as_uint(v.p[0].x), __float_as_uint(v.p[0].y), __float_as_uint(v.p[1].x),
                          __float_as_uint(v.p[1].y)));
    sts128(at + plane, make_uint4(__float_as_uint(v.p[2].x), __float_as_uint(v.p[2].y), __float_as_uint(v.p[3].x),
                                  __float_as_uint(v.p[3].y)));
}

// The weights of 8 channels (ones where there are none).
template <bool EO>
__device__ __forceinline__ V8 weights_of(const void* w, int64_t at, int dtype) {
    float f[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = 1.0f;
    if (w != nullptr) load_param8(w, at, dtype, f);
    return arrange<EO>(f);
}

// The norm over a token: the weights of Q and K into shared memory once a block,
// [tensor][plane][piece of the token].
template <bool EO>
__device__ __forceinline__ void stage_weights(const HeadsArgs& a, uint32_t at) {
    const int all = a.H * a.pieces;
    for (int i = 0; i < 2; ++i)
#pragma unroll 4
        for (int e = threadIdx.x; e < all; e += blockDim.x)
            planes_store(at + (i * 2 * all + e) * 16, all * 16,
                         weights_of<EO>(a.weight[i], static_cast<int64_t>(e) * 8, a.weight_dtype));
}

// A warp's slots: stages of [tensor][VPT][32 lanes] pieces and the angles.  Those
// of pieces that do not exist hold zeros throughout.
__host__ __device__ constexpr uint32_t stage_bytes(int tensors, int vpt) {
    return tensors * vpt * 512 + kAngleBytes;
}

template <int TENSORS, int VPT, int STAGES>
__device__ __forceinline__ uint32_t slots_of(uint32_t at, int count) {
    constexpr uint32_t kStage = stage_bytes(TENSORS, VPT);
    constexpr int kPieces = TENSORS * VPT;
    at += (threadIdx.x >> 5) * STAGES * kStage + (threadIdx.x & 31) * 16;
    for (int e = 0; e < STAGES * kPieces; ++e)
        if (e % VPT >= count) sts128(at + e / kPieces * kStage + e % kPieces * 512, make_uint4(0, 0, 0, 0));
    return at;
}

// Blocks of 4 warps an SM shall hold at least, by the registers a thread needs.
__host__ __device__ constexpr int forward_blocks(int vpt) { return vpt <= 2 ? 4 : 3; }

// The backward pass's block: warps, tokens a lane's pieces are fetched ahead plus
// one, and how many blocks an SM shall hold.
__host__ __device__ constexpr int backward_warps(int W) { return W <= 2 ? 4 : W; }
__host__ __device__ constexpr int backward_stages(bool token, int vpt) { return token && vpt == 1 ? 3 : 2; }
__host__ __device__ constexpr int backward_tensors(int norm) { return norm == BSS_HEAD_NORM_NONE ? 3 : 5; }
__host__ __device__ constexpr int backward_blocks(int W, int vpt) {
    return vpt > 2 && W == 8 ? 1 : vpt > 2 ? 12 / backward_warps(W) : 16 / backward_warps(W);
}

// W warps share a token, a lane holds up to VPT pieces of a tensor.
template <bool HALVES, int NORM, int W, int VPT>
__global__ void __launch_bounds__(128, forward_blocks(VPT)) heads_forward_kernel(const __grid_constant__ HeadsArgs a) {
    extern __shared__ __align__(16) float4 planes[];  // weights of a norm over a token, then the slots
    __shared__ float buf[2][4 * 2];
    constexpr int kTokens = 4 / W;
    constexpr uint32_t kStage = stage_bytes(2, VPT), kTurn = 2 * VPT * 512;
    const int warp = threadIdx.x / 32 % W, group = threadIdx.x / 32 / W;
    Lane me = lane_of<W, VPT>(a, warp);
    const bool rotary = a.rot.first[3] > 0;
    const Pairs<HALVES> pr = pairs_of<HALVES>(a, me.piece);
    const Angles angles = angles_of(a);
    const uint32_t all16 = a.H * a.pieces * 16, row_bytes = a.pieces * 16;
    const uint32_t base = smem_u32(planes);
    const uint32_t weights = base + (me.head0 * a.pieces + me.piece) * 16;
    const uint32_t slots = slots_of<2, VPT, 2>(base + (NORM == BSS_HEAD_NORM_TOKEN ? 4 * all16 : 0), me.count);
    constexpr uint32_t step = kTokens;
    uint32_t n = blockIdx.x * a.span + group;
    const uint32_t end = a.N - blockIdx.x * a.span > a.span ? (blockIdx.x + 1) * a.span : a.N;
    // the lane's first piece in token 0, and the step to its next piece
    const char* src[3];
    int64_t apart[3];
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        src[i] = reinterpret_cast<const char*>(a.in[i] + me.head0 * a.hs[i] + me.piece * 8);
        apart[i] = me.step * a.hs[i] * 2;
    }
    const uint32_t turn_at = kTurn - (threadIdx.x & 31) * 16;  // from a lane's slots to the warp's angles
    if (rotary) clear_angles(angles, slots + turn_at), clear_angles(angles, slots + kStage + turn_at);
    uint32_t next_row = 0;  // of the fetched token in temporal heads
    auto fetch = [&](uint32_t m, bool exists, uint32_t to) {
        if (exists) {
            const Token tok = token_of(a, m);
            next_row = tok.temporal_row;
            if (rotary) fetch_angles(angles, tok, to + turn_at);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                if (a.in[i] == nullptr) continue;
                const char* p = src[i] + static_cast<uint64_t>(m) * a.ts[i];
#pragma unroll
                for (int j = 0; j < VPT; ++j, p += apart[i])
                    if (j < me.count) cp_async_16(to + (i * VPT + j) * 512, p);
            }
        }
        cp_async_commit();
    };
    fetch(n, n < end, slots);
    me.temporal = temporal_heads<VPT>(a, me);
    V8 w[2];
    if (NORM == BSS_HEAD_NORM_TOKEN) {
        stage_weights<!HALVES>(a, base);
        __syncthreads();
    } else if (NORM == BSS_HEAD_NORM_HEAD) {
#pragma unroll
        for (int i = 0; i < 2; ++i) w[i] = weights_of<!HALVES>(a.weight[i], me.piece * 8, a.weight_dtype);
    }
    const int64_t head_bytes = static_cast<int64_t>(a.N) * row_bytes;
    const int64_t head_step = me.step * head_bytes;
    const int64_t dst = me.head0 * head_bytes + me.piece * 16;
    uint32_t now = slots, other = slots + kStage;
    int turn_buf = 0;
    for (; n < end; n += step, turn_buf ^= 1) {
        const uint32_t temporal_row = next_row;
        uint4 v_raw[VPT];  // V goes straight through, its loads under Q and K's arithmetic
        if (a.in[2] != nullptr) {
            const char* p = src[2] + static_cast<uint64_t>(n) * a.ts[2];
#pragma unroll
            for (int j = 0; j < VPT; ++j, p += apart[2])
                if (j < me.count) v_raw[j] = ld_row(p);
        }
        __syncwarp();  // every lane has read the angles in the slots to be filled
        fetch(n + step, end - n > step, other);
        cp_async_wait_group<1>();
        Turn<HALVES> turn;
        if (rotary) {
            __syncwarp();  // the other lanes' copies
            turn = read_turn<HALVES, false>(pr, now + turn_at);
        }
        float r[2] = {0.0f, 0.0f};
        if (NORM == BSS_HEAD_NORM_TOKEN) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if (a.in[i] != nullptr)
#pragma unroll
                    for (int j = 0; j < VPT; ++j) {
                        const V8 v = unpack_bf16<false>(lds128(now + (i * VPT + j) * 512));
                        r[i] += dot(v, v);
                    }
            token_sum<2, W>(r, buf[turn_buf] + 2 * W * group, group, warp);
#pragma unroll
            for (int i = 0; i < 2; ++i) r[i] = rsqrtf(r[i] * a.inv_width + a.eps);
        }
        int64_t at = dst;
#pragma unroll
        for (int j = 0; j < VPT; ++j, at += head_step) {
            const bool live = j < me.count;
            const int64_t to = at + static_cast<uint64_t>(me.temporal >> j & 1u ? temporal_row : n) * row_bytes;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                if (a.in[i] == nullptr) continue;
                V8 v = unpack_bf16<!HALVES>(lds128(now + (i * VPT + j) * 512));
                if (NORM == BSS_HEAD_NORM_HEAD)
                    v = mul(v, mul(w[i], rsqrtf(head_sum(dot(v, v), a.pieces) * a.inv_width + a.eps)));
                if (NORM == BSS_HEAD_NORM_TOKEN && live)
                    v = mul(v, mul(planes_load(weights + i * 2 * all16 + j * (W * 512), all16), r[i]));
                if (rotary) rotate8<HALVES>(v, turn, pr);
                if (live) st_row(reinterpret_cast<char*>(a.out[i]) + to, pack_bf16<!HALVES>(v));
            }
            if (a.in[2] != nullptr && live) st_row(reinterpret_cast<char*>(a.out[2]) + to, v_raw[j]);
        }
        const uint32_t t = now;
        now = other, other = t;
    }
    cp_async_wait_group<0>();
}

// The norm over a token: W warps share one, each lane one piece of a tensor where
// it can (VPT = 1, up to 8 warps: the piece's weights, weight gradients and both
// passes' values stay in registers); wider tokens take several pieces a lane and 8
// warps.  Otherwise one warp a token.
template <bool HALVES, int NORM, int W, int VPT>
__global__ void __launch_bounds__(32 * backward_warps(W), backward_blocks(W, VPT))
    heads_backward_kernel(const __grid_constant__ HeadsArgs a) {
    constexpr bool kToken = NORM == BSS_HEAD_NORM_TOKEN, kOne = kToken && VPT == 1;
    constexpr int kWarps = backward_warps(W), kTokens = kWarps / W;
    constexpr int kTensors = backward_tensors(NORM), kStages = backward_stages(kToken, VPT);  // dQ, dK, dV, q, k
    constexpr uint32_t kStage = stage_bytes(kTensors, VPT), kTurn = kTensors * VPT * 512;
    extern __shared__ __align__(16) float4 planes[];
    __shared__ float4 buf4[2][kWarps];
    const int warp = threadIdx.x / 32 % W, group = threadIdx.x / 32 / W;
    Lane me = lane_of<W, VPT>(a, warp);
    me.temporal = temporal_heads<VPT>(a, me);
    const bool rotary = a.rot.first[3] > 0;
    const Pairs<HALVES> pr = pairs_of<HALVES>(a, me.piece);
    const Angles angles = angles_of(a);
    const uint32_t all16 = a.H * a.pieces * 16, row_bytes = a.pieces * 16;
    const uint32_t base = smem_u32(planes);
    const uint32_t weights = base + (me.head0 * a.pieces + me.piece) * 16;
    const uint32_t slots = slots_of<kTensors, VPT, kStages>(base, me.count);
    constexpr uint32_t step = kTokens;
    uint32_t n = blockIdx.x * a.span + group;
    const uint32_t end = a.N - blockIdx.x * a.span > a.span ? (blockIdx.x + 1) * a.span : a.N;
    const int64_t head_bytes = static_cast<int64_t>(a.N) * row_bytes;
    const int64_t head_step = me.step * head_bytes;
    const int64_t grad0 = me.head0 * head_bytes + me.piece * 16;
    const char* src[2];
    char* dst[3];
    int64_t xapart[2], apart[3];
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        dst[i] = reinterpret_cast<char*>(a.out[i] + me.head0 * a.hs[i] + me.piece * 8);
        apart[i] = me.step * a.hs[i] * 2;
        if (i < 2) {
            src[i] = reinterpret_cast<const char*>(a.x[i] + me.head0 * a.xhs[i] + me.piece * 8);
            xapart[i] = me.step * a.xhs[i] * 2;
        }
    }
    const uint32_t turn_at = kTurn - (threadIdx.x & 31) * 16;  // from a lane's slots to the warp's angles
    if (rotary)
        for (int k = 0; k < kStages; ++k) clear_angles(angles, slots + k * kStage + turn_at);
    auto fetch = [&](uint32_t m, bool exists, uint32_t to) {
        if (exists) {
            const Token tok = token_of(a, m);
            if (rotary) fetch_angles(angles, tok, to + turn_at);
            int64_t at = grad0;
#pragma unroll
            for (int j = 0; j < VPT; ++j, at += head_step) {
                const int64_t from = at + static_cast<uint64_t>(me.temporal >> j & 1u ? tok.temporal_row : m) * row_bytes;
                if (j < me.count)
#pragma unroll
                    for (int i = 0; i < 3; ++i)
                        if (a.in[i] != nullptr)
                            cp_async_16(to + (i * VPT + j) * 512, reinterpret_cast<const char*>(a.in[i]) + from);
            }
            if (NORM != BSS_HEAD_NORM_NONE)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    if (a.in[i] == nullptr) continue;
                    const char* p = src[i] + static_cast<uint64_t>(m) * a.xts[i];
#pragma unroll
                    for (int j = 0; j < VPT; ++j, p += xapart[i])
                        if (j < me.count) cp_async_16(to + ((3 + i) * VPT + j) * 512, p);
                }
        }
        cp_async_commit();
    };
#pragma unroll
    for (int k = 0; k < kStages - 1; ++k) fetch(n + k * step, n < end && end - n > k * step, slots + k * kStage);
    constexpr int kHeld = kToken ? VPT : 1;
    constexpr bool kInRegisters = NORM == BSS_HEAD_NORM_HEAD || kOne;  // the weights
    V8 w[2], dw[2][kHeld];
    // elsewhere they are read again for every token (from L1: beside the slots of a
    // wide token there is no shared memory for them)
    auto weight = [&](int i, int j) {
        return weights_of<!HALVES>(
            a.weight[i], kToken ? static_cast<int64_t>(me.head0 + j * me.step) * (a.pieces * 8) + me.piece * 8 : me.piece * 8,
            a.weight_dtype);
    };
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        if (kInRegisters) w[i] = kToken && me.count == 0 ? unpack_bf16<!HALVES>(make_uint4(0, 0, 0, 0)) : weight(i, 0);
#pragma unroll
        for (int j = 0; j < kHeld; ++j) dw[i][j] = unpack_bf16<!HALVES>(make_uint4(0, 0, 0, 0));
    }
    uint32_t now = slots, ahead_at = slots + (kStages - 1) * kStage;
    int turn_buf = 0;
    for (; n < end; n += step, turn_buf ^= 1) {
        __syncwarp();  // every lane has read the angles in the slots to be filled
        fetch(n + (kStages - 1) * step, end - n > (kStages - 1) * step, ahead_at);
        cp_async_wait_group<kStages - 1>();
        Turn<HALVES> turn;
        if (rotary) {
            __syncwarp();  // the other lanes' copies
            turn = read_turn<HALVES, true>(pr, now + turn_at);
        }
        float sums[4] = {0.0f, 0.0f, 0.0f, 0.0f};  // x^2 and g w x of Q, then of K
        V8 gv[2], xv[2];                           // of one piece, for both passes
        if (kToken) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                if (a.in[i] == nullptr) continue;
#pragma unroll
                for (int j = 0; j < VPT; ++j) {
                    V8 v = unpack_bf16<!HALVES>(lds128(now + (i * VPT + j) * 512));
                    if (rotary) rotate8<HALVES>(v, turn, pr);
                    if (!kOne && j >= me.count) continue;
                    const V8 x = unpack_bf16<!HALVES>(lds128(now + ((3 + i) * VPT + j) * 512));
                    sums[2 * i] += dot(x, x);
                    sums[2 * i + 1] += dot(mul(v, kOne ? w[i] : weight(i, j)), x);
                    if (kOne) gv[i] = v, xv[i] = x;
                }
            }
            token_sum<4, W>(sums, reinterpret_cast<float*>(buf4[turn_buf] + W * group), group, warp);
        }
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            if (a.in[i] == nullptr) continue;
            char* to = dst[i] + static_cast<uint64_t>(n) * a.ts[i];
            const int k = i < 2 ? i : 0;
            float r = 0.0f, m = 0.0f;
            if (kToken && i < 2) {
                r = rsqrtf(sums[2 * k] * a.inv_width + a.eps);
                m = -r * r * (sums[2 * k + 1] * a.inv_width);
            }
#pragma unroll
            for (int j = 0; j < VPT; ++j, to += apart[i]) {
                const bool live = j < me.count;
                if (i == 2) {
                    if (live) st_row(to, lds128(now + (i * VPT + j) * 512));
                    continue;
                }
                V8 v;
                if (kOne) {
                    v = gv[k];
                } else {
                    v = unpack_bf16<!HALVES>(lds128(now + (i * VPT + j) * 512));
                    if (rotary) rotate8<HALVES>(v, turn, pr);
                }
                if (NORM != BSS_HEAD_NORM_NONE) {
                    const V8 x = kOne ? xv[k] : unpack_bf16<!HALVES>(lds128(now + ((3 + k) * VPT + j) * 512));
                    V8 gw = v;
                    if (kInRegisters)
                        gw = mul(v, w[k]);
                    else if (live)
                        gw = mul(v, weight(k, j));
                    if (!kToken) {
                        // a piece that does not exist: zeros, whose root with eps = 0 is infinite
                        r = rsqrtf(head_sum(dot(x, x), a.pieces) * a.inv_width + a.eps);
                        r = live ? r : 0.0f;
                        m = -r * r * (head_sum(dot(gw, x), a.pieces) * a.inv_width);
                    }
                    const V8 xr = mul(x, r);
                    V8& d = dw[k][kToken ? j : 0];
                    d = fma8(v, xr, d);  // zeros where there is no piece
                    v = fma8(xr, m, mul(gw, r));
                }
                if (live) st_row(to, pack_bf16<!HALVES>(v));
            }
        }
        now = now == slots + (kStages - 1) * kStage ? slots : now + kStage;
        ahead_at = ahead_at == slots + (kStages - 1) * kStage ? slots : ahead_at + kStage;
    }
    cp_async_wait_group<0>();
    if (NORM == BSS_HEAD_NORM_NONE || a.partial == nullptr) return;
    // the block's share of the weight gradients: over the tokens side by side in
    // it, and for the norm over a head over its heads, in a fixed order
    __syncthreads();
    if (kToken) {
#pragma unroll
        for (int j = 0; j < kHeld; ++j)
            if (j < me.count)
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    planes_store(weights + (group * 2 + i) * 2 * all16 + j * (W * 512), all16, dw[i][j]);
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            planes_store(base + (i * 2 * blockDim.x + threadIdx.x) * 16, blockDim.x * 16, dw[i][0]);
    }
    __syncthreads();
    // element of a channel: [source][tensor][plane][piece][4]
    const int all = a.H * a.pieces, channels = kToken ? all * 8 : a.pieces * 8;
    const int span = kToken ? all : blockDim.x;
    const int sources = kToken ? kTokens : blockDim.x / a.pieces;
    const int apart_src = kToken ? 4 * all : a.pieces;
    const float* acc = reinterpret_cast<const float*>(planes);
    float* out = a.partial + static_cast<int64_t>(blockIdx.y * gridDim.x + blockIdx.x) * 2 * channels;
    for (int e = threadIdx.x; e < 2 * channels; e += blockDim.x) {
        const int i = e / channels, c = e - i * channels;
        int slot = 0;  // the channel's place among the four pairs of its piece
#pragma unroll
        for (int q = 0; q < 8; ++q)
            if (channel_of<!HALVES>(q / 2, q % 2) == c % 8) slot = q;
        const int at = ((i * 2 + slot / 4) * span + c / 8) * 4 + slot % 4;
        float s = 0.0f;
        for (int k = 0; k < sources; ++k) s += acc[at + k * apart_src * 4];
        out[e] = s;
    }
}

// out[c] = sum over the blocks' partials [blocks][2][width]: blocks in order
// within 32 lanes, then the lanes' sums in order.
__global__ void __launch_bounds__(1024) heads_reduce_kernel(const float* __restrict__ partial, int blocks, int width,
                                                            float* dq_weight, float* dk_weight) {
    __shared__ float part[32][33];
    const int col = threadIdx.x % 32, lane = threadIdx.x / 32, c = blockIdx.x * 32 + col;
    float s = 0.0f;
    cudaGridDependencySynchronize();
    if (c < 2 * width) {
#pragma unroll 4
        for (int b = lane; b < blocks; b += 32) s += partial[static_cast<int64_t>(b) * 2 * width + c];
    }
    part[lane][col] = s;
    __syncthreads();
    if (lane != 0 || c >= 2 * width) return;
    s = 0.0f;
#pragma unroll
    for (int k = 0; k < 32; ++k) s += part[k][col];
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

// How a token's heads are dealt to warps and grid columns.
constexpr int kWaves = 4;  // of the forward pass's blocks

struct Shape {
    int warps, vpt, heads_per_block, threads, smem;
    uint32_t grid_x, grid_y;
};

// Warps that share a token under the norm over a token.  Forward: one up to 2048
// channels.  Backward: one for each warp-wide row of pieces, up to 8.
int warps_of(bool backward, int chunks) {
    if (!backward) return chunks <= 8 ? 1 : 4;
    return chunks <= 6 ? chunks : 8;
}

Shape shape_of(int32_t H, int pieces, int32_t norm, uint32_t N, bool backward) {
    Shape s;
    const int per = 32 / pieces, total = (H + per - 1) / per;  // warp-wide rows of pieces
    const bool token = norm == BSS_HEAD_NORM_TOKEN;
    s.warps = token ? warps_of(backward, total) : 1;
    const int columns = token ? 1 : (total + 4) / 5;  // up to 5 pieces a lane and column
    const int held = (total + s.warps * columns - 1) / (s.warps * columns);
    // the instances there are: 1, 2, 3, 5; for the norm over a token forward 8 too
    // (the only one of 4 warps), backward 1 .. 4 (8 warps)
    s.vpt = backward && token ? held : !backward && s.warps == 4 ? 8 : held == 4 ? 5 : held > 5 ? 8 : held;
    s.heads_per_block = columns == 1 ? H : held * per;
    s.grid_y = static_cast<uint32_t>((H + s.heads_per_block - 1) / s.heads_per_block);
    const int block_warps = backward ? backward_warps(s.warps) : 4, tokens = block_warps / s.warps;
    s.threads = 32 * block_warps;
    // shared memory: the stages of every piece (V's only backward) and, forward, the
    // weights of the norm over a token; at the end of the backward pass the weight
    // gradients
    const int all = H * pieces * 64;
    const int tensors = backward ? backward_tensors(norm) : 2, stages = backward ? backward_stages(token, s.vpt) : 2;
    s.smem = (token && !backward ? all : 0) + block_warps * stages * static_cast<int>(stage_bytes(tensors, s.vpt));
    const int grads = token ? all * tokens : s.threads * 64;
    if (backward && norm != BSS_HEAD_NORM_NONE && s.smem < grads) s.smem = grads;
    // as many blocks as an SM holds, each walking over tokens
    const uint32_t blocks = (N + tokens - 1) / tokens;
    int per_sm = 224 * 1024 / (s.smem + 1024);
    per_sm = per_sm < 1 ? 1 : per_sm > 1024 / s.threads ? 1024 / s.threads : per_sm;
    const uint32_t fill = static_cast<uint32_t>(per_sm * num_sms()) / s.grid_y;
    s.grid_x = blocks < fill ? blocks : (fill < 1 ? 1 : fill);
    return s;
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
    if (!span_ok(N, ts) || !span_ok(H, hs) || ts % 8 != 0 || hs % 8 != 0 || ts > kMaxTokenStride)
        return set_error(BSS_ERR_INVALID_ARG,
                         "%s: strides must be multiples of 8 elements, not negative, a token's at most 2^28", name);
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

// What a call reads and what it writes: no byte is both, nor written twice.
struct Touched {
    Region in[16], out[6];
    int ins = 0, outs = 0;
    void read(const Region& r) { in[ins++] = r; }
    void write(const Region& r) { out[outs++] = r; }
    void read(const void* p, int64_t bytes) {
        if (p != nullptr && bytes > 0) read(region_2d(p, 1, 0, bytes, 1));
    }
    void write(const void* p, int64_t bytes) {
        if (p != nullptr && bytes > 0) write(region_2d(p, 1, 0, bytes, 1));
    }
    // weights, rotary tables and flags
    void read_options(const HeadsArgs& a, const bss_heads_options* o, int32_t d) {
        if (o->norm != BSS_HEAD_NORM_NONE) {
            const int64_t width = o->norm == BSS_HEAD_NORM_TOKEN ? static_cast<int64_t>(a.H) * d : d;
            for (const void* w : a.weight) read(w, width * (a.weight_dtype == BSS_DTYPE_F32 ? 4 : 2));
        }
        for (int i = 0; i < 3; ++i)
            if (a.rot.pairs[i] > 0) read(a.rot.table[i], static_cast<int64_t>(o->rotary->length[i]) * a.rot.pairs[i] * 8);
        read(a.flags, a.H);
    }
    bss_status check() const {
        for (int i = 0; i < outs; ++i) {
            for (int j = 0; j < ins; ++j)
                if (!disjoint(out[i], in[j])) return set_error(BSS_ERR_INVALID_ARG, "an output overlaps an input");
            for (int j = 0; j < i; ++j)
                if (!disjoint(out[i], out[j])) return set_error(BSS_ERR_INVALID_ARG, "outputs overlap");
        }
        return BSS_OK;
    }
};

using Kernel = void (*)(const HeadsArgs);

template <bool HALVES, int NORM>
Kernel pick_forward(const Shape& s) {
    if (NORM == BSS_HEAD_NORM_TOKEN && s.warps == 4) return heads_forward_kernel<HALVES, BSS_HEAD_NORM_TOKEN, 4, 8>;
    switch (s.vpt) {
        case 1: return heads_forward_kernel<HALVES, NORM, 1, 1>;
        case 2: return heads_forward_kernel<HALVES, NORM, 1, 2>;
        case 3: return heads_forward_kernel<HALVES, NORM, 1, 3>;
        case 5: return heads_forward_kernel<HALVES, NORM, 1, 5>;
        default: return heads_forward_kernel<HALVES, BSS_HEAD_NORM_TOKEN, 1, 8>;
    }
}

template <bool HALVES, int NORM>
Kernel pick_backward(const Shape& s) {
    switch (s.vpt) {
        case 1: return heads_backward_kernel<HALVES, NORM, 1, 1>;
        case 2: return heads_backward_kernel<HALVES, NORM, 1, 2>;
        case 3: return heads_backward_kernel<HALVES, NORM, 1, 3>;
        default: return heads_backward_kernel<HALVES, NORM, 1, 5>;
    }
}

template <bool HALVES>
Kernel pick_backward_token(const Shape& s) {
    switch (s.warps * 10 + s.vpt) {
        case 11: return heads_backward_kernel<HALVES, BSS_HEAD_NORM_TOKEN, 1, 1>;
        case 21: return heads_backward_kernel<HALVES, BSS_HEAD_NORM_TOKEN, 2, 1>;
        case 31: return heads_backward_kernel<HALVES, BSS_HEAD_NORM_TOKEN, 3, 1>;
        case 41: return heads_backward_kernel<HALVES, BSS_HEAD_NORM_TOKEN, 4, 1>;
        case 51: return heads_backward_kernel<HALVES, BSS_HEAD_NORM_TOKEN, 5, 1>;
        case 61: return heads_backward_kernel<HALVES, BSS_HEAD_NORM_TOKEN, 6, 1>;
        case 81: return heads_backward_kernel<HALVES, BSS_HEAD_NORM_TOKEN, 8, 1>;
        case 82: return heads_backward_kernel<HALVES, BSS_HEAD_NORM_TOKEN, 8, 2>;
        case 83: return heads_backward_kernel<HALVES, BSS_HEAD_NORM_TOKEN, 8, 3>;
        default: return heads_backward_kernel<HALVES, BSS_HEAD_NORM_TOKEN, 8, 4>;
    }
}

template <bool HALVES>
Kernel pick(bool backward, int32_t norm, const Shape& s) {
    if (norm == BSS_HEAD_NORM_TOKEN)
        return backward ? pick_backward_token<HALVES>(s) : pick_forward<HALVES, BSS_HEAD_NORM_TOKEN>(s);
    if (norm == BSS_HEAD_NORM_HEAD)
        return backward ? pick_backward<HALVES, BSS_HEAD_NORM_HEAD>(s) : pick_forward<HALVES, BSS_HEAD_NORM_HEAD>(s);
    return backward ? pick_backward<HALVES, BSS_HEAD_NORM_NONE>(s) : pick_forward<HALVES, BSS_HEAD_NORM_NONE>(s);
}

// Launches as many blocks as the GPU holds at once (never more than the shape's
// in the backward pass), times the waves; *blocks: how many.
bss_status launch(bool backward, int pairing, int32_t norm, const HeadsArgs& args, const Shape& s, cudaStream_t stream,
                  const char* what, int* blocks) {
    const Kernel k = pairing == BSS_PAIR_HALVES ? pick<true>(backward, norm, s) : pick<false>(backward, norm, s);
    int resident = 1;
    const bss_status st = resident_blocks(reinterpret_cast<const void*>(k), s.threads, s.smem, &resident);
    if (st != BSS_OK) return st;
    const uint32_t fill = static_cast<uint32_t>(resident * num_sms()) / s.grid_y;
    uint32_t grid_x = s.grid_x < fill ? s.grid_x : (fill < 1 ? 1 : fill);
    const uint32_t tokens = s.threads / 32 / s.warps;
    HeadsArgs a = args;
    // forward four waves of blocks, so that SMs that finish early take more; backward
    // one, since every block leaves a partial sum (75,600 tokens x 10 heads, measured
    // on earlier forms of the kernels: forward 193 us in four waves, 203 in one;
    // backward 291 in one, 301 in two)
    const uint32_t many = grid_x * (backward ? 1 : kWaves);
    a.span = (a.N + many - 1) / many;
    a.span = (a.span + tokens - 1) / tokens * tokens;
    grid_x = (a.N + a.span - 1) / a.span;
    *blocks = static_cast<int>(grid_x * s.grid_y);
    k<<<dim3(grid_x, s.grid_y), s.threads, s.smem, stream>>>(a);
    return cuda_check(cudaGetLastError(), what);
}

void set_shape(const Shape& s, int32_t norm, int32_t d, HeadsArgs* a) {
    a->heads_per_block = s.heads_per_block;
    a->pieces = d / 8;
    a->inv_width = 1.0f / static_cast<float>(norm == BSS_HEAD_NORM_TOKEN ? a->H * d : d);
}

void set_geometry(const bss_mask_params* p, int32_t H, const uint8_t* flags, HeadsArgs* a) {
    a->F = p->F;
    a->S = static_cast<uint32_t>(p->Hs) * p->Ws;
    a->N = a->S * a->F;
    a->by_S = FastDiv(a->S);
    a->by_Ws = FastDiv(p->Ws);
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
    Touched touched;
    Region r;
    int given = 0;
    for (int i = 0; i < 3; ++i) {
        const bool has = in[i] != nullptr && in[i]->data != nullptr;
        if (has != (out[i] != nullptr))
            return set_error(BSS_ERR_INVALID_ARG, "%s and its output must be given together", names[i]);
        if (!has) continue;
        ++given;
        if ((st = check_tokens(in[i], names[i], a.N, H, d, &r)) != BSS_OK) return st;
        if (!is_aligned(out[i], 16)) return set_error(BSS_ERR_INVALID_ARG, "outputs must be 16-byte aligned");
        touched.read(r);
        touched.write(out[i], static_cast<int64_t>(H) * a.N * d * 2);
        a.in[i] = static_cast<const __nv_bfloat16*>(in[i]->data);
        a.out[i] = static_cast<__nv_bfloat16*>(out[i]);
        a.ts[i] = a.N > 1 ? static_cast<uint32_t>(in[i]->token_stride * 2) : 0;
        a.hs[i] = H > 1 ? in[i]->head_stride : 0;
    }
    if (given == 0) return set_error(BSS_ERR_INVALID_ARG, "no tensor given");
    touched.read_options(a, options, d);
    if ((st = touched.check()) != BSS_OK) return st;
    const Shape s = shape_of(H, d / 8, options->norm, a.N, false);
    set_shape(s, options->norm, d, &a);
    int blocks = 0;
    return launch(false, pairing, options->norm, a, s, stream, "heads launch", &blocks);
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
    const Shape s = shape_of(H, params->head_dim / 8, norm, static_cast<uint32_t>(params->F) * params->Hs * params->Ws, true);
    const int64_t width = norm == BSS_HEAD_NORM_TOKEN ? static_cast<int64_t>(H) * params->head_dim : params->head_dim;
    *bytes = static_cast<int64_t>(s.grid_x) * s.grid_y * 2 * width * 4;
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
    Touched touched;
    Region r;
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
        touched.read(grad[i], static_cast<int64_t>(H) * a.N * d * 2);
        if ((st = check_tokens(out[i], names[i], a.N, H, d, &r)) != BSS_OK) return st;
        if (r.self_overlap) return set_error(BSS_ERR_INVALID_ARG, "%s overlaps itself", names[i]);
        touched.write(r);
        a.in[i] = static_cast<const __nv_bfloat16*>(grad[i]);
        a.out[i] = static_cast<__nv_bfloat16*>(out[i]->data);
        a.ts[i] = a.N > 1 ? static_cast<uint32_t>(out[i]->token_stride * 2) : 0;
        a.hs[i] = H > 1 ? out[i]->head_stride : 0;
        if (i == 2 || norm == BSS_HEAD_NORM_NONE) continue;
        if (x[i] == nullptr || x[i]->data == nullptr)
            return set_error(BSS_ERR_INVALID_ARG, "the norm's gradient needs %s", xnames[i]);
        if ((st = check_tokens(x[i], xnames[i], a.N, H, d, &r)) != BSS_OK) return st;
        touched.read(r);
        a.x[i] = static_cast<const __nv_bfloat16*>(x[i]->data);
        a.xts[i] = a.N > 1 ? static_cast<uint32_t>(x[i]->token_stride * 2) : 0;
        a.xhs[i] = H > 1 ? x[i]->head_stride : 0;
    }
    if (given == 0) return set_error(BSS_ERR_INVALID_ARG, "no tensor given");
    const Shape s = shape_of(H, d / 8, norm, a.N, true);
    set_shape(s, norm, d, &a);
    const bool want = dq_weight != nullptr || dk_weight != nullptr;
    const int width = norm == BSS_HEAD_NORM_TOKEN ? H * d : d;
    if (want) {
        if (!is_aligned(dq_weight, 16) || !is_aligned(dk_weight, 16))
            return set_error(BSS_ERR_INVALID_ARG, "weight gradients must be 16-byte aligned");
        const int64_t need = static_cast<int64_t>(s.grid_x) * s.grid_y * 2 * width * 4;
        if (workspace == nullptr || !is_aligned(workspace, 16) || workspace_bytes < need)
            return set_error(BSS_ERR_INVALID_ARG, "the workspace must be 16-byte aligned and hold %lld bytes",
                             static_cast<long long>(need));
        a.partial = static_cast<float*>(workspace);
        touched.write(dq_weight, 4 * width);
        touched.write(dk_weight, 4 * width);
        touched.write(workspace, need);
    }
    touched.read_options(a, options, d);
    if ((st = touched.check()) != BSS_OK) return st;
    int blocks = 0;
    st = launch(true, pairing, norm, a, s, stream, "heads backward launch", &blocks);
    if (st != BSS_OK || !want) return st;
    return launch_behind(heads_reduce_kernel, dim3((2 * width + 31) / 32), 1024, stream, "weight gradient launch",
                         a.partial, blocks, width, dq_weight, dk_weight);
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
    // what the attention call would refuse, before the first launch
    if (!is_aligned(O, 16) || !is_aligned(lse, 4)) return set_error(BSS_ERR_INVALID_ARG, "tensors must be 16-byte aligned");
    if (!attention_supports_block_q(map->BQ) || !attention_supports_block_kv(map->BKV))
        return set_error(BSS_ERR_UNSUPPORTED, "attention needs a map built with BQ = 128 or 256 and BKV = 64 or 128 (got %d x %d)",
                         map->BQ, map->BKV);
    int device = 0;
    cudaGetDevice(&device);
    if (device != map->device) return set_error(BSS_ERR_INVALID_ARG, "tile map belongs to device %d", map->device);
    bss_status st = check_geometry(&map->p, H);
    if (st != BSS_OK) return st;
    // of both launches; the heads call checks its inputs against the workspaces
    const int64_t bytes = static_cast<int64_t>(H) * map->g.N * map->p.head_dim * 2;
    Touched touched;
    touched.read(head_is_temporal, H);
    for (const void* p : {O, Qh, Kh, Vh}) touched.write(p, bytes);
    touched.write(lse, static_cast<int64_t>(H) * map->g.N * 4);
    if ((st = touched.check()) != BSS_OK) return st;
    const uint8_t* permuted = map->p.temporal_permuted ? head_is_temporal : nullptr;
    st = bss_heads_from_tokens(q, k, v, Qh, Kh, Vh, permuted, H, &map->p, options, stream);
    if (st != BSS_OK) return st;
    if (permuted == nullptr)
        return bss_sparse_attention(Qh, Kh, Vh, O, lse, map, head_is_temporal, H, 0.0f, stream);
    return bss_sparse_attention_split(Qh, Kh, Vh, O, Qh, Kh, Vh, nullptr, lse, map, head_is_temporal, H, 0.0f, stream);
}

}  // extern "C"
