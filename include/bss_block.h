/*
 * bss_block.h -- C ABI of the operators on either side of the attention step in
 * a video transformer's block (implemented by the same library as bss.h).
 *
 * A block turns its token stream x into the next one around an attention call:
 *
 *   h = modulated norm of x             bss_residual_norm (x only)
 *   q, k, v = projections of h          the caller's matrix products
 *   Qh, Kh, Vh = heads of q, k, v       bss_heads_from_tokens: Q/K norm, rotary
 *                                       positions of the (time, height, width)
 *                                       axes, head-major layout with temporal
 *                                       heads in (H,W,F) order
 *   O = block-sparse attention          bss_sparse_attention_split, or both in
 *                                       one call: bss_attention_step_tokens
 *   y = projection of O                 the caller's matrix product
 *   r = a x + gate * y                  bss_residual_norm, which also writes the
 *   h = modulated norm of r             next block's input in the same pass
 *
 * Each operator has its backward pass.  The blog has no counterpart to these
 * calls: it treats Q, K, V as given; its section "Arrange tokens for efficient
 * temporal access" fixes the layout that bss_heads_from_tokens writes.
 *
 * Conventions as in bss.h: caller-owned device memory of the current device,
 * asynchronous on `stream`, host-detectable errors returned before anything is
 * launched, no call allocates device memory or synchronizes, every call may be
 * captured into a graph.  Results do not depend on timing: sums over tokens are
 * taken in a fixed order.
 */
#ifndef BSS_BLOCK_H_
#define BSS_BLOCK_H_

#include "bss.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of tensors that come in more than one. */
enum { BSS_DTYPE_BF16 = 0, BSS_DTYPE_F32 = 1 };

/* ------------------------------------------------------------------ rotary */

/* How a rotary pair's two channels are placed among the R rotated ones
 * (channels R .. head_dim - 1 pass unrotated). */
enum {
    BSS_PAIR_INTERLEAVED = 0, /* pair p = channels 2p, 2p + 1 */
    BSS_PAIR_HALVES = 1       /* pair p = channels p, p + R/2; R a multiple of 16 */
};

/* Rotary positions of three axes (0 time, 1 height, 2 width).  The R/2 pairs
 * are dealt to the axes in order: the first pairs[0] turn by the token's time
 * position, the next pairs[1] by its height, the last pairs[2] by its width;
 * R = 2 (pairs[0] + pairs[1] + pairs[2]) <= head_dim.
 *   table[a]   device float [length[a]][pairs[a]][2]: (cos, sin) of every
 *              position of the axis, 16-byte aligned (bss_rotary_table writes
 *              one); not read, and may be NULL, where pairs[a] = 0.
 *   offset[a]  >= 0: token (f, h, w) uses rows offset[0] + f, offset[1] + h and
 *              offset[2] + w, which must lie inside the tables.  A single token
 *              at its place in the clip is F = Hs = Ws = 1 with its offsets. */
typedef struct {
    const float* table[3];
    int32_t length[3];
    int32_t pairs[3];
    int32_t offset[3];
    int32_t pairing;
} bss_rotary;

/* Write one axis's table: out[i][j] = (cos, sin) of position_i * base^(-2 j / dim)
 * for i < length, j < pairs; angles in 64 bits, rounded once to float.
 *   positions  device double[length], or NULL for 0, 1, 2, ...
 *   dim        the divisor of the exponent: 2 * pairs gives each axis the whole
 *              range of frequencies of its own.
 *   base       > 0.
 *   out        device float [length][pairs][2], 16-byte aligned.
 * Errors: INVALID_ARG, UNSUPPORTED (length * pairs >= 2^31), CUDA. */
bss_status bss_rotary_table(const double* positions, int32_t length, int32_t pairs, int32_t dim, double base,
                            float* out, cudaStream_t stream);

/* ------------------------------------------------- heads from token-major Q, K, V */

/* Norm of Q and K before the rotary positions: x / sqrt(mean(x^2) + eps) * w. */
enum {
    BSS_HEAD_NORM_NONE = 0,
    BSS_HEAD_NORM_HEAD = 1, /* mean over each head's channels, w[head_dim] */
    BSS_HEAD_NORM_TOKEN = 2 /* mean over all heads of the token, w[H * head_dim]; H * head_dim <= 8192 */
};

/* One token-major tensor: element (token n, head h, channel c) at
 * data[n * token_stride + h * head_stride + c] (strides in elements, multiples
 * of 8, >= 0, the token stride at most 2^28; the stride of a dimension of size
 * 1 is not used).  [N][H][d] outputs, views of a packed [N][3][H][d] projection
 * and head-major [H][N][d] tensors are all of this form; inputs may also
 * broadcast (stride 0). */
typedef struct {
    void* data;           /* bf16, 16-byte aligned; NULL: this tensor is left out */
    int64_t token_stride;
    int64_t head_stride;
} bss_token_tensor;

/* Shared description of the two passes.
 *   norm, eps, weight_dtype, q_weight, k_weight   eps >= 0; weights of BSS_DTYPE_*,
 *              16-byte aligned, NULL = ones; all unused without a norm.  With
 *              eps = 0 a head (or token) of zeros gives NaN, as the formula does.
 *   rotary     NULL = no rotation. */
typedef struct {
    int32_t norm;
    float eps;
    int32_t weight_dtype;
    const void* q_weight;
    const void* k_weight;
    const bss_rotary* rotary;
} bss_heads_options;

/* Token-major Q, K, V -> the attention calls' head-major tensors in one pass:
 * Q and K normed and turned by their positions, every tensor written as
 * [H][N][d] with the heads whose flag is set in (H,W,F) order (row s*F + f), the
 * others in (F,H,W) order.  32-bit arithmetic, one rounding at the store.
 *   q, k, v     token-major inputs; any may be left out (data NULL) together
 *               with its output.  They are not written.
 *   Qh, Kh, Vh  device [H][N][d] bf16 outputs, 16-byte aligned, overlapping
 *               neither each other nor anything the call reads (weights, rotary
 *               tables and flags too).
 *   head_is_temporal  device uint8[H], NULL = no head permuted.
 * The results are what bss_sparse_attention takes for a map built with
 * temporal_permuted = 1.  Only F, Hs, Ws and head_dim of params are used.
 * Errors: INVALID_ARG, UNSUPPORTED, CUDA. */
bss_status bss_heads_from_tokens(const bss_token_tensor* q, const bss_token_tensor* k, const bss_token_tensor* v,
                                 void* Qh, void* Kh, void* Vh, const uint8_t* head_is_temporal, int32_t H,
                                 const bss_mask_params* params, const bss_heads_options* options,
                                 cudaStream_t stream);

/* Bytes of workspace the backward pass needs on the current device (0 when no
 * weight gradient is wanted). */
bss_status bss_heads_from_tokens_backward_workspace(int32_t H, const bss_mask_params* params, int32_t norm,
                                                    int64_t* bytes);

/* Gradients of bss_heads_from_tokens.  The library has no backward pass of the
 * attention: dQh, dKh and dVh are the caller's.
 *   dQh, dKh, dVh  device [H][N][d] bf16 gradients of its outputs, each head in
 *                  the layout it was written in; any may be NULL together with
 *                  its dq, dk or dv (data NULL).
 *   q, k           the forward inputs; read only with a norm (else may be NULL).
 *   dq, dk, dv     token-major outputs: all heads of a token lie within the token
 *                  stride, or all tokens of a head within the head stride.  They
 *                  may be views of one tensor, packed token by token ([N][3][H][d])
 *                  or head by head ([N][H][3][d]).
 *   dq_weight, dk_weight  device float [head_dim] or [H * head_dim] (by the norm)
 *                  gradients of the weights, overwritten; NULL = not wanted.
 *   workspace      device memory of at least the size that
 *                  bss_heads_from_tokens_backward_workspace gives, 16-byte
 *                  aligned, used by this call only until its work is done; NULL
 *                  when no weight gradient is wanted.
 * No output, nor the workspace, may overlap another or anything the call reads.
 * Errors: INVALID_ARG, UNSUPPORTED, CUDA. */
bss_status bss_heads_from_tokens_backward(const void* dQh, const void* dKh, const void* dVh,
                                          const bss_token_tensor* q, const bss_token_tensor* k,
                                          const bss_token_tensor* dq, const bss_token_tensor* dk,
                                          const bss_token_tensor* dv, float* dq_weight, float* dk_weight,
                                          const uint8_t* head_is_temporal, int32_t H, const bss_mask_params* params,
                                          const bss_heads_options* options, void* workspace,
                                          int64_t workspace_bytes, cudaStream_t stream);

/* The per-layer path from token-major projections: bss_heads_from_tokens into
 * Qh, Kh, Vh (workspaces of the caller, [H][N][d] bf16, all heads written), then
 * block-sparse attention on them with every head's O rows stored in (F,H,W)
 * order.  With a map built with temporal_permuted = 0, or head_is_temporal =
 * NULL, no head is permuted.  The same result as bss_heads_from_tokens without
 * flags followed by bss_attention_step, with one pass over Q, K, V less.  q, k
 * and v must all be given.  Two launches.  lse as in bss_attention_step.  O, lse,
 * Qh, Kh, Vh and the flags must not overlap one another.
 * Errors: those of the calls it makes. */
bss_status bss_attention_step_tokens(const bss_token_tensor* q, const bss_token_tensor* k,
                                     const bss_token_tensor* v, void* O, float* lse, bss_tile_map map,
                                     const uint8_t* head_is_temporal, int32_t H, const bss_heads_options* options,
                                     void* Qh, void* Kh, void* Vh, cudaStream_t stream);

/* --------------------------------------------------- norm, gate and residual */

enum {
    BSS_NORM_NONE = 0,
    BSS_NORM_LAYER = 1, /* (x - mean) / sqrt(variance + eps) */
    BSS_NORM_RMS = 2    /* x / sqrt(mean(x^2) + eps) */
};

/* The residual update of a block and the norm in front of the next one, for
 * `rows` tokens of `channels` channels (a multiple of 8, 8 .. 8192):
 *
 *   r = residual_scale * x + gate * y_norm(y) * y_weight
 *   h = (norm(r) * weight + bias) * (1 + scale) + shift
 *
 * computed in 32 bits; r and h are each rounded once when stored (h is made from
 * the unrounded r).
 *   x, r        stream_dtype, rows x_stride / r_stride elements apart.  y = NULL:
 *               there is no update, r must be NULL (and residual_scale 1) and h
 *               is made from x.  r may be NULL when only h is wanted, or equal x
 *               (updated in place, same stride).
 *   y, h        branch_dtype, likewise; h may be NULL when only r is wanted, or
 *               equal y (same stride).  Otherwise outputs overlap no input and
 *               no other output.  (x and y may be one tensor, then also with r or
 *               h over it.)
 *   gate, scale, shift   param_dtype [groups][channels], groups gate_stride ...
 *               elements apart (not used with one group); row i belongs to group
 *               i / rows_per_group, groups = ceil(rows / rows_per_group): one
 *               set of modulations a sample, a frame or a token.  Each may be
 *               NULL (gate 1, scale 0, shift 0).
 *   weight, bias, y_weight   param_dtype [channels], each may be NULL.
 *   norm        of r for h (BSS_NORM_NONE: h = modulated r); y_norm of y.
 *   stats, y_stats   optional device float [rows][2] outputs: each row's (mean,
 *               1 / deviation) of norm and y_norm (mean 0 for RMS), which the
 *               backward pass reads.
 * (stream_dtype, branch_dtype): (BF16, BF16), (F32, BF16) or (F32, F32).
 * Tensors are 16-byte aligned, their strides multiples of 8 elements of at most
 * 2^28; stats are 8-byte aligned. */
typedef struct {
    int64_t rows;
    int64_t rows_per_group;
    int32_t channels;
    int32_t stream_dtype, branch_dtype, param_dtype;
    int32_t norm, y_norm;
    float eps;
    float residual_scale;
    const void* x;
    const void* y;
    void* r;
    void* h;
    int64_t x_stride, y_stride, r_stride, h_stride;
    const void* gate;
    const void* scale;
    const void* shift;
    int64_t gate_stride, scale_stride, shift_stride;
    const void* weight;
    const void* bias;
    const void* y_weight;
    float* stats;
    float* y_stats;
} bss_residual_norm_args;

/* One launch.  Errors: INVALID_ARG, UNSUPPORTED, CUDA. */
bss_status bss_residual_norm(const bss_residual_norm_args* args, cudaStream_t stream);

/* Gradients of bss_residual_norm.
 *   r           the updated stream that the forward pass wrote (x when there was
 *               no update), with its stats; y with y_stats when it was normed.
 *   dr          gradient of r from its later uses (stream_dtype), dh of h
 *               (branch_dtype); one of them may be NULL.  stats are read when
 *               dh is given and norm is not BSS_NORM_NONE, y_stats when y is and
 *               y_norm is not.
 *   dx          gradient of x (stream_dtype); may equal dr (same stride).
 *   dy          gradient of y (branch_dtype), NULL when y is; may equal dh (same
 *               stride).  Otherwise outputs overlap no input and no other output.
 *   dgate, dscale, dshift   device float [groups][channels], contiguous;
 *   dweight, dbias, dy_weight   device float [channels]; all overwritten, each
 *               NULL when not wanted, 16-byte aligned.  dgate and dy_weight need
 *               y, the others dh; a factor that is NULL counts as in the forward
 *               pass (gate 1, scale 0, weight 1, bias 0).
 *   workspace   device memory of at least the size that
 *               bss_residual_norm_backward_workspace gives, 16-byte aligned, used
 *               by this call only until its work is done. */
typedef struct {
    int64_t rows;
    int64_t rows_per_group;
    int32_t channels;
    int32_t stream_dtype, branch_dtype, param_dtype;
    int32_t norm, y_norm;
    float residual_scale;
    const void* r;
    const void* y;
    const void* dr;
    const void* dh;
    void* dx;
    void* dy;
    int64_t r_stride, y_stride, dr_stride, dh_stride, dx_stride, dy_stride;
    const float* stats;
    const float* y_stats;
    const void* gate;
    const void* scale;
    int64_t gate_stride, scale_stride;
    const void* weight;
    const void* bias;
    const void* y_weight;
    float* dgate;
    float* dscale;
    float* dshift;
    float* dweight;
    float* dbias;
    float* dy_weight;
    void* workspace;
    int64_t workspace_bytes;
} bss_residual_norm_grads;

/* Bytes of workspace that bss_residual_norm_backward needs for these arguments
 * on the current device (its workspace fields are not looked at).  Where a
 * parameter's gradient is wanted every group takes at least 12 bytes a channel. */
bss_status bss_residual_norm_backward_workspace(const bss_residual_norm_grads* args, int64_t* bytes);

/* Errors: INVALID_ARG, UNSUPPORTED, CUDA. */
bss_status bss_residual_norm_backward(const bss_residual_norm_grads* args, cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* BSS_BLOCK_H_ */
