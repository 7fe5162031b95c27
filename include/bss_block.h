/*
 * bss_block.h -- C ABI of the operators around the attention step in a video
 * transformer's block (implemented by the same library as bss.h).
 *
 * A block turns its token stream x into the next one around an attention call:
 *
 *   h = modulated norm of x             bss_residual_norm (x only)
 *   q, k, v = projections of h          bss_linear
 *   Qh, Kh, Vh = heads of q, k, v       bss_heads_from_tokens: Q/K norm, rotary
 *                                       positions of the (time, height, width)
 *                                       axes, head-major layout with temporal
 *                                       heads in (H,W,F) order
 *   O = block-sparse attention          bss_sparse_attention_split, or both in
 *                                       one call: bss_attention_step_tokens
 *   y = projection of O                 bss_linear
 *   r = a x + gate * y                  bss_residual_norm, which also writes the
 *   h = modulated norm of r             next layer's input in the same pass (or
 *                                       bss_linear, in the product's epilogue)
 *   c = attention over an encoder's     bss_cross_attention, between two
 *       states (a prompt)               bss_linear
 *   feed-forward layer                  bss_linear with an activation, then with
 *                                       a gate and the residual
 *
 * Each of these operators has its backward pass (the block-sparse attention has
 * none).  The blog has no counterpart to these
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

/* ------------------------------------------------------------ matrix products */

enum {
    BSS_ACT_NONE = 0,
    BSS_ACT_GELU_TANH = 1, /* z / 2 (1 + tanh(sqrt(2 / pi) (z + 0.044715 z^3))) */
    BSS_ACT_GELU = 2,      /* z / 2 (1 + erf(z / sqrt(2))) */
    BSS_ACT_SILU = 3       /* z / (1 + exp(-z)) */
};

/* A linear layer with what follows it, for `rows` rows of in_channels channels:
 *
 *   z   = x weight^T + bias
 *   out = residual_scale * residual + gate * activation(z)
 *
 * Products of bf16 values, sums and everything behind them in 32 bits, one
 * rounding at the store.  (The tensor cores add 16 products at a time to a sum
 * whose last bits are cut off, not rounded: about in_channels / 16 times 2^-24
 * below its size at most, which shows in float outputs only.)
 *   x           bf16 [rows][in_channels], rows x_stride elements apart.
 *   weight      bf16 [out_channels][in_channels], rows weight_stride apart.
 *   bias        param_dtype [out_channels], or NULL.
 *   gate        param_dtype [groups][out_channels], groups gate_stride apart (not
 *               used with one group), or NULL; row i belongs to group
 *               i / rows_per_group, groups = ceil(rows / rows_per_group).
 *   residual    out_dtype [rows][out_channels], or NULL (then residual_scale is 1).
 *   out         out_dtype [rows][out_channels]; may equal residual (same stride).
 *   pre         optional bf16 [rows][out_channels] output: z, which the backward
 *               pass reads.  The activation takes the unrounded z.
 *   workspace   device memory of at least the size that bss_linear_workspace gives,
 *               16-byte aligned, used by this call only until its work is done;
 *               NULL where that is 0.
 * Outputs overlap no other tensor.  Tensors are 16-byte aligned, strides multiples
 * of 8 elements of at most 2^28; in_channels and out_channels are multiples of 8,
 * 8 .. 65536; rows < 2^31. */
typedef struct {
    int64_t rows;
    int64_t rows_per_group;
    int32_t in_channels, out_channels;
    int32_t out_dtype, param_dtype;
    int32_t activation;
    float residual_scale;
    const void* x;
    const void* weight;
    const void* bias;
    const void* gate;
    const void* residual;
    void* out;
    void* pre;
    int64_t x_stride, weight_stride, gate_stride, residual_stride, out_stride, pre_stride;
    void* workspace;
    int64_t workspace_bytes;
} bss_linear_args;

/* Bytes of workspace that bss_linear needs for these arguments on the current
 * device (its workspace fields are not looked at). */
bss_status bss_linear_workspace(const bss_linear_args* args, int64_t* bytes);

/* Errors: INVALID_ARG, UNSUPPORTED, CUDA. */
bss_status bss_linear(const bss_linear_args* args, cudaStream_t stream);

/* Gradients of bss_linear, with dz = gate * dout * activation'(z):
 *
 *   dx = dz weight      dweight = dz^T x      dbias = sum over rows of dz
 *   dgate = sum over a group's rows of dout * activation(z)
 *
 * (The residual's gradient is residual_scale * dout.)
 *   dout        gradient of out, dout_dtype [rows][out_channels].
 *   x, weight   the forward inputs; x is read for dweight, weight for dx.
 *   pre         bf16, what the forward pass kept; read with an activation or for
 *               dgate (else may be NULL).
 *   gate        as in the forward pass.
 *   dx          bf16 [rows][in_channels];
 *   dweight     dweight_dtype [out_channels][in_channels], rows dweight_stride
 *               apart;
 *   dbias       float [out_channels]; dgate float [groups][out_channels], both
 *               contiguous; all overwritten, each NULL when not wanted (one at
 *               least is).  dgate needs gate.
 * With an activation, a gate or a float dout, dz is rounded to bf16 before the two
 * products (dbias and dgate are made from 32 bits).  Sums over rows are taken in a
 * fixed order.  Alignment, strides and the workspace as for bss_linear. */
typedef struct {
    int64_t rows;
    int64_t rows_per_group;
    int32_t in_channels, out_channels;
    int32_t dout_dtype, param_dtype, dweight_dtype;
    int32_t activation;
    const void* dout;
    const void* x;
    const void* weight;
    const void* pre;
    const void* gate;
    void* dx;
    void* dweight;
    float* dbias;
    float* dgate;
    int64_t dout_stride, x_stride, weight_stride, pre_stride, gate_stride, dx_stride, dweight_stride;
    void* workspace;
    int64_t workspace_bytes;
} bss_linear_grads;

bss_status bss_linear_backward_workspace(const bss_linear_grads* args, int64_t* bytes);

/* Errors: INVALID_ARG, UNSUPPORTED, CUDA. */
bss_status bss_linear_backward(const bss_linear_grads* args, cudaStream_t stream);

/* ------------------------------------------------------------ cross attention */

/* Keys or values of an encoder's states: element (group g, state t, head h,
 * channel c) at data[g * group_stride + t * token_stride + h * head_stride + c]
 * (strides in elements, multiples of 8; the stride of a dimension of size 1 is not
 * used, the others are positive, a token's at most 2^28, the others at most 2^38).
 * [groups][keys][kv_heads][d] tensors and views of a packed projection are of this
 * form.  An input's group stride may be 0: one set of states for all groups. */
typedef struct {
    void* data; /* bf16, 16-byte aligned */
    int64_t group_stride, token_stride, head_stride;
} bss_state_tensor;

/* Attention of `rows` tokens over an encoder's states of another length:
 *
 *   O[i][h] = sum over t of softmax_t(softmax_scale * q[i][h] . k[g][t][h']) v[g][t][h']
 *
 * with g = i / rows_per_group the row's group (a sample, or a piece of a clip with
 * a prompt of its own; groups = ceil(rows / rows_per_group)), h' = h / (heads /
 * kv_heads) the key head that h shares, and t over the group's valid states.
 *   q, O        token-major [rows][heads][head_dim] (strides as bss_token_tensor,
 *               positive where the dimension is larger than 1); O may be q (same
 *               strides).
 *   k, v        [groups][keys][kv_heads][head_dim].
 *   lengths     device int32 [groups]: the first lengths[g] states of a group are
 *               valid (taken as 0 below 0 and as keys above), the others are not
 *               looked at, whatever they hold; NULL = all.  With none a row's O is
 *               0 and its lse minus infinity; so they are where all its scores are
 *               minus infinity.
 *   lse         optional device float [heads][rows] output, 4-byte aligned: the
 *               natural logarithm of the softmax's denominator, for the backward
 *               pass.
 *   softmax_scale  <= 0: 1 / sqrt(head_dim).
 * Sums in 32 bits; the softmax's weights are rounded to bf16 on the way to their
 * product with v, their sum is not (with rows * heads up to the number of SMs neither).
 * head_dim 64 or 128; kv_heads divides heads, at most 65535; rows and keys < 2^31. */
typedef struct {
    int64_t rows;
    int64_t rows_per_group;
    int32_t heads, kv_heads, head_dim, keys;
    float softmax_scale;
    bss_token_tensor q, O;
    bss_state_tensor k, v;
    const int32_t* lengths;
    float* lse;
} bss_cross_args;

/* One launch.  Errors: INVALID_ARG, UNSUPPORTED, CUDA. */
bss_status bss_cross_attention(const bss_cross_args* args, cudaStream_t stream);

/* Gradients of bss_cross_attention, with P its softmax and D = sum of dO O a head:
 *
 *   dS = P (dO v - D)      dq = softmax_scale dS k      dv = P^T dO
 *   dk = softmax_scale dS^T q       (dk, dv: summed over the heads that share a key head)
 *
 *   dO, q, k, v, O, lse, lengths   the gradient of O and the forward call's inputs and
 *               outputs (here O is an input, and not q).  k and v have a group
 *               stride of their own when there is more than one group: states that
 *               several groups share are refused (with equal lengths the groups are
 *               one; else give each its copy and add the copies' gradients).
 *   dq          token-major [rows][heads][head_dim];
 *   dk, dv      [groups][keys][kv_heads][head_dim], zero where a state is not
 *               valid; at least two of groups, keys and kv_heads follow one another
 *               without a gap, as in a view of a packed tensor.  All overwritten.
 *   workspace   device memory of at least the size that
 *               bss_cross_attention_backward_workspace gives, 16-byte aligned, used
 *               by this call only until its work is done; NULL where that is 0.
 * P and dS are rounded to bf16 on the way to their products (in the call of one
 * launch they are not).  Sums over rows are taken in a fixed order.  Outputs overlap
 * no other tensor. */
typedef struct {
    int64_t rows;
    int64_t rows_per_group;
    int32_t heads, kv_heads, head_dim, keys;
    float softmax_scale;
    bss_token_tensor dO, q, O, dq;
    bss_state_tensor k, v, dk, dv;
    const int32_t* lengths;
    const float* lse;
    void* workspace;
    int64_t workspace_bytes;
} bss_cross_grads;

bss_status bss_cross_attention_backward_workspace(const bss_cross_grads* args, int64_t* bytes);

/* Three launches; one, without a workspace, where at most 16 rows and heads share a
 * group's key head and the call has few pairs of rows and keys.  Errors: INVALID_ARG, UNSUPPORTED, CUDA. */
bss_status bss_cross_attention_backward(const bss_cross_grads* args, cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* BSS_BLOCK_H_ */
