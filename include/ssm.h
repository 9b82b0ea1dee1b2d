/*
 * ssm.h -- C ABI of the operators of a selective state space layer, for MI355X
 * (gfx950), in libwkv6.so next to the WKV operators of wkv6.h and the
 * linear-attention operators of linattn.h:
 *
 *   ssm_conv_fwd, ssm_conv_bwd   short causal convolution of each channel
 *   ssm_scan_fwd, ssm_scan_bwd   selective scan, gated: prompts, pieces of
 *                                prompts and single tokens
 *   ssm_block_norm, _bwd         norm after a block, gate, scaled addition to
 *                                the residual stream, norm before the next one
 *
 * Common to all, as in linattn.h.  Tensors are device memory of the caller,
 * 16-byte aligned (the tables A, weight, bias, skip and dt_bias among them);
 * the library keeps no pointer after returning.  Calls are asynchronous on
 * `stream` (a hipStream_t; the current device must be the stream's), do not
 * synchronise the host and are thread-safe.  They return a WKV6_* status
 * (wkv6.h); on INVALID_ARG, UNSUPPORTED and MISALIGNED nothing is enqueued and
 * wkv6_last_error says why.  Values are not checked: NaN and infinities
 * propagate (an infinity may become NaN on the way), never to an earlier token's
 * outputs or another channel's; in gradients, to what the formulas derive from them.
 * Outputs must not overlap inputs or one another except where it is said
 * below.  Every result is bit-for-bit the same for the same call (no atomics).
 *
 * `dtype` (WKV6_DTYPE_F32 or WKV6_DTYPE_BF16) is the type of the tensors with
 * a token dimension; everything is computed in float32 and rounded once, on
 * the way out.
 *
 * lengths: NULL, or B int32 values on the device: item b has min(max(lengths[b],
 * 0), T) tokens.  The rows of the inputs behind them are not read, those of the
 * outputs are set to zero, and states are those after the last token that
 * counts.
 *
 * strides: NULL: the tensors are contiguous.  Else distances in elements, >= 0
 * and multiples of 16 bytes (channels and states are always adjacent); a
 * distance of 0 repeats an input; rows of outputs must not share elements.
 * Slices of one buffer that lie side by side are fine.  The distance of a
 * dimension of one place does not matter.
 *
 * Workspace: the caller's (16-byte aligned, at least *_workspace_bytes bytes,
 * for the call alone until the stream has run it), or NULL to take it in stream
 * order from the library's pool (wkv6.h).  A call that is given its workspace, or needs
 * none, enqueues kernel launches only and can be captured in a HIP graph.
 */
#ifndef SSM_H
#define SSM_H

#include "wkv6.h"

#ifdef __cplusplus
extern "C" {
#endif

#define SSM_ABI_VERSION 1

/* Most states of a channel (N of ssm_scan_fwd and ssm_scan_bwd). */
#define SSM_MAX_STATES 64
/* Most inputs of a convolution (W of ssm_conv_fwd and ssm_conv_bwd). */
#define SSM_MAX_WINDOW 4
/* Most columns of a row of ssm_block_norm. */
#define SSM_MAX_COLUMNS 16384

/* activation of ssm_conv_fwd (NONE, SILU) and of the gate of ssm_block_norm */
#define SSM_ACT_NONE    0
#define SSM_ACT_SILU    1  /* v / (1 + exp(-v)) */
#define SSM_ACT_SIGMOID 2  /* 1 / (1 + exp(-v)) */

/*
 * ssm_conv_fwd -- short causal convolution of each channel:
 *
 *     p_t[d] = bias[d] + sum_{j < W} weight[d][j] x_{t-W+1+j}[d],    y_t = act(p_t)
 *
 * where the rows before the first token are those of the state.
 *
 *   B, T, D, W   batch, tokens, channels (a multiple of 8 up to 2^20) and inputs
 *             of the window, 2 to SSM_MAX_WINDOW; B * D is at most 2^25 and B * (T / 16
 *             + 258) * (D + 2) below 2^32
 *   x, y      [B, T, D] of `dtype`
 *   weight    [D, W] float32, contiguous; weight[d][W - 1] is the current token's
 *   bias      NULL (zero), or D float32 values
 *   act       SSM_ACT_NONE or SSM_ACT_SILU
 *   s_in      NULL (zero), or [B, W - 1, D] of `dtype`, contiguous: the last
 *             rows of x before this call, the newest last
 *   s_out     NULL, or the same shape: the last W - 1 rows of s_in followed by
 *             x; it may be s_in itself
 *   strides   NULL, or 4 values: (batch, token) distances of x, then of y
 *   T == 0    s_out receives s_in (or zero).  B == 0: nothing is done.
 */
int ssm_conv_fwd(int64_t B, int64_t T, int64_t D, int64_t W, const void* x, const float* weight, const float* bias,
                 int act, const int32_t* lengths, const void* s_in, void* y, void* s_out, const int64_t* strides,
                 int dtype, void* stream);

/*
 * ssm_conv_bwd -- gradients of sum(y * dy) + sum(s_out * ds_out).
 *
 *   dy, dx    [B, T, D] of `dtype`
 *   ds_out    NULL (zero), or [B, W - 1, D] of `dtype`
 *   ds_in     NULL, or the same: the gradient of s_in
 *   dweight   [D, W] float32;  dbias: NULL, or D float32 values.  Fully
 *             overwritten (zero when nothing counts).
 *   strides   NULL, or 6 values: (batch, token) distances of x, dy and dx
 *
 * A weight that is not finite makes NaN of its channel's dx and ds_in also in the first
 * and last W - 1 rows where no token's product with it counts.
 */
int ssm_conv_bwd(int64_t B, int64_t T, int64_t D, int64_t W, const void* x, const float* weight, const float* bias,
                 int act, const int32_t* lengths, const void* s_in, const void* dy, const void* ds_out, void* dx,
                 float* dweight, float* dbias, void* ds_in, const int64_t* strides, int dtype, void* workspace,
                 size_t workspace_bytes, void* stream);

/* Workspace of an ssm_conv_bwd call (partial sums of dweight and dbias). */
size_t ssm_conv_bwd_workspace_bytes(int64_t B, int64_t T, int64_t D, int64_t W, int dtype);

/*
 * ssm_scan_fwd -- selective scan: per batch item and channel d, of group g = d /
 * (D / G), with N float32 states that start at s_in (or zero),
 *
 *     delta_t = softplus(dt_t[d] + dt_bias[d])      (without softplus: the sum itself)
 *     h_t[n]  = exp(delta_t A[d][n]) h_{t-1}[n] + delta_t x_t[d] B_t[g][n]
 *     y_t[d]  = (sum_n C_t[g][n] h_t[n] + skip[d] x_t[d]) * silu(z_t[d])
 *
 *   B, T, D, N, G   batch, tokens, channels, states of a channel and groups: D
 *             and D / G are multiples of 8 (D up to 2^20), N a multiple of 8 up to
 *             SSM_MAX_STATES; B * D is at most 2^25
 *   x, dt, z, y   [B, T, D] of `dtype`; z may be NULL (no gate)
 *   A         [D, N] float32, contiguous: negative and finite, the states' rates of decay.
 *             Positive ones grow; exp(A times the steps of 128 tokens) has to be
 *             a finite float32.
 *   Bm, Cm    [B, T, G, N] of `dtype`
 *   skip, dt_bias   NULL (zero), or D float32 values each
 *   s_in      NULL (zero), or [B, D, N] float32, contiguous
 *   s_out     NULL, or the same: the state after the last token; it may be s_in
 *             itself
 *   strides   NULL, or 18 values: (batch, token, group) distances of x, dt, Bm,
 *             Cm, z and y (x, dt, z and y have no groups: theirs is not read)
 *   T == 0    s_out receives s_in (or zero).  B == 0: nothing is done.
 *
 * Calls of at most 8 tokens run token by token, longer ones over blocks of 32 to
 * 128 tokens whose tokens lie side by side over lanes.
 */
int ssm_scan_fwd(int64_t B, int64_t T, int64_t D, int64_t N, int64_t G, const void* x, const void* dt, const float* A,
                 const void* Bm, const void* Cm, const float* skip, const void* z, const float* dt_bias, int softplus,
                 const int32_t* lengths, const float* s_in, void* y, float* s_out, const int64_t* strides, int dtype,
                 void* stream);

/*
 * ssm_scan_bwd -- gradients of sum(y * dy) + sum(s_out * ds_out).
 *
 *   dy        [B, T, D] of `dtype`
 *   ds_out    NULL (zero), or [B, D, N] float32
 *   dx, ddt, dz   [B, T, D] of `dtype`; dz is given exactly where z is
 *   dB, dC    [B, T, G, N] of `dtype`: summed over the channels of a group
 *   dA        [D, N] float32;  dskip, ddt_bias: NULL, or D float32 values each.
 *             Fully overwritten (zero when nothing counts).
 *   ds_in     NULL, or [B, D, N] float32; it may be ds_out itself
 *   strides   NULL, or 33 values: (batch, token, group) distances of x, dt, Bm,
 *             Cm, z, dy, dx, ddt, dB, dC and dz.  An input with a distance of 0
 *             gets one gradient row for each place it is used at; their sum is
 *             the caller's.
 */
int ssm_scan_bwd(int64_t B, int64_t T, int64_t D, int64_t N, int64_t G, const void* x, const void* dt, const float* A,
                 const void* Bm, const void* Cm, const float* skip, const void* z, const float* dt_bias, int softplus,
                 const int32_t* lengths, const float* s_in, const void* dy, const float* ds_out, void* dx, void* ddt,
                 float* dA, void* dB, void* dC, float* dskip, void* dz, float* ddt_bias, float* ds_in,
                 const int64_t* strides, int dtype, void* workspace, size_t workspace_bytes, void* stream);

/* Workspace of an ssm_scan_bwd call: the states at the starts of blocks of
 * tokens and sums of dB and dC of blocks of channels. */
size_t ssm_scan_bwd_workspace_bytes(int64_t B, int64_t T, int64_t D, int64_t N, int64_t G, int dtype);

/*
 * ssm_block_norm -- between two blocks of a layer stack:
 *
 *     n = x / sqrt(mean(x^2) + eps) * post          (without post: x itself)
 *     h = residual + scale * act(gate) * n          (rounded to `dtype`; a missing term is 0, a
 *                                                    missing gate 1)
 *     y = h / sqrt(mean(h^2) + eps) * pre           (without pre there is no y)
 *
 * with means over the C columns of each row; y is the norm of h as it is stored.
 * Squares are added up in float32: rows whose sum of squares leaves its range,
 * 2^128, give n = 0 or y = 0; squares below 2^-126 lose places and count for little
 * or nothing next to eps.
 *
 *   rows, C   C is a multiple of 8 up to SSM_MAX_COLUMNS; at most 2^25 rows, or
 *             2^21 of more than 512 columns
 *   x, residual, h, y   [rows, C] of `dtype`, contiguous.  residual may be NULL;
 *             h may be x or residual itself; y is NULL exactly where pre is.
 *   gate      NULL, or [rows / gate_rows, C] of `dtype`: each gate_rows rows in a
 *             row share a row of the gate (1: one for every row; the tokens of a
 *             sequence: one for each sequence; rows: one for all).  gate_rows
 *             divides rows; gates that more than one row share are at most 2^22.
 *   act       SSM_ACT_*, of the gate (NONE without one)
 *   post, pre   NULL, or C float32 values
 *   scale     finite;  eps: finite, >= 0
 */
int ssm_block_norm(int64_t rows, int64_t C, const void* x, const void* residual, const void* gate, int64_t gate_rows,
                   const float* post, const float* pre, float scale, int act, float eps, void* h, void* y, int dtype,
                   void* stream);

/*
 * ssm_block_norm_bwd -- gradients of sum(y * dy) + sum(h * dh).
 *
 *   x, gate, post, pre, scale, act, eps   as in the forward call
 *   h         [rows, C] of `dtype`, of the forward call (not read without pre:
 *             may be NULL)
 *   dy        [rows, C] of `dtype`; NULL exactly where pre is
 *   dh        NULL (zero), or [rows, C] of `dtype`: the gradient that reaches h
 *             by the residual stream
 *   dx        [rows, C] of `dtype`; it may be dy itself
 *   dresidual   NULL, or [rows, C] of `dtype`; it may be dh itself
 *   dgate     [rows / gate_rows, C] of `dtype`, summed over the rows that share a
 *             gate; NULL exactly where gate is
 *   dpost, dpre   C float32 values each, fully overwritten (zero when rows ==
 *             0); NULL exactly where post and pre are
 */
int ssm_block_norm_bwd(int64_t rows, int64_t C, const void* x, const void* h, const void* gate, int64_t gate_rows,
                       const float* post, const float* pre, float scale, int act, float eps, const void* dy,
                       const void* dh, void* dx, void* dresidual, void* dgate, float* dpost, float* dpre, int dtype,
                       void* workspace, size_t workspace_bytes, void* stream);

/* Workspace of an ssm_block_norm_bwd call (partial sums of dpost, dpre and of a
 * gate that rows share): post, gate and pre say which of them there are.  The rows of
 * each such gate are added up apart, at least C floats for each sum and gate, written and
 * read again: with all three sums in bfloat16 three times the bytes of x where two
 * rows share a gate, a fifth of them where 32 or more do. */
size_t ssm_block_norm_bwd_workspace_bytes(int64_t rows, int64_t C, int64_t gate_rows, int post, int gate, int pre,
                                          int dtype);

/* SSM_ABI_VERSION of the loaded library. */
int ssm_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* SSM_H */
