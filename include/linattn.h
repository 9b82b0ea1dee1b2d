/*
 * linattn.h -- C ABI of the operators of a linear-attention (retention) layer
 * with one decay for each head, for MI355X (gfx950), in libwkv6.so next to
 * the WKV operators of wkv6.h, whose status codes, data types, workspace pool
 * and error text they share:
 *
 *   linattn_fwd        prompts, pieces of prompts and single tokens
 *   linattn_bwd        its gradients
 *   linattn_rope       rotary positions of the queries and keys
 *   linattn_rms_norm   root-mean-square norm with the residual's addition,
 *   linattn_rms_norm_q8   ... with an 8-bit output and its scales,
 *   linattn_rms_norm_bwd  ... and its gradients
 *
 * Common to all.  Tensors are device memory of the caller, 16-byte aligned
 * (log_decay and positions: 4-byte); the library keeps no pointer after
 * returning.  Calls are asynchronous on `stream` (a hipStream_t; the current
 * device must be the stream's), do not synchronise the host and are
 * thread-safe.  They return a WKV6_* status (wkv6.h); on INVALID_ARG, UNSUPPORTED and MISALIGNED nothing is enqueued
 * and wkv6_last_error says why.  Values are not checked: NaN and infinities
 * propagate.  Outputs must not overlap inputs or one another except where it
 * is said below.  Every result is bit-for-bit the same for the same call (no
 * atomics).
 *
 * Workspace.  Calls that need device workspace say how much in a
 * *_workspace_bytes function (host arithmetic).  `workspace` is the caller's
 * (16-byte aligned, at least that many bytes, for the call alone until the
 * stream has run it), or NULL to take it in stream order from the library's
 * pool (see wkv6.h).  A call that is given its workspace, or needs none,
 * enqueues kernel launches only and can be captured in a HIP graph.
 */
#ifndef LINATTN_H
#define LINATTN_H

#include "wkv6.h"

#ifdef __cplusplus
extern "C" {
#endif

#define LINATTN_ABI_VERSION 1

/* Largest head size (K and V of linattn_fwd and linattn_bwd, D of linattn_rope). */
#define LINATTN_MAX_HEAD 128
/* Most columns of a normalised row. */
#define LINATTN_MAX_COLUMNS 16384

/*
 * linattn_fwd -- linear attention with one decay for each head.
 *
 * Per batch item b and head h, with a = exp(log_decay[h]) and a K x V float32
 * state S that starts at s_in (or zero):
 *
 *     S_t = a S_{t-1} + k_t^T v_t,      o_t = scale * q_t S_t
 *
 * i.e. token i <= t reaches t with weight a^(t-i) (the current token with
 * weight 1).  Calls of at most 8 tokens run the recurrence token by token;
 * longer ones run in chunks of 64 tokens on matrix cores.
 *
 *   B, T, H, K, V   batch, tokens, heads, key and value channels of a head;
 *             K and V are multiples of 8 from 8 to 128, B * H is at most 2^21
 *             (else UNSUPPORTED).
 *   q, k      [B, T, H, K] of `dtype` (WKV6_DTYPE_F32 or WKV6_DTYPE_BF16)
 *   v         [B, T, H, V] of `dtype`
 *   log_decay H float32 values: the natural logarithms of the decays.
 *             Finite, or -inf (a = 0: each token sees itself alone).  Above 0
 *             the state grows: a^64 has to be a finite float32 (1.38 at most).
 *   scale     factor of every output
 *   lengths   NULL, or B int32 values on the device: item b has
 *             min(max(lengths[b], 0), T) tokens.  The rows of q, k and v
 *             behind them are not read, those of o are set to zero, and
 *             s_out is the state after the last token that counts.
 *   s_in      NULL (zero), or [B, H, K, V] float32, contiguous
 *   o         [B, T, H, V] of `out_dtype`: fully overwritten.  float32 inputs
 *             take a float32 output; bfloat16 inputs either type.
 *   s_out     NULL, or [B, H, K, V] float32, contiguous; it may be s_in itself.
 *   strides   NULL: q, k, v and o are contiguous.  Else 12 values: the
 *             distances in elements between batch items, tokens and heads of
 *             q, then of k, v and o; channels are always adjacent.  Each is
 *             >= 0 and a multiple of 16 bytes; a distance of 0 repeats an
 *             input (keys shared by all heads); the rows of o must not share
 *             elements.  Outputs and inputs may be slices of one buffer that
 *             lie side by side (the same distances, but for those of heads that
 *             differ in size: all q of a token, then all k, then all v).  The
 *             distance of a dimension of one place does not matter.  In calls
 *             of more than 8 tokens (linattn_bwd: one) the token distance, also
 *             that of contiguous tensors, is at most 33554288 bytes (else
 *             UNSUPPORTED).
 *   T == 0    s_out receives s_in (or zero).  B == 0: nothing is done.
 *
 * Precision: products run on matrix cores on bfloat16 parts of their operands
 * with float32 accumulation.  With a float32 output every operand is carried
 * whole (three parts); with a bfloat16 output, weights between tokens and the
 * state as it meets the queries are rounded once to bfloat16, like the output.
 * The state itself is float32 throughout.  The outputs are the same bits
 * whether or not s_out is asked for.  A NaN or infinity in q reaches the
 * outputs of its token, one in k those of its token and of later ones; in calls
 * of more than 8 tokens one in v can also reach those of the up to 31 tokens
 * before it in its chunk (their weight, 0, times it is NaN).
 */
int linattn_fwd(int64_t B, int64_t T, int64_t H, int64_t K, int64_t V, const void* q, const void* k, const void* v,
                const float* log_decay, float scale, const int32_t* lengths, const float* s_in, void* o, float* s_out,
                const int64_t* strides, int dtype, int out_dtype, void* workspace, size_t workspace_bytes,
                void* stream);

/* Workspace of a linattn_fwd call (0: none, or the arguments are invalid):
 * states at the starts of the segments that a long call over few heads is cut
 * into, B*H*segments*K*V*4 bytes (K and V rounded up to 64 or 128).  `state_out`: s_out is given. */
size_t linattn_fwd_workspace_bytes(int64_t B, int64_t T, int64_t H, int64_t K, int64_t V, int dtype, int out_dtype,
                                   int state_out);

/*
 * linattn_bwd -- gradients of L = sum(o * d_o) + sum(s_out * ds_out) for the
 * outputs of linattn_fwd.
 *
 *   d_o       [B, T, H, V] of `dtype`: the gradient of o
 *   s_in      as given to linattn_fwd (NULL: zero)
 *   ds_out    NULL (zero), or [B, H, K, V] float32: the gradient of s_out
 *   dq, dk    [B, T, H, K] of `grad_dtype` (float32 for float32 inputs, either
 *   dv        type for bfloat16 ones); [B, T, H, V] of `grad_dtype`.  Fully
 *             overwritten; zero behind a sequence's last token.
 *   ds_in     NULL, or [B, H, K, V] float32: the gradient of s_in; it may be
 *             ds_out itself.
 *   strides   NULL, or 21 values: as in linattn_fwd, of q, k, v, d_o, dq, dk
 *             and dv.  An input with a distance of 0 gets one gradient row for
 *             each place it is used at; their sum is the caller's.
 *   T == 0    ds_in receives ds_out (or zero).
 * Float32 gradients with K and V above 64 take up to 1398096 (batch, head)
 * pairs (else UNSUPPORTED).
 * The decays are constants of the model and get no gradient.  Everything else
 * as linattn_fwd, the precision by grad_dtype.  What is not finite in k can also
 * reach dq of the up to 31 tokens before its own; in q dk, and in d_o dv, of the
 * up to 31 behind (these two run from the last token to the first).
 */
int linattn_bwd(int64_t B, int64_t T, int64_t H, int64_t K, int64_t V, const void* q, const void* k, const void* v,
                const float* log_decay, float scale, const int32_t* lengths, const float* s_in, const void* d_o,
                const float* ds_out, void* dq, void* dk, void* dv, float* ds_in, const int64_t* strides, int dtype,
                int grad_dtype, void* workspace, size_t workspace_bytes, void* stream);

/* Workspace of a linattn_bwd call (0: none, or the arguments are invalid). */
size_t linattn_bwd_workspace_bytes(int64_t B, int64_t T, int64_t H, int64_t K, int64_t V, int dtype, int grad_dtype,
                                   int state_grad);

/* layout of linattn_rope */
#define LINATTN_ROPE_HALF        0  /* pairs (i, i + R/2) */
#define LINATTN_ROPE_INTERLEAVED 1  /* pairs (2i, 2i + 1) */

/*
 * linattn_rope -- rotary positions: pair i of the first R channels of every
 * head is turned by the angle position * freqs[i]:
 *
 *     (x, y) -> (x cos - y sin, x sin + y cos)
 *
 *   B, T, H, D, R   batch, tokens, heads, channels of a head (a multiple of 8
 *             up to LINATTN_MAX_HEAD) and rotated channels (even, from 2 to
 *             D); channels from R on are copied.  Fastest where R (half
 *             layout: R / 2) is a multiple of 8.  B * T is at most 2^27, H 2^20.
 *   q, k      [B, T, H, D] of `dtype`; k may be NULL (q alone is turned)
 *   q_out, k_out   the same shape and type; q_out may be q itself and k_out k
 *             itself (with the same strides), in place.
 *   positions NULL: token t has position start + t.  Else [B, T] int32,
 *             contiguous: its position is start + positions[b][t].
 *   start     added to every position, from -2^52 to 2^52 (else UNSUPPORTED).
 *             Angles are exact products, reduced before they are rounded: any
 *             position is turned as precisely as a near one.
 *   freqs     R / 2 float64 values on the device: radians per position.
 *             Scaling for longer contexts is a matter of these values.
 *   inverse   nonzero: turn by the negative angle (the gradient of the
 *             rotation: inputs are then gradients of the outputs)
 *   strides   NULL: contiguous.  Else 12 values: (batch, token, head)
 *             distances of q, k, q_out, k_out, as in linattn_fwd.
 */
int linattn_rope(int64_t B, int64_t T, int64_t H, int64_t D, int64_t R, const void* q, const void* k, void* q_out,
                 void* k_out, const int32_t* positions, int64_t start, const double* freqs, int layout, int inverse,
                 const int64_t* strides, int dtype, void* stream);

/*
 * linattn_rms_norm -- root-mean-square norm with the residual's addition:
 *
 *     h = x + residual  (rounded to `dtype`);   y = h / sqrt(mean(h^2) + eps) * weight
 *
 * with the mean over the C columns of each row.  The norm is that of h as it
 * is stored, so that linattn_rms_norm_bwd sees the same values.  Squares are
 * added up in float32: rows whose sum of squares leaves its range, 2^128, give
 * y = 0.
 *
 *   rows, C   C is a multiple of 8 up to LINATTN_MAX_COLUMNS; at most 2^25
 *             rows, or 2^21 of more than 1024 columns
 *   x, residual, h, y   [rows, C] of `dtype`, contiguous.  residual and h are
 *             both NULL (h = x) or both given; h may be x or residual itself.
 *   weight    C float32 values
 *   eps       finite, >= 0
 */
int linattn_rms_norm(int64_t rows, int64_t C, const void* x, const void* residual, const float* weight, float eps,
                     void* h, void* y, int dtype, void* stream);

/*
 * linattn_rms_norm_q8 -- the same with an 8-bit output: each group of columns
 * has the scale max|y| / 448 (at least 2^-126; 1 where every y is 0), and
 *
 *     codes = y / scale, rounded to the nearest e4m3 value (OCP e4m3fn, ties
 *     to even)
 *
 *   codes     [rows, C] bytes
 *   scales    [rows, groups] float32: groups = 1 for group == 0 (the whole
 *             row), or ceil(C / 128) for group == 128
 * A NaN counts for nothing in max|y|; its code is NaN.
 */
int linattn_rms_norm_q8(int64_t rows, int64_t C, const void* x, const void* residual, const float* weight, float eps,
                        void* h, void* codes, float* scales, int group, int dtype, void* stream);

/*
 * linattn_rms_norm_bwd -- gradients of sum(y * dy) + sum(h * dh) with respect
 * to h (and so to x and to residual alike) and to weight:
 *
 *     dx = (dy w - n mean(dy w n)) / rms + dh,   dweight = sum over rows of dy n,   n = h / rms
 *
 *   dy, h     [rows, C] of `dtype`: the gradient of y, and h of the forward
 *   dh        NULL (zero), or [rows, C] of `dtype`: the gradient that reaches
 *             h by the residual stream
 *   dx        [rows, C] of `dtype`; it may be dy or dh itself
 *   dweight   C float32 values, fully overwritten (zero when rows == 0)
 */
int linattn_rms_norm_bwd(int64_t rows, int64_t C, const void* dy, const void* h, const void* dh, const float* weight,
                         float eps, void* dx, float* dweight, int dtype, void* workspace, size_t workspace_bytes,
                         void* stream);

/* Workspace of a linattn_rms_norm_bwd call (partial sums of dweight). */
size_t linattn_rms_norm_bwd_workspace_bytes(int64_t rows, int64_t C, int dtype);

/* LINATTN_ABI_VERSION of the loaded library. */
int linattn_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* LINATTN_H */
