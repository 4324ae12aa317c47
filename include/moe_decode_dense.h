/*
 * moe_decode_dense.h -- a dense layer's gated feed-forward block, its backward pass,
 * and matrix products in 8-bit integers, for any number of rows.
 *
 * Models with mixture-of-experts layers have dense ones beside them, and linear maps
 * around both. The operators here run those as moe_decode_rows.h's run the experts:
 *
 *   moe_decode_quantise      rows -> 8-bit integers and one scale a row
 *   moe_decode_project_int8  a projection with a scale for each row and output channel
 *   moe_decode_ff            out = W2 (silu(Wg x) * (Wu x)) (+ residual)
 *   moe_decode_ff_backward   the gradients of x and of the weights
 *
 * What moe_decode_rows.h says of its calls holds for these: they keep no state, take
 * their workspace from the caller, enqueue on `stream` and return without waiting,
 * allocate nothing, can be captured in a CUDA graph, check their arguments on the host
 * (MOE_ERR_INVALID_ARG and MOE_ERR_UNSUPPORTED: nothing was enqueued), do not touch
 * rows beyond `rows`, and use the current device, which must be the buffers'.
 * moe_decode_rows_status reads from the workspace whether a call's device-side waits
 * ended in time. Results do not depend on the order in which blocks run: the same call
 * on the same device gives the same bits.
 */
#ifndef MOE_DECODE_DENSE_H
#define MOE_DECODE_DENSE_H

#include "moe_decode_rows.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Beside moe_dtype: rows that come as codes with a scale each. */
enum { MOE_I8 = 2 };
/* Beside moe_wdtype: 8-bit integers, fp32 scale for each row of the matrix (output channel). */
enum { MOE_W_INT8 = 3 };

/*
 * Rows of x to 8-bit integers:
 *   scale_t = fp32(max_k |x_tk| / 127)
 *   codes_tk = 127 x_tk / max_k |x_tk| to the nearest whole number, halves to the even one
 * The rounding is that of the exact quotient. A row of zeros has scale 0 and codes 0; a
 * row that holds a NaN or an infinity has scale NaN and codes 0, so that its products are NaN.
 *   dtype  moe_dtype of x: row r at x + r * x_stride elements
 *   codes  int8 [rows, inner]; scale fp32 [rows]
 * Supported: inner % 8 == 0, <= 65536; x and codes 16-byte aligned, x_stride a multiple of
 * 16 bytes. codes and scale share no byte with x.
 */
moe_status moe_decode_quantise(int32_t dtype, int32_t inner, const void* x, int64_t x_stride, int64_t rows,
                               int8_t* codes, float* scale, moe_stream_t stream);

/*
 * A projection in 8-bit integers:
 *   y_t[o] = s_t c_o sum_k q_tk W[o, k] (+ addend_t[o])
 *   out_t = y_t, or with swiglu silu(y_t[0..O)) * y_t[O..2O)
 * The products of the integers are exact; they are summed in fp32 (exact while the sums stay
 * below 2^24), and the result is rounded once to out_dtype.
 * x_dtype MOE_I8: x is int8 codes with x_scale fp32 [rows], as moe_decode_quantise makes them;
 * MOE_BF16 or MOE_F32: rows that the call quantises, by that definition (x_scale is not read).
 * Supported: inner % 16 == 0, outer % 8 == 0, both <= 65536.
 */
typedef struct moe_int8_config {
  int32_t inner;     /* K                                                 */
  int32_t outer;     /* O: columns of out                                 */
  int32_t swiglu;    /* 1: W has 2 O rows, gate rows first                */
  int32_t x_dtype;   /* MOE_I8, MOE_BF16 or MOE_F32                       */
  int32_t out_dtype; /* moe_dtype                                         */
} moe_int8_config;

moe_status moe_decode_project_int8_check(const moe_int8_config* cfg);
/* 0 for few rows of codes: such a call takes NULL, and has no device-side waits. */
moe_status moe_decode_project_int8_workspace(const moe_int8_config* cfg, int64_t rows, size_t* bytes);
/*
 *   w       int8 [O, K] ([2 O, K] with swiglu); w_scale fp32, one a row of w
 *   x       row r at x + r * x_stride elements; x_stride * element size a multiple of 16
 *   addend  bf16 [rows, O] or NULL; not with swiglu. May be out (out_dtype MOE_BF16)
 *   out     [rows, O] of out_dtype
 * x, w, w_scale, addend, out and workspace 16-byte aligned. Other overlaps of out with an input,
 * the weights among them, are refused.
 */
moe_status moe_decode_project_int8(const moe_int8_config* cfg, const int8_t* w, const float* w_scale, const void* x,
                                   const float* x_scale, int64_t x_stride, const void* addend, void* out,
                                   int64_t rows, void* workspace, size_t workspace_bytes, moe_stream_t stream);

/*
 * The gated feed-forward block of T rows, W13 = [Wg; Wu] [2 I, H], W2 [H, I]:
 *   [g; u]_t = W13 x_t,  h_t = silu(g_t) * u_t,  out_t = W2 h_t (+ residual_t)
 * with fp32 sums and one rounding to bf16. MOE_W_BF16: h is rounded to bf16 (it is an operand of
 * the tensor cores; of up to 4 rows, and of up to 16 where W13 has 16 MB at most, it is the sum of two
 * bf16 numbers: a row's last bits may depend on how many come with it). MOE_W_INT8: the codes of
 * x_t and of h_t (in fp32) are those of moe_decode_quantise.
 * Supported: hidden, inter % 8 == 0 (MOE_W_INT8: % 16), <= 65536.
 */
typedef struct moe_ff_config {
  int32_t hidden; /* H */
  int32_t inter;  /* I */
  int32_t wdtype; /* MOE_W_BF16 or MOE_W_INT8 */
} moe_ff_config;

typedef struct moe_ff_weights {
  const void* w13;
  const void* w2;
  const float* s13; /* MOE_W_INT8: fp32 [2 I] */
  const float* s2;  /* MOE_W_INT8: fp32 [H]   */
} moe_ff_weights;

moe_status moe_decode_ff_check(const moe_ff_config* cfg);
moe_status moe_decode_ff_workspace(const moe_ff_config* cfg, int64_t rows, size_t* bytes);
/*
 *   x         bf16 [rows, H], row r at x + r * x_stride elements (x_stride % 8 == 0)
 *   residual  bf16 [rows, H] or NULL; gate_up bf16 [rows, 2 I] or NULL: receives [g; u], rounded,
 *             for moe_decode_ff_backward (MOE_W_BF16 only)
 *   out       bf16 [rows, H]; may be the residual, and x (rows without gaps, x_stride H)
 * All addresses 16-byte aligned. Other overlaps of out or gate_up with an input (the weights among
 * them) or with each other are refused.
 */
moe_status moe_decode_ff(const moe_ff_config* cfg, const moe_ff_weights* weights, const void* x, int64_t x_stride,
                         const void* residual, void* gate_up, void* out, int64_t rows, void* workspace,
                         size_t workspace_bytes, moe_stream_t stream);

/*
 * The block's backward pass (MOE_W_BF16), from grad = d loss / d out and the kept gate_up:
 *   dh = W2^T grad,  dg = dh * u * silu'(g),  du = dh * silu(g),  h = silu(g) * u
 *   dx = W13^T [dg; du],  dW13 = sum_t [dg; du]_t x_t^T,  dW2 = sum_t grad_t h_t^T
 * with fp32 sums; dg, du and h are rounded to bf16 (operands of the tensor cores; of few rows of
 * a narrow block, up to 4096 values, they are the sums of two bf16 numbers, of which the second
 * makes NaN of an infinity that it meets in grad, x or a weight), dx to bf16. The
 * residual's gradient is grad itself. dx, dw13 and dw2 may be NULL: what is not wanted is not
 * computed. dw_dtype is the weight gradients' type; with MOE_F32 and accumulate they are added
 * to what dw13 and dw2 hold (gradients of several batches). With rows 0 dw13 and dw2 become zero
 * (accumulate: stay as they are).
 *   grad bf16 [rows, H] and x as for moe_decode_ff, each with a row stride of its own
 *   gate_up bf16 [rows, 2 I]; dx bf16 [rows, H]; dw13 [2 I, H], dw2 [H, I]
 * All addresses 16-byte aligned. Outputs share no byte with inputs or each other.
 */
moe_status moe_decode_ff_backward_workspace(const moe_ff_config* cfg, int64_t rows, size_t* bytes);
moe_status moe_decode_ff_backward(const moe_ff_config* cfg, const moe_ff_weights* weights, const void* grad,
                                  int64_t grad_stride, const void* x, int64_t x_stride, const void* gate_up, void* dx,
                                  void* dw13, void* dw2, int32_t dw_dtype, int32_t accumulate, int64_t rows,
                                  void* workspace, size_t workspace_bytes, moe_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* MOE_DECODE_DENSE_H */
