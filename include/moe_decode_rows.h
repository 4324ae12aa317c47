/*
 * moe_decode_rows.h -- the MoE layer's operators for any number of rows.
 *
 * moe_decode.h computes a layer step for 1..16 token rows as one call. The
 * operators here are the same layer's parts for batches of any size -- a chunk of
 * a prompt, the rows of many requests -- over the same weights:
 *
 *   moe_decode_route    router logits -> chosen experts and their weights
 *   moe_decode_experts  the chosen (and the shared) experts' SwiGLU MLPs,
 *                       weighted, added to the residual
 *   moe_decode_project  one projection that all rows share, beside it a low-rank
 *                       adapter per row (requests with adapters of their own)
 *
 * Addresses are multiples of 16 where it says so below, and of their type elsewhere.
 * They keep no state: every call gets its buffers, and the workspace that two of
 * them need, from the caller. Calls may run at the same time on different streams
 * or threads when their workspaces and outputs are different memory. Each enqueues its work on
 * `stream` and returns without waiting, allocates nothing, and can be captured in a
 * CUDA graph (the graph then owns the workspace: two graphs that may run at the
 * same time need one each). Arguments are checked on the host: a call that
 * returns MOE_ERR_INVALID_ARG or MOE_ERR_UNSUPPORTED has enqueued nothing. After
 * MOE_ERR_CUDA (a launch failed) a part of its work may be on the stream, and its
 * outputs are undefined. Rows beyond `rows` are not touched.
 * The calls use the current CUDA device, which must be the buffers'.
 */
#ifndef MOE_DECODE_ROWS_H
#define MOE_DECODE_ROWS_H

#include "moe_decode.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum moe_dtype { MOE_BF16 = 0, MOE_F32 = 1 } moe_dtype;

/* Scores of moe_decode_route. */
typedef enum moe_route_score {
  MOE_ROUTE_SOFTMAX = 0, /* s_e = exp(l_e) / sum_i exp(l_i), over the row's unmasked experts */
  MOE_ROUTE_SIGMOID = 1  /* s_e = 1 / (1 + exp(-l_e))                                        */
} moe_route_score;

/*
 * Routing of T rows of logits l [T, E]:
 *   key_e = s_e + bias_e (bias NULL: s_e); the bias steers the choice only
 *   groups: the experts form num_groups groups of E / num_groups neighbours. A
 *     group's value is the sum of its group_best (1 or 2) largest keys; the
 *     top_groups groups of largest value are kept, the other groups' experts are
 *     out of the choice. num_groups = 1 (or top_groups = num_groups): no groups.
 *   the top_k largest keys are chosen, in descending order
 *   w_j = scale * s_j / sum_chosen s_i (renormalise), or scale * s_j
 * Ties, among experts and among groups, go to the lower index. Where keys in fp32 cannot tell
 * two candidates apart, the row is decided in fp64. Without a bias experts are ordered by
 * their logits, and so are groups of one best key (also where 64 bits hold the scores as equal).
 * A logit that is NaN or at most -1e38 masks its expert (-inf and the lowest
 * bf16 / fp32 value do): it is never chosen. A row with fewer than top_k experts
 * to choose from fills up with index -1 and weight 0. Logits above 3e38 count as 3e38.
 * An expert whose bias is -inf or NaN is not chosen either.
 * Supported: 1 <= E <= 1024, top_k <= 16, num_groups <= 32 and dividing E,
 * top_k <= top_groups * E / num_groups.
 */
typedef struct moe_route_config {
  int32_t num_experts;
  int32_t top_k;
  int32_t score;        /* moe_route_score              */
  int32_t num_groups;
  int32_t top_groups;
  int32_t group_best;   /* 1 or 2                       */
  int32_t renormalise;
  int32_t logits_dtype; /* moe_dtype                    */
  float scale;          /* finite                       */
} moe_route_config;

moe_status moe_decode_route_check(const moe_route_config* cfg);
/*
 *   logits      [rows, E] of logits_dtype, row r at logits + r * logits_stride elements
 *   bias        fp32 [E] or NULL
 *   topk_idx    int32 [rows, top_k]; topk_w fp32 [rows, top_k]
 */
moe_status moe_decode_route(const moe_route_config* cfg, const void* logits, int64_t logits_stride,
                            const float* bias, int64_t rows, int32_t* topk_idx, float* topk_w,
                            moe_stream_t stream);

/*
 * The experts' products of T rows:
 *   out_t = bf16_rne(r_t + sum_j w_tj y_e(x_t) + sum_s y_s(x_t)),  e = idx_tj,
 *   y(x) = W2 bf16_rne(silu(Wg x) * (Wu x))
 * with fp32 sums. An index outside 0..E-1 (-1 from moe_decode_route, padding) takes no part; an
 * expert that a row names twice counts twice. The intermediate row is rounded to
 * bf16 (it is an operand of the tensor cores), silu is off by at most 2^-16 of itself
 * before that; FP8 weights are rounded to bf16 after their block scale. (moe_decode_run keeps
 * all three in fp32: its outputs are 1.66e-3 off the exact ones relative to their norm, the
 * output's own rounding, and these 1.75e-3, with FP8 weights 2.0e-3.) The weights are those of moe_decode_create with
 * w2_layout MOE_W2_H_I; the router's are not used.
 * Supported: 1 <= E <= 1024, 0 <= S <= 4, 1 <= top_k <= 16; bf16: hidden, inter % 8 == 0;
 * FP8: % 128; NVFP4: % 256; hidden, inter <= 16384.
 */
typedef struct moe_experts_config {
  int32_t hidden;
  int32_t inter;
  int32_t num_experts;
  int32_t top_k;
  int32_t num_shared;
  int32_t wdtype;         /* moe_wdtype            */
  int32_t residual_dtype; /* moe_dtype of residual */
} moe_experts_config;

moe_status moe_decode_experts_check(const moe_experts_config* cfg);
/*
 * Bytes of workspace that a call with at most `rows` rows needs: for each of the pairs of a
 * row and a chosen or shared expert 4 H + 2 I bytes and a few more, for 16384 rows at most (a
 * longer call goes through its rows in rounds). 1.7 GB for 16384 rows with H = 2560, I = 768,
 * 8 + 1 experts; 32 GB at the limits above.
 */
moe_status moe_decode_experts_workspace(const moe_experts_config* cfg, int64_t rows, size_t* bytes);
/*
 *   x        bf16 [rows, H], row r at x + r * x_stride elements (x_stride % 8 == 0, >= H)
 *   idx, w   int32 / fp32 [rows, top_k]
 *   residual [rows, H] of residual_dtype or NULL (zero); out bf16 [rows, H], may be a bf16 residual
 * x, residual, out and workspace 16-byte aligned. out may be x as well (rows without gaps,
 * x_stride H); any other overlap of out with x or the residual is refused.
 */
moe_status moe_decode_experts(const moe_experts_config* cfg, const moe_decode_weights* weights, const void* x,
                              int64_t x_stride, const int32_t* idx, const float* w, const void* residual,
                              void* out, int64_t rows, void* workspace, size_t workspace_bytes,
                              moe_stream_t stream);

/*
 * A projection that all rows share, with the rows' adapters beside it:
 *   y_t = W x_t + B_a (scale_a A_a x_t) (+ addend_t),  a = adapter_ids[t]
 *   out_t = y_t, or with swiglu silu(y_t[0..O)) * y_t[O..2O)
 * with fp32 sums, rounded once to out_dtype (silu as above). With many rows scale_a A_a x_t is held
 * as the sum of two bf16 numbers (operands of the tensor cores), and an NVFP4 weight
 * is rounded to bf16 after both its scales. Rows whose id is outside 0..num_adapters-1 have no adapter. Rows
 * may come in any order. What an adapter holds reaches its own rows only.
 * Supported: inner % 8 == 0, outer even (FP8: both % 128, NVFP4: % 256), <= 16384;
 * rank % 8 == 0, <= 256; num_adapters <= 1024 (0: no adapters, their arguments are not read).
 */
typedef struct moe_project_config {
  int32_t inner;        /* K                                             */
  int32_t outer;        /* O: columns of out                             */
  int32_t swiglu;       /* 1: W, B have 2 O rows, gate rows first        */
  int32_t wdtype;       /* moe_wdtype of W                               */
  int32_t rank;
  int32_t num_adapters;
  int32_t out_dtype;    /* moe_dtype (swiglu: MOE_BF16)                  */
} moe_project_config;

typedef struct moe_project_weights {
  const void* w;         /* [O, K] ([2 O, K] with swiglu), as w13 / w2 of one expert */
  const void* w_scale;   /* FP8 / NVFP4 block scales                                 */
  const float* w_gscale; /* NVFP4 tensor scale: 1 value, with swiglu 2               */
  const void* a;         /* bf16 [L, rank, K]                                        */
  const void* b;         /* bf16 [L, O, rank] ([L, 2 O, rank] with swiglu)           */
  const float* scale;    /* fp32 [L] or NULL (1)                                     */
} moe_project_weights;

moe_status moe_decode_project_check(const moe_project_config* cfg);
moe_status moe_decode_project_workspace(const moe_project_config* cfg, int64_t rows, size_t* bytes);
/*
 *   x           bf16 [rows, K], row r at x + r * x_stride elements (x_stride % 8 == 0, >= K)
 *   adapter_ids int32 [rows]
 *   addend      bf16 [rows, O] or NULL; not with swiglu. May be out (out_dtype MOE_BF16)
 *   out         [rows, O] of out_dtype
 * x, addend, out, workspace and the weights 16-byte aligned; an overlap of out with x, or
 * another one with addend, is refused.
 */
moe_status moe_decode_project(const moe_project_config* cfg, const moe_project_weights* weights, const void* x,
                              int64_t x_stride, const int32_t* adapter_ids, const void* addend, void* out,
                              int64_t rows, void* workspace, size_t workspace_bytes, moe_stream_t stream);

/*
 * Synchronises `stream` and reports on the last call of one row or more that used
 * `workspace`, whose first 4096 bytes it reads (MOE_ERR_INVALID_ARG for a stream under
 * capture):
 * MOE_ERR_DEVICE_TIMEOUT when one of its device-side waits ran into its limit
 * (its outputs are undefined then), MOE_OK otherwise.
 */
moe_status moe_decode_rows_status(const void* workspace, moe_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* MOE_DECODE_ROWS_H */
