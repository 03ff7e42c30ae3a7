/*
 * cgd_experts.h - C ABI of libcgd's computing operators, which stand before,
 * between and after the moves of cgd.h: the router that makes topk_idx and
 * topk_weights, the experts' products over the rows that dispatch delivers,
 * and the dense product of a gate or a shared expert.
 *
 * The conventions are those of cgd.h: device pointers, kernels enqueued on
 * `stream` only, nothing allocated, nothing synchronised, a cgd_status
 * returned and a message in cgd_last_error(). Workspaces here need no initial
 * contents and keep nothing from call to call, so any two calls that may run
 * at the same time need two of them.
 */
#ifndef CGD_EXPERTS_H
#define CGD_EXPERTS_H

#include "cgd.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { CGD_DTYPE_BF16 = 0, CGD_DTYPE_F32 = 1, CGD_DTYPE_FP8 = 2 } cgd_dtype;
typedef enum { CGD_SCORE_SOFTMAX = 0, CGD_SCORE_SIGMOID = 1 } cgd_scoring;
typedef enum {
    CGD_ACT_NONE = 0,
    CGD_ACT_RELU = 1,
    CGD_ACT_SILU = 2,
    CGD_ACT_GELU = 3,  /* 0.5 v (1 + erf(v / sqrt 2)) */
    CGD_ACT_SWIGLU = 4 /* silu(gate) * up: the weight holds out_features gate rows, then out_features up rows */
} cgd_activation;

/* Router: the experts of each token and their weights.
 *   logits        [num_tokens, num_experts], logits_type CGD_DTYPE_F32 or CGD_DTYPE_BF16;
 *                 NaN counts as -inf, +inf as the largest finite value
 *   scoring       score s = softmax over the token's logits, or sigmoid of each
 *   bias          fp32 [num_experts] or NULL: added to the score for the choice only
 *   num_groups    divides num_experts, at most 64. With num_topk_groups < num_groups only the
 *                 experts of the best groups can be chosen; a group's value is the sum of its
 *                 group_score_topk (1 or 2) largest choice values
 *   renormalize   weights are divided by their sum over the token's chosen experts
 *   scale         multiplies every weight
 *   topk_idx      int64 [num_tokens, num_topk] out, by descending choice value, ties to the lower
 *                 index; topk_weights fp32 [num_tokens, num_topk] out. An expert whose logit or
 *                 choice value is -inf (or NaN) is never chosen: slots left over hold -1 and 0
 * The choice value is s + bias in 64 bits; without a bias, and without groups or with
 * group_score_topk 1, it is the logit. num_topk in [1,16], num_experts in [1,512]. */
int cgd_route(const void* logits, int logits_type, int64_t num_tokens, int num_experts, int num_topk, int scoring,
              const float* bias, int num_groups, int num_topk_groups, int group_score_topk, int renormalize,
              float scale, int64_t* topk_idx, float* topk_weights, hipStream_t stream);

/* Gradient of topk_weights with respect to the logits (the choice itself has none):
 *   grad_topk_weights fp32 [num_tokens, num_topk]; topk_idx as cgd_route gave it (entries outside
 *   [0, num_experts) are no slot; an expert in several slots collects all of them)
 *   grad_logits [num_tokens, num_experts] of logits_type, every element written. */
int cgd_route_backward(const float* grad_topk_weights, const void* logits, int logits_type, const int64_t* topk_idx,
                       int64_t num_tokens, int num_experts, int num_topk, int scoring, int renormalize, float scale,
                       void* grad_logits, hipStream_t stream);

/* Dense product with its epilogue: out = act(x W^T + bias) + residual.
 *   x             [num_tokens, in_features], x_type CGD_DTYPE_BF16 or CGD_DTYPE_FP8
 *   x_scales      FP8: one scale for 128 values of a row at x_scales + row * scale_row_stride +
 *                 block * scale_block_stride (elements; fp32, or UE8M0 bytes for scale_format 2)
 *   weight        [rows, in_features] of x's type, rows = out_features, or 2 * out_features for SwiGLU
 *   weight_scales FP8: fp32 [ceil(rows / 128), in_features / 128], one for each block of 128 x 128
 *   bias          bf16 [rows] or NULL; residual bf16 [num_tokens, out_features] or NULL
 *   out           [num_tokens, out_features], out_type CGD_DTYPE_BF16, or CGD_DTYPE_F32 for bf16 x;
 *                 may be residual itself (bf16), no other input
 *   preact        bf16 [num_tokens, rows] or NULL: x W^T + bias, as cgd_linear_backward takes it
 * Sums are fp32, rounded once (FP8: the matrix unit adds 8 neighbouring products at a time and cuts
 * each 13 bits below the largest of them, under 2^-10 of it all told; these sums are fp32).
 * in_features: a multiple of 8 (FP8: of 128) up to 2^20; FP8 SwiGLU:
 * out_features a multiple of 128. x, weight, residual, out and preact 16-byte aligned. */
size_t cgd_linear_workspace_bytes(int64_t num_tokens, int64_t in_features, int64_t out_features, int activation,
                                  int x_type);
int cgd_linear(const void* x, int x_type, const void* x_scales, int64_t scale_row_stride, int64_t scale_block_stride,
               int scale_format, const void* weight, const float* weight_scales, int64_t num_tokens,
               int64_t in_features, int64_t out_features, const void* bias, int activation, const void* residual,
               void* out, int out_type, void* preact, void* workspace, size_t workspace_bytes, hipStream_t stream);

/* The same for each group of rows with a weight of its own: the experts' products.
 *   x             [num_rows, in_features]; weight [num_groups, rows, in_features]; weight_scales
 *                 [num_groups, ceil(rows / 128), in_features / 128]; bias [num_groups, rows]
 *   group_offset  int32 [num_groups + 1]: group e is rows [offset[e], offset[e+1]) (expert_offset
 *                 of a dispatch), non-decreasing within [0, num_rows]; or NULL: group e is rows
 *                 [e * group_capacity, (e+1) * group_capacity) (the packed layout), num_rows =
 *                 num_groups * group_capacity
 *   group_count   int32 [num_groups] or NULL: only the first count[e] rows of group e hold data
 *                 (num_tokens_per_expert; packed_recv_count)
 *   out           bf16 [num_rows, out_features]; rows that hold no data are left as they were
 * num_groups in [1,512], num_rows <= INT32_MAX. */
size_t cgd_grouped_linear_workspace_bytes(int64_t num_rows, int num_groups, int64_t group_capacity,
                                          int64_t in_features, int64_t out_features, int activation, int x_type);
int cgd_grouped_linear(const void* x, int x_type, const void* x_scales, int64_t scale_row_stride,
                       int64_t scale_block_stride, int scale_format, const void* weight, const float* weight_scales,
                       int64_t num_rows, int num_groups, const int32_t* group_offset, int64_t group_capacity,
                       const int32_t* group_count, int64_t in_features, int64_t out_features, const void* bias,
                       int activation, void* out, void* preact, void* workspace, size_t workspace_bytes,
                       hipStream_t stream);

/* Gradients, bf16: with d = grad_out * act'(preact) (rounded to bf16 once),
 *   grad_x = d W, grad_weight = d^T x, grad_bias = sum of d's rows (from fp32).
 * grad_x, grad_weight and grad_bias may each be NULL (not wanted). preact is needed with an
 * activation. The residual's gradient is grad_out. A group without rows gets zero gradients; rows
 * of grad_x that hold no data are left as they were. With an activation, grad_bias or
 * weight rows that are no multiple of 8, up to about 2^29 rows; what no launch holds is refused. */
size_t cgd_linear_backward_workspace_bytes(int64_t num_tokens, int64_t in_features, int64_t out_features,
                                           int activation, int bias_grad);
int cgd_linear_backward(const void* grad_out, const void* x, const void* weight, int64_t num_tokens,
                        int64_t in_features, int64_t out_features, const void* preact, int activation, void* grad_x,
                        void* grad_weight, void* grad_bias, void* workspace, size_t workspace_bytes,
                        hipStream_t stream);
size_t cgd_grouped_linear_backward_workspace_bytes(int64_t num_rows, int num_groups, int64_t in_features,
                                                   int64_t out_features, int activation, int bias_grad);
int cgd_grouped_linear_backward(const void* grad_out, const void* x, const void* weight, int64_t num_rows,
                                int num_groups, const int32_t* group_offset, int64_t group_capacity,
                                const int32_t* group_count, int64_t in_features, int64_t out_features,
                                const void* preact, int activation, void* grad_x, void* grad_weight, void* grad_bias,
                                void* workspace, size_t workspace_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* CGD_EXPERTS_H */
