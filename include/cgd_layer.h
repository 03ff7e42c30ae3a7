/*
 * cgd_layer.h - C ABI of the operators that a layer needs beside the moves of
 * cgd.h and the products of cgd_experts.h: the norm that makes its input (bf16,
 * or the FP8 payload of a dispatch), low-rank adapters beside its projections,
 * dropout, and the gradient of its combine.
 *
 * The conventions are those of cgd_experts.h: device pointers, kernels enqueued
 * on `stream` only, nothing allocated, nothing synchronised, a cgd_status
 * returned and a message in cgd_last_error(). Workspaces need no initial
 * contents and keep nothing from call to call, so any two calls that may run at
 * the same time need two of them. Sums are fp32; no result depends on timing.
 */
#ifndef CGD_LAYER_H
#define CGD_LAYER_H

#include "cgd_experts.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Root-mean-square norm: s = x + residual, y = s / sqrt(mean(s^2) + eps) * weight, row by row.
 *   x             bf16 [num_rows, hidden]; residual the same or NULL
 *   weight        [hidden], weight_type CGD_DTYPE_BF16 or CGD_DTYPE_F32
 *   y             bf16 [num_rows, hidden] out, or NULL
 *   codes, scales FP8 e4m3 [num_rows, hidden] and [num_rows, hidden / 128] (fp32, or UE8M0 bytes for
 *                 scale_format 2) out, or NULL: y as cgd_cast_to_fp8 encodes it, but from fp32 values
 *   sum           bf16 [num_rows, hidden] out or NULL: s rounded (y is made from s before that)
 * At least one of y and codes. sum may be x or residual itself; the outputs share no other memory.
 * hidden: a multiple of 8 (FP8: of 128) up to 32768. A finite row whose squares add up to more than
 * fp32 holds gives zeros; one whose squares are too small for it is normed as any other, and only
 * zeros without eps are 0 / 0. All but scales 16-byte aligned. */
int cgd_rms_norm(const void* x, const void* residual, const void* weight, int weight_type, float eps, int64_t num_rows,
                 int hidden, void* y, void* codes, void* scales, int scale_format, void* sum, hipStream_t stream);

/* Its gradient at x, the values that were normed (with a residual: their sum, whose gradient is that
 * of both), also of rows whose squares are more, or less, than fp32 holds:
 *   grad_y        bf16 [num_rows, hidden]
 *   grad_sum      bf16 [num_rows, hidden] or NULL: what reaches the sum on another way, added
 *   grad_x        bf16 [num_rows, hidden] out or NULL; shares no memory with an input
 *   grad_weight   [hidden] of weight_type out or NULL, which needs the workspace */
size_t cgd_rms_norm_backward_workspace_bytes(int64_t num_rows, int hidden);
int cgd_rms_norm_backward(const void* grad_y, const void* x, const void* weight, int weight_type, float eps,
                          int64_t num_rows, int hidden, const void* grad_sum, void* grad_x, void* grad_weight,
                          void* workspace, size_t workspace_bytes, hipStream_t stream);

/* Low-rank adapters of many requests: out[t] = residual[t] + scale[j] * b[j] (a[j] x[t]), j = adapter_idx[t].
 *   x             bf16 [num_tokens, in_features]
 *   a, b          bf16 [num_adapters, rank, in_features], [num_adapters, out_features, rank]
 *   scale         fp32 [num_adapters] or NULL (1)
 *   adapter_idx   int64 [num_tokens]; outside [0, num_adapters): no adapter, out = residual or 0
 *   residual      bf16 [num_tokens, out_features] or NULL
 *   out           bf16 [num_tokens, out_features]; may be residual itself, no other input
 *   hidden        fp32 [num_tokens, rank] out or NULL: a[j] x[t] (0 without an adapter), as the
 *                 gradient takes it
 * a[j] x[t] is kept to 2^-16 of itself and out is rounded once. (Where it is a projection's residual,
 * cgd_linear rounds the sum of both once more.) rank: a multiple of 8 up to 256 (pad
 * smaller ones with zeros); num_adapters in [1,512]; num_tokens up to 2^26; in_features a multiple of 8
 * up to 2^20. x, a, b, residual, out and hidden 16-byte aligned. */
size_t cgd_adapter_linear_workspace_bytes(int64_t num_tokens, int num_adapters, int rank, int64_t in_features,
                                          int64_t out_features);
int cgd_adapter_linear(const void* x, const void* a, const void* b, const float* scale, const int64_t* adapter_idx,
                       int64_t num_tokens, int num_adapters, int rank, int64_t in_features, int64_t out_features,
                       const void* residual, void* out, float* hidden, void* workspace, size_t workspace_bytes,
                       hipStream_t stream);

/* Gradients, bf16, each may be NULL (not wanted): with gh[t] = scale[j] * b[j]^T grad_out[t],
 *   grad_x[t] = a[j]^T gh[t] (0 without an adapter), grad_a[j] = sum of gh[t] x[t]^T and
 *   grad_b[j] = sum of scale[j] grad_out[t] hidden[t]^T over j's tokens (0 without any).
 * The residual's gradient is grad_out. out_features: a multiple of 8. */
size_t cgd_adapter_linear_backward_workspace_bytes(int64_t num_tokens, int num_adapters, int rank, int64_t in_features,
                                                   int64_t out_features);
int cgd_adapter_linear_backward(const void* grad_out, const void* x, const void* a, const void* b, const float* scale,
                                const int64_t* adapter_idx, const float* hidden, int64_t num_tokens, int num_adapters,
                                int rank, int64_t in_features, int64_t out_features, void* grad_x, void* grad_a,
                                void* grad_b, void* workspace, size_t workspace_bytes, hipStream_t stream);

/* Dropout: out[i] = (u[i] >= limit ? x[i] * 65536 / (65536 - limit) : 0) + residual[i], bf16, where
 * limit = round(p * 65536) and u[i] are 16 bits of Philox4x32-10 (J. Salmon et al., 2011): elements
 * 8 v .. 8 v + 7 take the words of counter (v, offset) under the key `seed`, two to a word, the low half
 * first (64-bit numbers: low word first). The mask is nowhere stored: the gradient is this call on the
 * gradient, without residual. A dropped element is 0 whatever it held.
 *   state         int64 [2] on the device or NULL: added to seed and offset when the kernel runs, so
 *                 that a captured graph can be replayed with other numbers
 *   out           may be x or residual itself. p in [0, 1]. x, residual and out 16-byte aligned. */
int cgd_dropout(const void* x, const void* residual, int64_t num_elements, double p, uint64_t seed, uint64_t offset,
                const int64_t* state, void* out, hipStream_t stream);

/* Gradient of cgd_combine: for every slot (t, k) whose dst_row is a receive row,
 *   grad_expert_out[dst_row] = topk_weights[t, k] * grad_out[t]   (bf16 [recv_capacity, hidden])
 *   grad_topk_weights[t, k]  = <grad_out[t], expert_out[dst_row]> (fp32; 0 for other slots)
 * Receive rows that no slot names are left as they were; no two slots name one row (a dispatch gives
 * each its own). grad_expert_out shares no memory with an input. (The gradient of a dispatch is
 * cgd_combine with weights of 1.) */
int cgd_combine_backward(const void* grad_out, const void* expert_out, int64_t recv_capacity, int hidden,
                         const int32_t* dst_row, const float* topk_weights, int64_t num_tokens, int num_topk,
                         void* grad_expert_out, float* grad_topk_weights, hipStream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* CGD_LAYER_H */
