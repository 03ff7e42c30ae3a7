// C-ABI entry points of the norm, the adapters, dropout and combine's gradient:
// argument checks, workspace sizing, launches. Declarations and the contract of
// every call are in include/cgd_layer.h.
#include "cgd_layer.h"

#include <math.h>
#include <stdarg.h>
#include <stdio.h>

#include "cgd_launch.h"
#include "cgd_layer_launch.h"

namespace {

int fail(int code, const char* fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof(buf), fmt, ap);
    va_end(ap);
    return cgd::report(code, buf);
}

int done(hipError_t err, const char* what) {
    return err == hipSuccess ? CGD_OK : fail(CGD_ERR_HIP, "%s: %s", what, hipGetErrorString(err));
}

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int check_workspace(const void* ws, size_t have, size_t need) {
    if (need == 0) return CGD_OK;
    if (!ws || have < need || !aligned(ws, 256))
        return fail(CGD_ERR_WORKSPACE, "workspace needs %zu bytes, 256-byte aligned (got %zu)", need, have);
    return CGD_OK;
}

int check_norm(int64_t rows, int width, int weight_type, float eps) {
    if (rows < 0 || rows > INT32_MAX) return fail(CGD_ERR_INVALID_ARG, "num_rows must be in [0, INT32_MAX] (got %lld)", (long long)rows);
    if (width < 8 || width % 8 || width > cgd::kMaxNormWidth)
        return fail(CGD_ERR_INVALID_ARG, "hidden must be a multiple of 8 in [8,%d] (got %d)", cgd::kMaxNormWidth, width);
    if (weight_type != CGD_DTYPE_BF16 && weight_type != CGD_DTYPE_F32) return fail(CGD_ERR_INVALID_ARG, "weight must be bf16 or fp32");
    if (!(eps >= 0.0f) || !isfinite(eps)) return fail(CGD_ERR_INVALID_ARG, "eps must be finite and not negative");
    return CGD_OK;
}

int check_adapters(int64_t tokens, int adapters, int rank, int64_t in, int64_t out) {
    if (tokens < 0 || tokens > cgd::kMaxAdapterTokens)
        return fail(CGD_ERR_INVALID_ARG, "num_tokens must be in [0, 2^26] (got %lld)", (long long)tokens);
    if (adapters < 1 || adapters > cgd::kMaxExperts) return fail(CGD_ERR_INVALID_ARG, "num_adapters must be in [1,512] (got %d)", adapters);
    if (rank < 8 || rank % 8 || rank > cgd::kMaxRank)
        return fail(CGD_ERR_INVALID_ARG, "rank must be a multiple of 8 in [8,%d] (got %d)", cgd::kMaxRank, rank);
    if (in < 8 || in % 8 || in > (int64_t(1) << 20))
        return fail(CGD_ERR_INVALID_ARG, "in_features must be a positive multiple of 8 up to 2^20 (got %lld)", (long long)in);
    if (out < 1 || out > (int64_t(1) << 20)) return fail(CGD_ERR_INVALID_ARG, "out_features must be in [1, 2^20] (got %lld)", (long long)out);
    return CGD_OK;
}

}  // namespace

extern "C" {

int cgd_rms_norm(const void* x, const void* residual, const void* weight, int weight_type, float eps, int64_t num_rows,
                 int hidden, void* y, void* codes, void* scales, int scale_format, void* sum, hipStream_t stream) {
    const int rc = check_norm(num_rows, hidden, weight_type, eps);
    if (rc) return rc;
    if (!weight || (num_rows > 0 && !x)) return fail(CGD_ERR_INVALID_ARG, "null x or weight");
    if (num_rows > 0 && !y && !codes) return fail(CGD_ERR_INVALID_ARG, "neither y nor codes");
    if (!codes != !scales && num_rows > 0) return fail(CGD_ERR_INVALID_ARG, "codes and scales go together");
    if (sum && !residual && num_rows > 0) return fail(CGD_ERR_INVALID_ARG, "sum goes with residual");
    if (!aligned(x, 16) || !aligned(residual, 16) || !aligned(weight, 16) || !aligned(y, 16) || !aligned(codes, 16) || !aligned(sum, 16))
        return fail(CGD_ERR_INVALID_ARG, "x, residual, weight, y, codes and sum must be 16-byte aligned");
    if (codes) {
        if (hidden % 128) return fail(CGD_ERR_INVALID_ARG, "hidden must be a multiple of 128 for FP8 (got %d)", hidden);
        if (scale_format < CGD_SCALE_F32 || scale_format > CGD_SCALE_UE8M0)
            return fail(CGD_ERR_INVALID_ARG, "scale_format must be 0, 1 or 2 (got %d)", scale_format);
        if (!aligned(scales, scale_format == CGD_SCALE_UE8M0 ? 1 : 4)) return fail(CGD_ERR_INVALID_ARG, "misaligned scales");
    }
    cgd::NormArgs a;
    a.x = static_cast<const uint16_t*>(x);
    a.residual = static_cast<const uint16_t*>(residual);
    a.weight = weight;
    a.weight_f32 = weight_type == CGD_DTYPE_F32;
    a.eps = eps;
    a.rows = num_rows;
    a.width = hidden;
    a.y = static_cast<uint16_t*>(y);
    a.codes = static_cast<uint8_t*>(codes);
    a.scales = scales;
    a.format = scale_format;
    a.sum = static_cast<uint16_t*>(sum);
    return done(cgd::launch_norm(a, stream), "norm launch");
}

size_t cgd_rms_norm_backward_workspace_bytes(int64_t num_rows, int hidden) {
    if (check_norm(num_rows, hidden, CGD_DTYPE_F32, 0.0f)) return 0;
    return (size_t)cgd::norm_grad_blocks(num_rows, hidden) * hidden * 4;
}

int cgd_rms_norm_backward(const void* grad_y, const void* x, const void* weight, int weight_type, float eps,
                          int64_t num_rows, int hidden, const void* grad_sum, void* grad_x, void* grad_weight,
                          void* workspace, size_t workspace_bytes, hipStream_t stream) {
    int rc = check_norm(num_rows, hidden, weight_type, eps);
    if (rc) return rc;
    if (!weight || (num_rows > 0 && (!x || !grad_y))) return fail(CGD_ERR_INVALID_ARG, "null grad_y, x or weight");
    if (!aligned(x, 16) || !aligned(grad_y, 16) || !aligned(weight, 16) || !aligned(grad_sum, 16) || !aligned(grad_x, 16) ||
        !aligned(grad_weight, weight_type == CGD_DTYPE_F32 ? 4 : 2))
        return fail(CGD_ERR_INVALID_ARG, "grad_y, x, weight, grad_sum and grad_x must be 16-byte aligned");
    if (grad_weight) {
        rc = check_workspace(workspace, workspace_bytes, cgd_rms_norm_backward_workspace_bytes(num_rows, hidden));
        if (rc) return rc;
    }
    cgd::NormGradArgs a;
    a.grad = static_cast<const uint16_t*>(grad_y);
    a.x = static_cast<const uint16_t*>(x);
    a.weight = weight;
    a.weight_f32 = weight_type == CGD_DTYPE_F32;
    a.eps = eps;
    a.rows = num_rows;
    a.width = hidden;
    a.grad_sum = static_cast<const uint16_t*>(grad_sum);
    a.grad_x = static_cast<uint16_t*>(grad_x);
    a.partial = grad_weight ? static_cast<float*>(workspace) : nullptr;
    a.grad_weight = grad_weight;
    return done(cgd::launch_norm_grad(a, stream), "norm gradient launch");
}

int cgd_dropout(const void* x, const void* residual, int64_t num_elements, double p, uint64_t seed, uint64_t offset,
                const int64_t* state, void* out, hipStream_t stream) {
    if (num_elements < 0) return fail(CGD_ERR_INVALID_ARG, "num_elements must not be negative (got %lld)", (long long)num_elements);
    if (!(p >= 0.0 && p <= 1.0)) return fail(CGD_ERR_INVALID_ARG, "p must be in [0, 1] (got %g)", p);
    if (num_elements > 0 && (!x || !out)) return fail(CGD_ERR_INVALID_ARG, "null x or out");
    if (!aligned(x, 16) || !aligned(residual, 16) || !aligned(out, 16))
        return fail(CGD_ERR_INVALID_ARG, "x, residual and out must be 16-byte aligned");
    if (!aligned(state, 8)) return fail(CGD_ERR_INVALID_ARG, "misaligned state");
    cgd::DropoutArgs a;
    a.x = static_cast<const uint16_t*>(x);
    a.residual = static_cast<const uint16_t*>(residual);
    a.out = static_cast<uint16_t*>(out);
    a.n = num_elements;
    a.limit = (uint32_t)floor(p * 65536.0 + 0.5);
    a.scale = a.limit < 65536 ? (float)(65536.0 / (65536 - a.limit)) : 0.0f;
    a.seed = seed;
    a.offset = offset;
    a.state = state;
    return done(cgd::launch_dropout(a, stream), "dropout launch");
}

int cgd_combine_backward(const void* grad_out, const void* expert_out, int64_t recv_capacity, int hidden,
                         const int32_t* dst_row, const float* topk_weights, int64_t num_tokens, int num_topk,
                         void* grad_expert_out, float* grad_topk_weights, hipStream_t stream) {
    if (num_tokens < 0 || num_tokens > INT32_MAX)
        return fail(CGD_ERR_INVALID_ARG, "num_tokens must be in [0, INT32_MAX] (got %lld)", (long long)num_tokens);
    if (num_topk < 1 || num_topk > cgd::kMaxTopk) return fail(CGD_ERR_INVALID_ARG, "num_topk must be in [1,16] (got %d)", num_topk);
    if (hidden < 8 || hidden % 8) return fail(CGD_ERR_INVALID_ARG, "hidden must be a positive multiple of 8 (got %d)", hidden);
    if (recv_capacity < 0 || recv_capacity > INT32_MAX)
        return fail(CGD_ERR_INVALID_ARG, "recv_capacity must be in [0, INT32_MAX] (got %lld)", (long long)recv_capacity);
    if (num_tokens > 0 && (!grad_out || !dst_row || !topk_weights || !grad_topk_weights))
        return fail(CGD_ERR_INVALID_ARG, "null grad_out, dst_row, topk_weights or grad_topk_weights");
    if (num_tokens > 0 && recv_capacity > 0 && (!expert_out || !grad_expert_out))
        return fail(CGD_ERR_INVALID_ARG, "null expert_out or grad_expert_out");
    if (!aligned(grad_out, 16) || !aligned(expert_out, 16) || !aligned(grad_expert_out, 16))
        return fail(CGD_ERR_INVALID_ARG, "grad_out, expert_out and grad_expert_out must be 16-byte aligned");
    if (!aligned(dst_row, 4) || !aligned(topk_weights, 4) || !aligned(grad_topk_weights, 4))
        return fail(CGD_ERR_INVALID_ARG, "misaligned pointer");
    cgd::CombineGradArgs a;
    a.grad = static_cast<const uint16_t*>(grad_out);
    a.y = static_cast<const uint16_t*>(expert_out);
    a.capacity = recv_capacity;
    a.width = hidden;
    a.dst_row = dst_row;
    a.weights = topk_weights;
    a.tokens = num_tokens;
    a.topk = num_topk;
    a.grad_y = static_cast<uint16_t*>(grad_expert_out);
    a.grad_weights = grad_topk_weights;
    return done(cgd::launch_combine_grad(a, stream), "combine gradient launch");
}

size_t cgd_adapter_linear_workspace_bytes(int64_t num_tokens, int num_adapters, int rank, int64_t in_features,
                                          int64_t out_features) {
    if (check_adapters(num_tokens, num_adapters, rank, in_features, out_features)) return 0;
    return cgd::adapter_workspace_bytes(num_tokens, num_adapters, rank, in_features, out_features);
}

int cgd_adapter_linear(const void* x, const void* a, const void* b, const float* scale, const int64_t* adapter_idx,
                       int64_t num_tokens, int num_adapters, int rank, int64_t in_features, int64_t out_features,
                       const void* residual, void* out, float* hidden, void* workspace, size_t workspace_bytes,
                       hipStream_t stream) {
    int rc = check_adapters(num_tokens, num_adapters, rank, in_features, out_features);
    if (rc) return rc;
    if (!a || !b || (num_tokens > 0 && (!x || !adapter_idx || !out))) return fail(CGD_ERR_INVALID_ARG, "null x, a, b, adapter_idx or out");
    if (!aligned(x, 16) || !aligned(a, 16) || !aligned(b, 16) || !aligned(residual, 16) || !aligned(out, 16) || !aligned(hidden, 16))
        return fail(CGD_ERR_INVALID_ARG, "x, a, b, residual, out and hidden must be 16-byte aligned");
    if (!aligned(adapter_idx, 8) || !aligned(scale, 4)) return fail(CGD_ERR_INVALID_ARG, "misaligned adapter_idx or scale");
    rc = check_workspace(workspace, workspace_bytes, cgd::adapter_workspace_bytes(num_tokens, num_adapters, rank, in_features, out_features));
    if (rc) return rc;
    cgd::AdapterArgs p;
    p.x = static_cast<const uint16_t*>(x);
    p.a = static_cast<const uint16_t*>(a);
    p.b = static_cast<const uint16_t*>(b);
    p.scale = scale;
    p.index = adapter_idx;
    p.tokens = num_tokens;
    p.in = in_features;
    p.out_features = out_features;
    p.adapters = num_adapters;
    p.rank = rank;
    p.residual = static_cast<const uint16_t*>(residual);
    p.out = static_cast<uint16_t*>(out);
    p.hidden = hidden;
    return done(cgd::launch_adapters(p, workspace, stream), "adapter launch");
}

size_t cgd_adapter_linear_backward_workspace_bytes(int64_t num_tokens, int num_adapters, int rank, int64_t in_features,
                                                   int64_t out_features) {
    if (check_adapters(num_tokens, num_adapters, rank, in_features, out_features)) return 0;
    return cgd::adapter_grad_workspace_bytes(num_tokens, num_adapters, rank, in_features, out_features);
}

int cgd_adapter_linear_backward(const void* grad_out, const void* x, const void* a, const void* b, const float* scale,
                                const int64_t* adapter_idx, const float* hidden, int64_t num_tokens, int num_adapters,
                                int rank, int64_t in_features, int64_t out_features, void* grad_x, void* grad_a,
                                void* grad_b, void* workspace, size_t workspace_bytes, hipStream_t stream) {
    int rc = check_adapters(num_tokens, num_adapters, rank, in_features, out_features);
    if (rc) return rc;
    if (out_features % 8) return fail(CGD_ERR_INVALID_ARG, "gradients need out_features to be a multiple of 8 (got %lld)", (long long)out_features);
    if (!a || !b || (num_tokens > 0 && (!grad_out || !adapter_idx))) return fail(CGD_ERR_INVALID_ARG, "null grad_out, a, b or adapter_idx");
    if (num_tokens > 0 && ((grad_a && !x) || (grad_b && !hidden))) return fail(CGD_ERR_INVALID_ARG, "grad_a needs x, grad_b needs hidden");
    if (!aligned(grad_out, 16) || !aligned(x, 16) || !aligned(a, 16) || !aligned(b, 16) || !aligned(grad_x, 16) ||
        !aligned(grad_a, 16) || !aligned(grad_b, 16))
        return fail(CGD_ERR_INVALID_ARG, "grad_out, x, a, b and the gradients must be 16-byte aligned");
    if (!aligned(adapter_idx, 8) || !aligned(scale, 4) || !aligned(hidden, 4))
        return fail(CGD_ERR_INVALID_ARG, "misaligned adapter_idx, scale or hidden");
    rc = check_workspace(workspace, workspace_bytes, cgd::adapter_grad_workspace_bytes(num_tokens, num_adapters, rank, in_features, out_features));
    if (rc) return rc;
    cgd::AdapterGradArgs p;
    p.grad = static_cast<const uint16_t*>(grad_out);
    p.x = static_cast<const uint16_t*>(x);
    p.a = static_cast<const uint16_t*>(a);
    p.b = static_cast<const uint16_t*>(b);
    p.scale = scale;
    p.index = adapter_idx;
    p.hidden = hidden;
    p.tokens = num_tokens;
    p.in = in_features;
    p.out_features = out_features;
    p.adapters = num_adapters;
    p.rank = rank;
    p.grad_x = static_cast<uint16_t*>(grad_x);
    p.grad_a = static_cast<uint16_t*>(grad_a);
    p.grad_b = static_cast<uint16_t*>(grad_b);
    return done(cgd::launch_adapters_grad(p, workspace, stream), "adapter gradient launch");
}

}  // extern "C"
