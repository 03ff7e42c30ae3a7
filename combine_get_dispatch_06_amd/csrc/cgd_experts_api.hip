// C-ABI entry points of the router and of the dense and grouped products:
// argument checks, workspace sizing, launches. Declarations and the contract of
// every call are in include/cgd_experts.h.
#include "cgd_experts.h"

#include <stdarg.h>
#include <stdio.h>

#include "cgd_experts_launch.h"
#include "cgd_launch.h"

namespace {

int fail(int code, const char* fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof(buf), fmt, ap);
    va_end(ap);
    return cgd::report(code, buf);
}

int hip_fail(hipError_t err, const char* what) { return fail(CGD_ERR_HIP, "%s: %s", what, hipGetErrorString(err)); }

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

constexpr int64_t kMaxFeatures = int64_t(1) << 20;

int check_route(int64_t T, int E, int K, int type, int scoring) {
    if (T < 0 || T > INT32_MAX) return fail(CGD_ERR_INVALID_ARG, "num_tokens must be in [0, INT32_MAX] (got %lld)", (long long)T);
    if (E < 1 || E > cgd::kMaxExperts) return fail(CGD_ERR_INVALID_ARG, "num_experts must be in [1,512] (got %d)", E);
    if (K < 1 || K > cgd::kMaxTopk) return fail(CGD_ERR_INVALID_ARG, "num_topk must be in [1,16] (got %d)", K);
    if (K > E) return fail(CGD_ERR_INVALID_ARG, "num_topk (%d) exceeds num_experts (%d)", K, E);
    if (type != CGD_DTYPE_F32 && type != CGD_DTYPE_BF16) return fail(CGD_ERR_INVALID_ARG, "logits must be fp32 or bf16");
    if (scoring != CGD_SCORE_SOFTMAX && scoring != CGD_SCORE_SIGMOID)
        return fail(CGD_ERR_INVALID_ARG, "scoring must be 0 or 1 (got %d)", scoring);
    return CGD_OK;
}

// A product's arguments that all entry points share.
struct Sizes {
    int64_t rows;    // of x
    int64_t in, out; // features
    int64_t width;   // rows of a group's weight
    int act;
    bool fp8;
    bool grouped;
    cgd::Groups g;
};

int check_sizes(Sizes* s, int64_t rows, int groups, const int32_t* offset, int64_t capacity, const int32_t* count,
                int64_t in, int64_t out, int act, int x_type, bool grouped) {
    if (rows < 0 || rows > INT32_MAX) return fail(CGD_ERR_INVALID_ARG, "rows must be in [0, INT32_MAX] (got %lld)", (long long)rows);
    if (x_type != CGD_DTYPE_BF16 && x_type != CGD_DTYPE_FP8) return fail(CGD_ERR_INVALID_ARG, "x must be bf16 or FP8");
    const bool fp8 = x_type == CGD_DTYPE_FP8;
    const int unit = fp8 ? 128 : 8;
    if (in < unit || in % unit || in > kMaxFeatures)
        return fail(CGD_ERR_INVALID_ARG, "in_features must be a positive multiple of %d up to 2^20 (got %lld)", unit, (long long)in);
    if (act < CGD_ACT_NONE || act > CGD_ACT_SWIGLU) return fail(CGD_ERR_INVALID_ARG, "activation must be in [0,4] (got %d)", act);
    if (out < 1 || out > kMaxFeatures / 2)
        return fail(CGD_ERR_INVALID_ARG, "out_features must be in [1, 2^19] (got %lld)", (long long)out);
    if (fp8 && act == CGD_ACT_SWIGLU && out % 128)
        return fail(CGD_ERR_INVALID_ARG, "FP8 SwiGLU needs out_features to be a multiple of 128 (got %lld)", (long long)out);
    s->rows = rows;
    s->in = in;
    s->out = out;
    s->act = act;
    s->fp8 = fp8;
    s->width = act == CGD_ACT_SWIGLU ? 2 * out : out;
    s->grouped = grouped;
    s->g = cgd::Groups{nullptr, nullptr, rows, rows, 1};
    if (grouped) {
        if (groups < 1 || groups > cgd::kMaxExperts) return fail(CGD_ERR_INVALID_ARG, "num_groups must be in [1,512] (got %d)", groups);
        if (!offset) {
            if (capacity < 0 || capacity > INT32_MAX || capacity * groups != rows)
                return fail(CGD_ERR_INVALID_ARG, "num_rows must be num_groups * group_capacity without group_offset");
        }
        if (!aligned(offset, 4) || !aligned(count, 4)) return fail(CGD_ERR_INVALID_ARG, "misaligned group_offset or group_count");
        s->g = cgd::Groups{offset, count, capacity, rows, groups};
    }
    return CGD_OK;
}

int check_workspace(const void* ws, size_t have, size_t need) {
    if (need == 0) return CGD_OK;
    if (!ws || have < need || !aligned(ws, 256))
        return fail(CGD_ERR_WORKSPACE, "workspace needs %zu bytes, 256-byte aligned (got %zu)", need, have);
    return CGD_OK;
}

cgd::GemmPlan forward_plan(const Sizes& s) {
    return cgd::plan_forward(s.out, s.act == CGD_ACT_SWIGLU, s.in, s.fp8, s.g, s.grouped);
}

int forward(const Sizes& s, const void* x, const void* xs, int64_t st, int64_t sb, int fmt, const void* w,
            const float* ws_, const void* bias, const void* residual, void* out, int out_type, void* preact,
            void* workspace, size_t workspace_bytes, hipStream_t stream) {
    if (out_type != CGD_DTYPE_BF16 && out_type != CGD_DTYPE_F32) return fail(CGD_ERR_INVALID_ARG, "out must be bf16 or fp32");
    if (s.fp8 && out_type != CGD_DTYPE_BF16)
        return fail(CGD_ERR_INVALID_ARG, "FP8 products are given in bf16");
    if (!w || (s.rows > 0 && (!x || !out))) return fail(CGD_ERR_INVALID_ARG, "null x, weight or out");
    if (!aligned(x, 16) || !aligned(w, 16) || !aligned(out, 16) || !aligned(residual, 16) || !aligned(preact, 16))
        return fail(CGD_ERR_INVALID_ARG, "x, weight, residual, out and preact must be 16-byte aligned");
    if (!aligned(bias, 2)) return fail(CGD_ERR_INVALID_ARG, "misaligned bias");
    if (s.fp8) {
        if (fmt < CGD_SCALE_F32 || fmt > CGD_SCALE_UE8M0) return fail(CGD_ERR_INVALID_ARG, "scale_format must be 0, 1 or 2 (got %d)", fmt);
        if (!ws_ || (s.rows > 0 && !xs)) return fail(CGD_ERR_INVALID_ARG, "null scales");
        if (st < 0 || sb < 0 || st > (1 << 20)) return fail(CGD_ERR_INVALID_ARG, "scale strides must be >= 0, the row stride at most 2^20");
        if (!aligned(xs, fmt == CGD_SCALE_UE8M0 ? 1 : 4) || !aligned(ws_, 4)) return fail(CGD_ERR_INVALID_ARG, "misaligned scales");
    }
    const cgd::GemmPlan plan = forward_plan(s);
    if (plan.blocks > cgd::kMaxGemmBlocks) return fail(CGD_ERR_INVALID_ARG, "these sizes need more tiles than one launch holds");
    const int rc = check_workspace(workspace, workspace_bytes, plan.partial_bytes);
    if (rc) return rc;
    if (s.rows == 0) return CGD_OK;
    const int es = s.fp8 ? 1 : 2;
    cgd::GemmArgs a = {};
    a.q = x;
    a.p = w;
    a.ldq = a.ldp = s.in * es;
    a.p_group = s.width * s.in * es;
    a.n = s.out;
    a.k = s.in;
    a.g = s.g;
    a.qs = xs;
    a.ps = ws_;
    a.qs_row = st;
    a.qs_blk = sb;
    a.ps_row = s.in / 128;
    a.ps_group = (s.width + 127) / 128 * (s.in / 128);
    a.qs_byte = fmt == CGD_SCALE_UE8M0;
    a.glu = s.act == CGD_ACT_SWIGLU;
    a.act = a.glu ? 0 : s.act;
    a.bias = bias;
    a.residual = residual;
    a.out = out;
    a.out_f32 = out_type == CGD_DTYPE_F32;
    a.preact = preact;
    a.partial = static_cast<float*>(workspace);
    const hipError_t err = cgd::launch_forward(a, plan, s.fp8, s.grouped, stream);
    if (err != hipSuccess) return hip_fail(err, "product launch");
    return CGD_OK;
}

// Workspace of a backward call: d with its row pitch (a multiple of 8
// elements), then the partial column sums, then the weight gradient's pieces.
struct GradPlan {
    bool make_d;
    int64_t ldd;
    int splits;
    size_t d_bytes, partial_bytes, piece_bytes;
    size_t bytes() const { return d_bytes + partial_bytes + piece_bytes; }
};

GradPlan grad_plan(const Sizes& s, bool bias_grad) {
    GradPlan p;
    p.make_d = s.act != CGD_ACT_NONE || s.width % 8 != 0;
    p.ldd = (s.width + 7) / 8 * 8;
    p.splits = cgd::weight_grad_splits(s.g, s.width, s.in);
    p.d_bytes = p.make_d ? ((size_t)s.rows * p.ldd * 2 + 255) / 256 * 256 : 0;
    p.partial_bytes = (cgd::act_grad_workspace_bytes(s.rows, s.g.groups, s.width, bias_grad) + 255) / 256 * 256;
    p.piece_bytes = p.splits > 1 ? (size_t)p.splits * s.g.groups * s.width * s.in * 4 : 0;  // (in: a multiple of 8)
    return p;
}

int backward(const Sizes& s, const void* grad_out, const void* x, const void* w, const void* preact, void* grad_x,
             void* grad_w, void* grad_b, void* workspace, size_t workspace_bytes, hipStream_t stream) {
    if (s.rows > 0 && !grad_out) return fail(CGD_ERR_INVALID_ARG, "null grad_out");
    if (s.rows > 0 && grad_w && !x) return fail(CGD_ERR_INVALID_ARG, "null x");
    if (grad_x && !w) return fail(CGD_ERR_INVALID_ARG, "null weight");
    if (s.rows > 0 && s.act != CGD_ACT_NONE && !preact) return fail(CGD_ERR_INVALID_ARG, "an activation's gradient needs preact");
    if (!aligned(grad_out, 16) || !aligned(x, 16) || !aligned(w, 16) || !aligned(preact, 16) || !aligned(grad_x, 16) ||
        !aligned(grad_w, 16) || !aligned(grad_b, 2))
        return fail(CGD_ERR_INVALID_ARG, "grad_out, x, weight, preact, grad_x and grad_weight must be 16-byte aligned");
    const GradPlan p = grad_plan(s, grad_b != nullptr);
    // a launch has fewer than 2^32 work-items along a dimension
    const bool too_many = (p.make_d || grad_b) && cgd::act_grad_blocks(s.g, s.grouped) > UINT32_MAX / cgd::kActGradThreads;
    if (too_many || cgd::grad_blocks(s.g, s.grouped, s.width, s.in) > cgd::kMaxGemmBlocks)
        return fail(CGD_ERR_INVALID_ARG, "these sizes need more tiles than one launch holds");
    const int rc = check_workspace(workspace, workspace_bytes, p.bytes());
    if (rc) return rc;
    hipError_t err = hipSuccess;
    char* wsp = static_cast<char*>(workspace);
    if (p.make_d || grad_b) {
        err = cgd::launch_act_grad(grad_out, preact, s.act, s.out, s.g, s.grouped, p.make_d ? wsp : nullptr, p.ldd,
                                   grad_b, grad_b ? reinterpret_cast<float*>(wsp + p.d_bytes) : nullptr, stream);
        if (err != hipSuccess) return hip_fail(err, "activation gradient launch");
    }
    const void* d = p.make_d ? wsp : grad_out;
    cgd::GemmArgs a = {};
    a.g = s.g;
    a.q = d;
    a.ldq = (p.make_d ? p.ldd : s.width) * 2;
    a.splits = 1;
    if (grad_x && s.rows > 0) {
        a.p = w;
        a.ldp = s.in * 2;
        a.p_group = s.width * s.in * 2;
        a.n = s.in;
        a.k = a.ksplit = s.width;
        a.out = grad_x;
        err = cgd::launch_input_grad(a, s.grouped, stream);
        if (err != hipSuccess) return hip_fail(err, "input gradient launch");
    }
    if (grad_w) {
        a.p = x;
        a.ldp = s.in * 2;
        a.p_group = 0;
        a.m = s.width;
        a.n = s.in;
        a.out = grad_w;
        a.splits = p.splits;
        a.partial = reinterpret_cast<float*>(wsp + p.d_bytes + p.partial_bytes);
        err = cgd::launch_weight_grad(a, stream);
        if (err != hipSuccess) return hip_fail(err, "weight gradient launch");
    }
    return CGD_OK;
}

}  // namespace

extern "C" {

int cgd_route(const void* logits, int logits_type, int64_t num_tokens, int num_experts, int num_topk, int scoring,
              const float* bias, int num_groups, int num_topk_groups, int group_score_topk, int renormalize,
              float scale, int64_t* topk_idx, float* topk_weights, hipStream_t stream) {
    int rc = check_route(num_tokens, num_experts, num_topk, logits_type, scoring);
    if (rc) return rc;
    if (num_groups < 1 || num_groups > 64 || num_experts % num_groups)
        return fail(CGD_ERR_INVALID_ARG, "num_groups must be in [1,64] and divide num_experts (got %d of %d)", num_groups, num_experts);
    if (num_topk_groups < 1 || num_topk_groups > num_groups)
        return fail(CGD_ERR_INVALID_ARG, "num_topk_groups must be in [1, num_groups] (got %d)", num_topk_groups);
    if (group_score_topk != 1 && group_score_topk != 2)
        return fail(CGD_ERR_INVALID_ARG, "group_score_topk must be 1 or 2 (got %d)", group_score_topk);
    if (num_topk > num_experts / num_groups * num_topk_groups)
        return fail(CGD_ERR_INVALID_ARG, "num_topk (%d) exceeds the experts of num_topk_groups groups", num_topk);
    if (num_tokens > 0 && (!logits || !topk_idx || !topk_weights))
        return fail(CGD_ERR_INVALID_ARG, "null logits, topk_idx or topk_weights");
    if (!aligned(logits, logits_type == CGD_DTYPE_F32 ? 4 : 2) || !aligned(topk_idx, 8) || !aligned(topk_weights, 4) || !aligned(bias, 4))
        return fail(CGD_ERR_INVALID_ARG, "misaligned pointer");
    cgd::RouteArgs a;
    a.logits = logits;
    a.logits_bf16 = logits_type == CGD_DTYPE_BF16;
    a.T = num_tokens;
    a.E = num_experts;
    a.K = num_topk;
    a.sigmoid = scoring == CGD_SCORE_SIGMOID;
    a.bias = bias;
    a.groups = num_groups;
    a.topk_groups = num_topk_groups;
    a.group_top = group_score_topk;
    a.renormalize = renormalize != 0;
    a.scale = scale;
    a.topk_idx = topk_idx;
    a.topk_weights = topk_weights;
    const hipError_t err = cgd::launch_route(a, stream);
    if (err != hipSuccess) return hip_fail(err, "route launch");
    return CGD_OK;
}

int cgd_route_backward(const float* grad_topk_weights, const void* logits, int logits_type, const int64_t* topk_idx,
                       int64_t num_tokens, int num_experts, int num_topk, int scoring, int renormalize, float scale,
                       void* grad_logits, hipStream_t stream) {
    int rc = check_route(num_tokens, num_experts, num_topk, logits_type, scoring);
    if (rc) return rc;
    if (num_tokens > 0 && (!logits || !topk_idx || !grad_topk_weights || !grad_logits))
        return fail(CGD_ERR_INVALID_ARG, "null grad_topk_weights, logits, topk_idx or grad_logits");
    const size_t la = logits_type == CGD_DTYPE_F32 ? 4 : 2;
    if (!aligned(logits, la) || !aligned(grad_logits, la) || !aligned(topk_idx, 8) || !aligned(grad_topk_weights, 4))
        return fail(CGD_ERR_INVALID_ARG, "misaligned pointer");
    cgd::RouteGradArgs a;
    a.logits = logits;
    a.logits_bf16 = logits_type == CGD_DTYPE_BF16;
    a.T = num_tokens;
    a.E = num_experts;
    a.K = num_topk;
    a.sigmoid = scoring == CGD_SCORE_SIGMOID;
    a.renormalize = renormalize != 0;
    a.scale = scale;
    a.topk_idx = topk_idx;
    a.grad_weights = grad_topk_weights;
    a.grad_logits = grad_logits;
    const hipError_t err = cgd::launch_route_grad(a, stream);
    if (err != hipSuccess) return hip_fail(err, "route gradient launch");
    return CGD_OK;
}

size_t cgd_linear_workspace_bytes(int64_t num_tokens, int64_t in_features, int64_t out_features, int activation,
                                  int x_type) {
    Sizes s;
    if (check_sizes(&s, num_tokens, 1, nullptr, 0, nullptr, in_features, out_features, activation, x_type, false)) return 0;
    return forward_plan(s).partial_bytes;
}

int cgd_linear(const void* x, int x_type, const void* x_scales, int64_t scale_row_stride, int64_t scale_block_stride,
               int scale_format, const void* weight, const float* weight_scales, int64_t num_tokens,
               int64_t in_features, int64_t out_features, const void* bias, int activation, const void* residual,
               void* out, int out_type, void* preact, void* workspace, size_t workspace_bytes, hipStream_t stream) {
    Sizes s;
    const int rc = check_sizes(&s, num_tokens, 1, nullptr, 0, nullptr, in_features, out_features, activation, x_type, false);
    if (rc) return rc;
    return forward(s, x, x_scales, scale_row_stride, scale_block_stride, scale_format, weight, weight_scales, bias,
                   residual, out, out_type, preact, workspace, workspace_bytes, stream);
}

// group_offset only says which of the two layouts is sized here.
static const int32_t kSomeOffset = 0;

size_t cgd_grouped_linear_workspace_bytes(int64_t num_rows, int num_groups, int64_t group_capacity,
                                          int64_t in_features, int64_t out_features, int activation, int x_type) {
    Sizes s;
    if (check_sizes(&s, num_rows, num_groups, group_capacity > 0 ? nullptr : &kSomeOffset, group_capacity, nullptr,
                    in_features, out_features, activation, x_type, true))
        return 0;
    return forward_plan(s).partial_bytes;
}

int cgd_grouped_linear(const void* x, int x_type, const void* x_scales, int64_t scale_row_stride,
                       int64_t scale_block_stride, int scale_format, const void* weight, const float* weight_scales,
                       int64_t num_rows, int num_groups, const int32_t* group_offset, int64_t group_capacity,
                       const int32_t* group_count, int64_t in_features, int64_t out_features, const void* bias,
                       int activation, void* out, void* preact, void* workspace, size_t workspace_bytes,
                       hipStream_t stream) {
    Sizes s;
    const int rc = check_sizes(&s, num_rows, num_groups, group_offset, group_capacity, group_count, in_features,
                               out_features, activation, x_type, true);
    if (rc) return rc;
    return forward(s, x, x_scales, scale_row_stride, scale_block_stride, scale_format, weight, weight_scales, bias,
                   nullptr, out, CGD_DTYPE_BF16, preact, workspace, workspace_bytes, stream);
}

size_t cgd_linear_backward_workspace_bytes(int64_t num_tokens, int64_t in_features, int64_t out_features,
                                           int activation, int bias_grad) {
    Sizes s;
    if (check_sizes(&s, num_tokens, 1, nullptr, 0, nullptr, in_features, out_features, activation, CGD_DTYPE_BF16, false)) return 0;
    return grad_plan(s, bias_grad != 0).bytes();
}

int cgd_linear_backward(const void* grad_out, const void* x, const void* weight, int64_t num_tokens,
                        int64_t in_features, int64_t out_features, const void* preact, int activation, void* grad_x,
                        void* grad_weight, void* grad_bias, void* workspace, size_t workspace_bytes,
                        hipStream_t stream) {
    Sizes s;
    const int rc = check_sizes(&s, num_tokens, 1, nullptr, 0, nullptr, in_features, out_features, activation,
                               CGD_DTYPE_BF16, false);
    if (rc) return rc;
    return backward(s, grad_out, x, weight, preact, grad_x, grad_weight, grad_bias, workspace, workspace_bytes, stream);
}

size_t cgd_grouped_linear_backward_workspace_bytes(int64_t num_rows, int num_groups, int64_t in_features,
                                                   int64_t out_features, int activation, int bias_grad) {
    Sizes s;
    if (check_sizes(&s, num_rows, num_groups, &kSomeOffset, 0, nullptr, in_features, out_features, activation,
                    CGD_DTYPE_BF16, true))
        return 0;
    return grad_plan(s, bias_grad != 0).bytes();
}

int cgd_grouped_linear_backward(const void* grad_out, const void* x, const void* weight, int64_t num_rows,
                                int num_groups, const int32_t* group_offset, int64_t group_capacity,
                                const int32_t* group_count, int64_t in_features, int64_t out_features,
                                const void* preact, int activation, void* grad_x, void* grad_weight, void* grad_bias,
                                void* workspace, size_t workspace_bytes, hipStream_t stream) {
    Sizes s;
    const int rc = check_sizes(&s, num_rows, num_groups, group_offset, group_capacity, group_count, in_features,
                               out_features, activation, CGD_DTYPE_BF16, true);
    if (rc) return rc;
    return backward(s, grad_out, x, weight, preact, grad_x, grad_weight, grad_bias, workspace, workspace_bytes, stream);
}

}  // extern "C"
