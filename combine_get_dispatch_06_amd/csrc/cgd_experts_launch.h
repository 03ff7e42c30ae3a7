// Internal launchers of the router and of the dense and grouped products
// (host side). Arguments are validated by cgd_experts_api.hip before these
// are called.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace cgd {

// Sets cgd_last_error's message for this thread and returns `code`.
int report(int code, const char* message);

enum { kActNone = 0, kActRelu = 1, kActSilu = 2, kActGelu = 3, kActSwiglu = 4 };

// The rows of each group: [offset[e], offset[e + 1]) of `total` rows, or
// [e * capacity, (e + 1) * capacity) without offsets; of those the first
// count[e] where counts are given. A dense product is one group of all rows.
struct Groups {
    const int32_t* offset;
    const int32_t* count;
    int64_t capacity;
    int64_t total;
    int groups;
};

struct GemmArgs {
    const void* q;        // row operand, ldq bytes from row to row
    const void* p;        // column operand, ldp bytes from row to row, p_group bytes from group to group
    int64_t ldq, ldp, p_group;
    int64_t m, n, k;      // m: weight gradients only; n: output columns; k: the reduction (not of weight gradients)
    Groups g;
    const void* qs;       // FP8: scales of q (element strides; bytes: UE8M0) and of p ([group][row block][k block])
    const void* ps;
    int64_t qs_row, qs_blk, ps_row, ps_group;
    int qs_byte;
    int glu;              // SwiGLU: p has n gate rows, then n up rows
    int act;
    const void* bias;     // bf16 [group, rows of p]
    const void* residual; // bf16 [row, n]
    void* out;
    int out_f32;
    void* preact;         // bf16 [row, rows of p], or null
    int splits;           // pieces of the reduction (1: none), ksplit long
    int64_t ksplit;
    float* partial;       // [splits, total rows, rows of p] where splits > 1
};

// How a product is tiled: decided from its sizes alone.
struct GemmPlan {
    int tile;       // index of a tile shape
    int splits;
    int64_t ksplit;
    size_t partial_bytes;
    int64_t blocks; // launched at most
};
constexpr int64_t kMaxGemmBlocks = int64_t(1) << 22;  // of up to 512 threads: work-item ids stay within 32 bits

GemmPlan plan_forward(int64_t n, int glu, int64_t k, bool fp8, const Groups& g, bool grouped);
hipError_t launch_join(const GemmArgs& a, bool grouped, hipStream_t stream);  // of a split reduction's pieces
hipError_t launch_forward(const GemmArgs& a, const GemmPlan& p, bool fp8, bool grouped, hipStream_t stream);

// Input gradient (a.p: weights [groups][k][n], read transposed) and weight
// gradient (both operands read transposed; out [groups][m][n], partial
// [splits][groups][m][n padded to 8] where a.splits > 1).
int64_t grad_blocks(const Groups& g, bool grouped, int64_t width, int64_t k);  // of the larger of the two launches
int weight_grad_splits(const Groups& g, int64_t width, int64_t k);  // pieces of each group's rows
hipError_t launch_input_grad(const GemmArgs& a, bool grouped, hipStream_t stream);
hipError_t launch_weight_grad(const GemmArgs& a, hipStream_t stream);

// d = grad_out * act'(preact), bf16 [total, ldd elements per row], and the
// sums of d over each group's rows (bf16 [groups, width]); either may be null.
int64_t act_grad_blocks(const Groups& g, bool grouped);  // launched at most along the rows, kActGradThreads each
constexpr int kActGradThreads = 256;
size_t act_grad_workspace_bytes(int64_t total, int groups, int64_t width, bool bias_grad);
hipError_t launch_act_grad(const void* grad_out, const void* preact, int act, int64_t n, const Groups& g, bool grouped,
                           void* d, int64_t ldd, void* bias_grad, float* partial, hipStream_t stream);

// Router.
struct RouteArgs {
    const void* logits;
    int logits_bf16;
    int64_t T;
    int E, K;
    int sigmoid;
    const float* bias;
    int groups, topk_groups, group_top;
    int renormalize;
    float scale;
    int64_t* topk_idx;
    float* topk_weights;
};
hipError_t launch_route(const RouteArgs& a, hipStream_t stream);
struct RouteGradArgs {
    const void* logits;
    int logits_bf16;
    int64_t T;
    int E, K;
    int sigmoid;
    int renormalize;
    float scale;
    const int64_t* topk_idx;
    const float* grad_weights;
    void* grad_logits;
};
hipError_t launch_route_grad(const RouteGradArgs& a, hipStream_t stream);

hipError_t preload_route();
hipError_t preload_gemm();
hipError_t preload_gemm_fp8();
hipError_t preload_gemm_grad();
hipError_t preload_act_grad();

}  // namespace cgd
