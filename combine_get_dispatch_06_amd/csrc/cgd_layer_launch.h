// Internal launchers of the norm, dropout, the adapters and combine's gradient
// (host side). Arguments are validated by cgd_layer_api.hip before these are
// called.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace cgd {

// Sets cgd_last_error's message for this thread and returns `code`.
int report(int code, const char* message);

// Work-items of one launch along its first dimension: rows go in ranges.
constexpr int64_t kMaxWorkItems = int64_t(1) << 31;

// ---- norm
constexpr int kMaxNormWidth = 32768;

struct NormArgs {
    const uint16_t* x;
    const uint16_t* residual;  // or null
    const void* weight;
    int weight_f32;
    float eps;
    int64_t rows;
    int width;
    uint16_t* y;    // or null
    uint8_t* codes; // or null: no FP8 output
    void* scales;   // [rows, width / 128]: fp32, or one UE8M0 byte (format 2)
    int format;
    uint16_t* sum;  // x + residual, or null
};
hipError_t launch_norm(const NormArgs& a, hipStream_t stream);

struct NormGradArgs {
    const uint16_t* grad;
    const uint16_t* x;
    const void* weight;
    int weight_f32;
    float eps;
    int64_t rows;
    int width;
    const uint16_t* grad_sum;  // or null
    uint16_t* grad_x;          // or null
    float* partial;            // [norm_grad_blocks][width], where grad_weight is wanted
    void* grad_weight;         // of the weight's type, or null
};
int64_t norm_grad_blocks(int64_t rows, int width);
hipError_t launch_norm_grad(const NormGradArgs& a, hipStream_t stream);

// ---- dropout
struct DropoutArgs {
    const uint16_t* x;
    const uint16_t* residual;  // or null
    uint16_t* out;
    int64_t n;
    uint32_t limit;            // of 65536: elements whose number is below it are dropped
    float scale;
    uint64_t seed, offset;
    const int64_t* state;      // or null: {seed, offset} on the device, added to the two above
};
hipError_t launch_dropout(const DropoutArgs& a, hipStream_t stream);

// ---- gradient of combine
struct CombineGradArgs {
    const uint16_t* grad;
    const uint16_t* y;
    int64_t capacity;
    int width;
    const int32_t* dst_row;
    const float* weights;
    int64_t tokens;
    int topk;
    uint16_t* grad_y;
    float* grad_weights;
};
hipError_t launch_combine_grad(const CombineGradArgs& a, hipStream_t stream);

// ---- adapters
constexpr int kMaxRank = 256;
constexpr int64_t kMaxAdapterTokens = int64_t(1) << 26;

struct AdapterArgs {
    const uint16_t* x;   // [tokens, in]
    const uint16_t* a;   // [adapters, rank, in]
    const uint16_t* b;   // [adapters, out, rank]
    const float* scale;  // [adapters] or null
    const int64_t* index;
    int64_t tokens, in, out_features;
    int adapters, rank;
    const uint16_t* residual;
    uint16_t* out;
    float* hidden;       // [tokens, rank] or null
};
struct AdapterGradArgs {
    const uint16_t* grad;   // [tokens, out]
    const uint16_t* x;
    const uint16_t* a;
    const uint16_t* b;
    const float* scale;
    const int64_t* index;
    const float* hidden;
    int64_t tokens, in, out_features;
    int adapters, rank;
    uint16_t* grad_x;  // each may be null
    uint16_t* grad_a;
    uint16_t* grad_b;
};
size_t adapter_workspace_bytes(int64_t tokens, int adapters, int rank, int64_t in, int64_t out);
size_t adapter_grad_workspace_bytes(int64_t tokens, int adapters, int rank, int64_t in, int64_t out);
hipError_t launch_adapters(const AdapterArgs& a, void* workspace, hipStream_t stream);
hipError_t launch_adapters_grad(const AdapterGradArgs& a, void* workspace, hipStream_t stream);

hipError_t preload_norm();
hipError_t preload_dropout();
hipError_t preload_combine_grad();
hipError_t preload_adapters();

}  // namespace cgd
