// Gradient of the weighted combine out[t] = sum_k w[t,k] y[dst_row[t,k]]:
//   grad_y[dst_row[t,k]] = w[t,k] grad[t]          (bf16)
//   grad_w[t,k] = <grad[t], y[dst_row[t,k]]>        (fp32 sum)
// A block takes a token, a wave one of its slots: it reads the slot's expert row,
// writes the row's gradient and adds up their product, so a slot needs no other
// wave. The token's gradient row is read by all waves of the block and comes from
// the caches after the first. Slots without a row have a gradient of 0; rows that
// no slot names are left as they were.
#include "cgd_device.h"
#include "cgd_layer_launch.h"

namespace cgd {

namespace {

__device__ __forceinline__ float dot2(uint32_t a, uint32_t b, float s) {
    s = __builtin_fmaf(bf16_lo(a), bf16_lo(b), s);
    return __builtin_fmaf(bf16_hi(a), bf16_hi(b), s);
}
__device__ __forceinline__ uint32_t scale2(uint32_t a, float w) { return pack_bf16x2(bf16_lo(a) * w, bf16_hi(a) * w); }

constexpr int kGradRow = 4;  // vectors of a row on their way at a time

__global__ __launch_bounds__(1024) void combine_grad_kernel(const CombineGradArgs a) {
    const int64_t t = blockIdx.x;
    const int k = threadIdx.x / kWave, lane = lane_id();
    const int nvec = a.width / 8;
    const int64_t slot = t * a.topk + k;
    const int row = __builtin_amdgcn_readfirstlane(a.dst_row[slot]);
    if (row < 0 || row >= a.capacity) {
        if (lane == 0) a.grad_weights[slot] = 0.0f;
        return;
    }
    const float w = a.weights[slot];
    const uint4* g = reinterpret_cast<const uint4*>(a.grad) + t * nvec;
    const uint4* y = reinterpret_cast<const uint4*>(a.y) + (int64_t)row * nvec;
    uint4* o = reinterpret_cast<uint4*>(a.grad_y) + (int64_t)row * nvec;
    float s = 0.0f;
    for (int v0 = lane; v0 < nvec; v0 += kGradRow * kWave) {
        uint4 gs[kGradRow], ys[kGradRow];
#pragma unroll
        for (int u = 0; u < kGradRow; ++u) {
            const int v = v0 + u * kWave;
            gs[u] = ys[u] = make_uint4(0, 0, 0, 0);
            if (v < nvec) {
                ys[u] = load_nt(y + v);
                gs[u] = g[v];
            }
        }
#pragma unroll
        for (int u = 0; u < kGradRow; ++u) {
            const int v = v0 + u * kWave;
            if (v >= nvec) break;
            s = dot2(gs[u].x, ys[u].x, s);
            s = dot2(gs[u].y, ys[u].y, s);
            s = dot2(gs[u].z, ys[u].z, s);
            s = dot2(gs[u].w, ys[u].w, s);
            store_nt(o + v, make_uint4(scale2(gs[u].x, w), scale2(gs[u].y, w), scale2(gs[u].z, w), scale2(gs[u].w, w)));
        }
    }
#pragma unroll
    for (int d = 32; d; d >>= 1) s += __shfl_xor(s, d, kWave);
    if (lane == 0) a.grad_weights[slot] = s;
}

}  // namespace

hipError_t launch_combine_grad(const CombineGradArgs& all, hipStream_t stream) {
    if (all.tokens == 0) return hipSuccess;
    const int64_t most = kMaxWorkItems / (16 * kWave);
    for (int64_t t0 = 0; t0 < all.tokens; t0 += most) {
        CombineGradArgs a = all;
        a.tokens = all.tokens - t0 < most ? all.tokens - t0 : most;
        a.grad += t0 * all.width;
        a.dst_row += t0 * all.topk;
        a.weights += t0 * all.topk;
        a.grad_weights += t0 * all.topk;
        hipLaunchKernelGGL(combine_grad_kernel, dim3((unsigned)a.tokens), dim3((unsigned)(a.topk * kWave)), 0, stream, a);
    }
    return hipGetLastError();
}

hipError_t preload_combine_grad() {
    hipFuncAttributes at;
    return hipFuncGetAttributes(&at, reinterpret_cast<const void*>(&combine_grad_kernel));
}

}  // namespace cgd
