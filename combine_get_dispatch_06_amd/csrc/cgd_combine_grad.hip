// Gradient of the weighted combine out[t] = sum_k w[t,k] y[dst_row[t,k]]:
//   grad_y[dst_row[t,k]] = w[t,k] grad[t]          (bf16)
//   grad_w[t,k] = <grad[t], y[dst_row[t,k]]>        (fp32 sum)
// A block takes a token, a wave one of its slots: it reads the slot's expert row,
// writes the row's gradient and adds up their product, so a slot needs no other
// wave. The token's gradient row is read by all waves of the block and comes from
// the caches after the first. Slots without a row have a gradient of 0; rows that
// no slot names are left as they were.
// 4096 tokens, top-8, hidden 7168: 190 us for 1.0 GB (5.3 TB/s): what the row copy and
// the combine take together on these rows (98 and 88). In the rows' own order instead,
// every slot reads the token's gradient once more from the Infinity Cache: 195.
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

// FROM_CACHE: the rows were just made and are still in the caches.
template <bool FROM_CACHE>
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
                ys[u] = FROM_CACHE ? y[v] : load_nt(y + v);
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
    // rows that fit the Infinity Cache: 127 tokens of top-16, hidden 4096, 7.4 us with
    // ordinary loads and 10 with non-temporal ones; the 470 MB above 200 and 189. Stores are
    // non-temporal in both: 256 tokens of top-8, hidden 7168, 9.7 us alone for 10.9 with ordinary
    // ones, though the product's gradient that reads the rows next is slower (both: 174 for 167)
    const bool cached = all.tokens * all.topk * all.width * 2 <= int64_t(64) << 20;
    for (int64_t t0 = 0; t0 < all.tokens; t0 += most) {
        CombineGradArgs a = all;
        a.tokens = all.tokens - t0 < most ? all.tokens - t0 : most;
        a.grad += t0 * all.width;
        a.dst_row += t0 * all.topk;
        a.weights += t0 * all.topk;
        a.grad_weights += t0 * all.topk;
        const dim3 grid((unsigned)a.tokens), block((unsigned)(a.topk * kWave));
        if (cached)
            hipLaunchKernelGGL(combine_grad_kernel<true>, grid, block, 0, stream, a);
        else
            hipLaunchKernelGGL(combine_grad_kernel<false>, grid, block, 0, stream, a);
    }
    return hipGetLastError();
}

hipError_t preload_combine_grad() {
    hipFuncAttributes at;
    return hipFuncGetAttributes(&at, reinterpret_cast<const void*>(&combine_grad_kernel<true>));
}

}  // namespace cgd
