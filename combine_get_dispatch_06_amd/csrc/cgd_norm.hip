// Root-mean-square norm with the residual's addition, bf16 and FP8 outputs, and
// its gradient.
//   s = x + residual (fp32);  r = 1 / sqrt(mean(s^2) + eps);  y = s r w
//   sum = bf16(s): the next residual. y is made from s before that rounding.
//   FP8: y in fp32 goes straight into codes and scales (one for 128 values of a
//   row, the formats of the per-token cast): a bf16 step in between would cost
//   2^-9 of a scale for nothing.
//   gradient, with g = dy w and h = s r:  ds = r (g - h mean(g h)) + d_sum,
//   dw = sum over rows of dy h
// Memory-bound: every input is read once into registers and every output written
// once; a row's sums go over its lanes with shuffles and, where a row has more
// than a wave, over its waves through LDS.
#include "cgd_device.h"
#include "cgd_layer_launch.h"

namespace cgd {

namespace {

// Sum of v over the LANES lanes (16, 32, 64) or all LANES threads of the block
// that hold a row; every one of them gets it. `slot`: LDS, one float per wave.
template <int LANES>
__device__ __forceinline__ float row_sum(float v, float* slot) {
#pragma unroll
    for (int d = (LANES < kWave ? LANES : kWave) / 2; d; d >>= 1) v += __shfl_xor(v, d, kWave);
    if constexpr (LANES > kWave) {
        const int wave = threadIdx.x / kWave;
        if (lane_id() == 0) slot[wave] = v;
        __syncthreads();
        v = 0.0f;
#pragma unroll
        for (int w = 0; w < LANES / kWave; ++w) v += slot[w];
    }
    return v;
}

// The same of two values.
template <int LANES>
__device__ __forceinline__ void row_sums(float& a, float& b, float (*slot)[2]) {
#pragma unroll
    for (int d = (LANES < kWave ? LANES : kWave) / 2; d; d >>= 1) {
        a += __shfl_xor(a, d, kWave);
        b += __shfl_xor(b, d, kWave);
    }
    if constexpr (LANES > kWave) {
        const int wave = threadIdx.x / kWave;
        if (lane_id() == 0) {
            slot[wave][0] = a;
            slot[wave][1] = b;
        }
        __syncthreads();
        a = b = 0.0f;
#pragma unroll
        for (int w = 0; w < LANES / kWave; ++w) {
            a += slot[w][0];
            b += slot[w][1];
        }
    }
}

__device__ __forceinline__ void unpack8(const uint4& q, float (&v)[8]) {
    v[0] = bf16_lo(q.x), v[1] = bf16_hi(q.x), v[2] = bf16_lo(q.y), v[3] = bf16_hi(q.y);
    v[4] = bf16_lo(q.z), v[5] = bf16_hi(q.z), v[6] = bf16_lo(q.w), v[7] = bf16_hi(q.w);
}
__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
    return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
}
__device__ __forceinline__ uint4 vec_at(const uint16_t* p, int64_t v) { return reinterpret_cast<const uint4*>(p)[v]; }

__device__ __forceinline__ void weight8(const void* w, int f32, int v, float (&out)[8]) {
    if (f32) {
        const float4 a = static_cast<const float4*>(w)[2 * v], b = static_cast<const float4*>(w)[2 * v + 1];
        out[0] = a.x, out[1] = a.y, out[2] = a.z, out[3] = a.w;
        out[4] = b.x, out[5] = b.y, out[6] = b.z, out[7] = b.w;
    } else {
        unpack8(static_cast<const uint4*>(w)[v], out);
    }
}

// LANES threads hold a row, V 16-byte vectors each; a block has THREADS threads.
template <int THREADS, int LANES, int V>
__global__ __launch_bounds__(THREADS) void norm_kernel(const NormArgs a) {
    __shared__ float slot[THREADS / kWave];
    const int nvec = a.width / 8;
    const int64_t row = (int64_t)blockIdx.x * (THREADS / LANES) + threadIdx.x / LANES;
    const int l = threadIdx.x % LANES;
    if (LANES <= kWave && row >= a.rows) return;  // (a row of a whole block always exists)
    const int64_t base = row * nvec;
    uint4 xs[V], rs[V];
#pragma unroll
    for (int u = 0; u < V; ++u) {
        const int v = l + u * LANES;
        xs[u] = rs[u] = make_uint4(0, 0, 0, 0);
        if (v < nvec) {
            xs[u] = vec_at(a.x, base + v);
            if (a.residual) rs[u] = vec_at(a.residual, base + v);
        }
    }
    float s[V][8];
    float ss = 0.0f;
#pragma unroll
    for (int u = 0; u < V; ++u) {
        float r[8];
        unpack8(xs[u], s[u]);
        unpack8(rs[u], r);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (a.residual) s[u][i] += r[i];
            ss = __builtin_fmaf(s[u][i], s[u][i], ss);
        }
    }
    const float r = rsqrtf(row_sum<LANES>(ss, slot) / (float)a.width + a.eps);
#pragma unroll
    for (int u = 0; u < V; ++u) {
        const int v = l + u * LANES;
        const bool in = v < nvec;
        if (in && a.sum) reinterpret_cast<uint4*>(a.sum)[base + v] = pack8(s[u]);
        float y[8];
        float w[8];
        if (in) weight8(a.weight, a.weight_f32, v, w);
        float m = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            y[i] = in ? s[u][i] * r * w[i] : 0.0f;
            m = fmaxf(m, fabsf(y[i]));
        }
        if (in && a.y) reinterpret_cast<uint4*>(a.y)[base + v] = pack8(y);
        if (a.codes) {  // 16 lanes hold a block of 128: all of them are in the row or none
            const Fp8Scale sc = fp8_block_scale(group16_max(m), a.format);
            if (in) {
                uint2 q;
                q.x = pack_e4m3x4(y[0] * sc.mul, y[1] * sc.mul, y[2] * sc.mul, y[3] * sc.mul);
                q.y = pack_e4m3x4(y[4] * sc.mul, y[5] * sc.mul, y[6] * sc.mul, y[7] * sc.mul);
                reinterpret_cast<uint2*>(a.codes)[base + v] = q;
                if ((v & 15) == 0) {
                    const int64_t at = (base + v) / 16;
                    if (a.format == 2)
                        static_cast<uint8_t*>(a.scales)[at] = (uint8_t)sc.ue8m0;
                    else
                        static_cast<float*>(a.scales)[at] = sc.scale;
                }
            }
        }
    }
}

template <int THREADS, int LANES, int V>
hipError_t norm_rows(const NormArgs& all, hipStream_t stream) {
    constexpr int kRows = THREADS / LANES;
    const int64_t most = kMaxWorkItems / LANES;  // whole blocks of rows
    for (int64_t r0 = 0; r0 < all.rows; r0 += most) {
        NormArgs a = all;
        a.rows = all.rows - r0 < most ? all.rows - r0 : most;
        const int64_t at = r0 * all.width;
        a.x += at;
        if (a.residual) a.residual += at;
        if (a.y) a.y += at;
        if (a.sum) a.sum += at;
        if (a.codes) {
            a.codes += at;
            a.scales = static_cast<char*>(a.scales) + at / kFp8Block * (a.format == 2 ? 1 : 4);
        }
        hipLaunchKernelGGL((norm_kernel<THREADS, LANES, V>), dim3((unsigned)((a.rows + kRows - 1) / kRows)), dim3(THREADS), 0, stream, a);
    }
    return hipGetLastError();
}

// Gradient. A block takes every gridDim.x-th group of rows and keeps the
// weight's gradient of its columns in registers: one row of sums a block.
template <int THREADS, int LANES, int V>
__global__ __launch_bounds__(THREADS) void norm_grad_kernel(const NormGradArgs a) {
    constexpr int kRows = THREADS / LANES;
    __shared__ float slot[2][THREADS / kWave][2];
    const int nvec = a.width / 8;
    const int l = threadIdx.x % LANES;
    float w[V][8], dw[V][8];
#pragma unroll
    for (int u = 0; u < V; ++u) {
#pragma unroll
        for (int i = 0; i < 8; ++i) w[u][i] = dw[u][i] = 0.0f;
        if (l + u * LANES < nvec) weight8(a.weight, a.weight_f32, l + u * LANES, w[u]);
    }
    int turn = 0;
    const float mean = 1.0f / (float)a.width;
    for (int64_t row0 = (int64_t)blockIdx.x * kRows; row0 < a.rows; row0 += (int64_t)gridDim.x * kRows) {
        const int64_t row = row0 + threadIdx.x / LANES;
        const bool there = LANES > kWave || row < a.rows;
        const int64_t base = row * nvec;
        uint4 xs[V], gs[V], ds[V];
#pragma unroll
        for (int u = 0; u < V; ++u) {
            const int v = l + u * LANES;
            xs[u] = gs[u] = ds[u] = make_uint4(0, 0, 0, 0);
            if (there && v < nvec) {
                xs[u] = vec_at(a.x, base + v);
                gs[u] = vec_at(a.grad, base + v);
                if (a.grad_sum) ds[u] = vec_at(a.grad_sum, base + v);
            }
        }
        float ss = 0.0f, gx = 0.0f;
#pragma unroll
        for (int u = 0; u < V; ++u) {
            float x[8], g[8];
            unpack8(xs[u], x);
            unpack8(gs[u], g);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                ss = __builtin_fmaf(x[i], x[i], ss);
                gx = __builtin_fmaf(g[i] * w[u][i], x[i], gx);
            }
        }
        row_sums<LANES>(ss, gx, slot[turn]);  // (two sets of slots: a wave may be one row ahead, not two)
        turn ^= 1;
        const float r = rsqrtf(ss * mean + a.eps);
        const float c = gx * r * r * mean;  // times s: h mean(g h)
#pragma unroll
        for (int u = 0; u < V; ++u) {
            const int v = l + u * LANES;
            float x[8], g[8], d[8];
            unpack8(xs[u], x);
            unpack8(gs[u], g);
            unpack8(ds[u], d);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (there) dw[u][i] = __builtin_fmaf(g[i] * r, x[i], dw[u][i]);  // (r of no row may be infinite)
                const float t = r * (g[i] * w[u][i] - x[i] * c);
                d[i] = a.grad_sum ? d[i] + t : t;
            }
            if (a.grad_x && there && v < nvec) reinterpret_cast<uint4*>(a.grad_x)[base + v] = pack8(d);
        }
    }
    if (!a.partial) return;
    if constexpr (LANES <= kWave) {  // the block's groups of lanes, in order
        __shared__ float part[THREADS][9];
        float* out = a.partial + (int64_t)blockIdx.x * a.width;
#pragma unroll
        for (int u = 0; u < V; ++u) {
            __syncthreads();
#pragma unroll
            for (int i = 0; i < 8; ++i) part[threadIdx.x][i] = dw[u][i];
            __syncthreads();
            for (int c = threadIdx.x; c < LANES * 8; c += THREADS) {
                float s = 0.0f;
#pragma unroll
                for (int k = 0; k < kRows; ++k) s += part[k * LANES + c / 8][c % 8];
                if (c + u * LANES * 8 < a.width) out[c + u * LANES * 8] = s;
            }
        }
    } else {
        float4* out = reinterpret_cast<float4*>(a.partial + (int64_t)blockIdx.x * a.width);
#pragma unroll
        for (int u = 0; u < V; ++u) {
            const int v = l + u * LANES;
            if (v >= nvec) continue;
            out[2 * v] = make_float4(dw[u][0], dw[u][1], dw[u][2], dw[u][3]);
            out[2 * v + 1] = make_float4(dw[u][4], dw[u][5], dw[u][6], dw[u][7]);
        }
    }
}

// Adds the blocks' rows of sums in a fixed order: a block takes 64 columns, its
// 16 waves every 16th row.
__global__ __launch_bounds__(1024) void norm_weight_kernel(const float* partial, int blocks, int width, void* out, int f32) {
    __shared__ float sums[16][kWave];
    const int c = blockIdx.x * kWave + lane_id(), wave = threadIdx.x / kWave;
    float s = 0.0f;
    if (c < width) {
        int i = wave;
        for (; i + 7 * 16 < blocks; i += 8 * 16) {
            float v[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) v[u] = partial[(int64_t)(i + 16 * u) * width + c];
#pragma unroll
            for (int u = 0; u < 8; ++u) s += v[u];
        }
        for (; i < blocks; i += 16) s += partial[(int64_t)i * width + c];
    }
    sums[wave][lane_id()] = s;
    __syncthreads();
    if (wave || c >= width) return;
    for (int k = 1; k < 16; ++k) s += sums[k][lane_id()];
    if (f32)
        static_cast<float*>(out)[c] = s;
    else
        static_cast<uint16_t*>(out)[c] = (uint16_t)pack_bf16x2(s, 0.0f);
}

template <int THREADS, int LANES, int V>
void norm_grad_rows(const NormGradArgs& a, int64_t blocks, hipStream_t stream) {
    hipLaunchKernelGGL((norm_grad_kernel<THREADS, LANES, V>), dim3((unsigned)blocks), dim3(THREADS), 0, stream, a);
}

// Threads that hold a row of the gradient, and a block's threads.
int grad_lanes(int width) { return width <= 128 ? 16 : width <= 256 ? 32 : width <= 2048 ? 64 : width <= 8192 ? 512 : 1024; }
int grad_threads(int width) { return width <= 2048 ? 256 : width <= 8192 ? 512 : 1024; }

}  // namespace

hipError_t launch_norm(const NormArgs& a, hipStream_t stream) {
    if (a.rows == 0) return hipSuccess;
    const int w = a.width;
    if (w <= 128) return norm_rows<256, 16, 1>(a, stream);
    if (w <= 256) return norm_rows<256, 32, 1>(a, stream);
    if (w <= 512) return norm_rows<256, 64, 1>(a, stream);
    if (w <= 1024) return norm_rows<256, 64, 2>(a, stream);
    if (w <= 2048) return norm_rows<256, 256, 1>(a, stream);
    if (a.rows <= 512) {  // few rows: more threads for each
        if (w <= 8192) return norm_rows<1024, 1024, 1>(a, stream);
        if (w <= 16384) return norm_rows<1024, 1024, 2>(a, stream);
        return norm_rows<1024, 1024, 4>(a, stream);
    }
    if (w <= 4096) return norm_rows<256, 256, 2>(a, stream);
    if (w <= 8192) return norm_rows<256, 256, 4>(a, stream);
    if (w <= 16384) return norm_rows<512, 512, 4>(a, stream);
    return norm_rows<1024, 1024, 4>(a, stream);
}

int64_t norm_grad_blocks(int64_t rows, int width) {
    const int per = grad_threads(width) / grad_lanes(width);
    const int64_t groups = (rows + per - 1) / per;
    const int64_t most = width <= 2048 ? 1024 : width <= 8192 ? 512 : 256;
    return groups < most ? groups : most;
}

hipError_t launch_norm_grad(const NormGradArgs& a, hipStream_t stream) {
    const int w = a.width;
    const int64_t blocks = norm_grad_blocks(a.rows, w);
    if (blocks > 0) {
        if (w <= 128)
            norm_grad_rows<256, 16, 1>(a, blocks, stream);
        else if (w <= 256)
            norm_grad_rows<256, 32, 1>(a, blocks, stream);
        else if (w <= 512)
            norm_grad_rows<256, 64, 1>(a, blocks, stream);
        else if (w <= 1024)
            norm_grad_rows<256, 64, 2>(a, blocks, stream);
        else if (w <= 2048)
            norm_grad_rows<256, 64, 4>(a, blocks, stream);
        else if (w <= 4096)
            norm_grad_rows<512, 512, 1>(a, blocks, stream);
        else if (w <= 8192)
            norm_grad_rows<512, 512, 2>(a, blocks, stream);
        else if (w <= 16384)
            norm_grad_rows<1024, 1024, 2>(a, blocks, stream);
        else
            norm_grad_rows<1024, 1024, 4>(a, blocks, stream);
        const hipError_t err = hipGetLastError();
        if (err != hipSuccess) return err;
    }
    if (a.grad_weight)
        hipLaunchKernelGGL(norm_weight_kernel, dim3((unsigned)((w + kWave - 1) / kWave)), dim3(1024), 0, stream, a.partial,
                           (int)blocks, w, a.grad_weight, a.weight_f32);
    return hipGetLastError();
}

hipError_t preload_norm() {
    hipFuncAttributes at;
    return hipFuncGetAttributes(&at, reinterpret_cast<const void*>(&norm_weight_kernel));
}

}  // namespace cgd
