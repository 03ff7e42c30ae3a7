// Gradient through an activation and the bias gradient.
//   d[m, c] = grad_out[m, c] * act'(preact[m, c])
//   SwiGLU: d[m, c] = g * up * silu'(gate), d[m, n + c] = g * silu(gate)
//   grad_b[e][c] = sum over e's rows of d, from the fp32 values
// d is rounded to bf16 once: it is the operand of two matrix products, and the
// matrix cores take bf16 pairs. It shows: gradients behind an activation are off by
// 2.3e-3 of their size (root mean square; SwiGLU, 4095 rows, 2048 columns), of which
// their own rounding is 1.7e-3. A second bf16 part of d would keep those 1.7e-3 and
// double both products' time; grad_out itself comes in bf16, rounded as coarsely.
// Memory-bound: one pass over grad_out and preact, 16 bytes per lane. A block
// takes 32 rows of one group and 512 columns (short enough for many blocks, long
// enough that the sums' traffic is a 32nd of the rows'); column sums go up through
// LDS in a fixed order, one fp32 row per block, which a second kernel adds in order.
// SwiGLU, 4095 rows, 2048 columns, with the bias gradient: 25 us for 84 MB
// (3.4 TB/s), 5 us for the sums.
#include "cgd_gemm_launch.h"

namespace cgd {

constexpr int kActRows = 32;

__device__ __forceinline__ float act_slope(float v, int act) {
    if (act == kActRelu) return v > 0.0f ? 1.0f : (v <= 0.0f ? 0.0f : v);
    if (act == kActSilu) {
        const float s = sigmoid_f(v);
        return s + v * s * (1.0f - s);
    }
    if (act == kActGelu)
        return normal_cdf(v) + v * 0.39894228040143268f * __expf(-0.5f * v * v);
    return 1.0f;
}

struct ActGradArgs {
    const uint16_t* grad;
    const uint16_t* pre;
    int act;
    int64_t n, ldd;
    Groups g;
    uint16_t* d;
    float* partial;  // [piece][width] or null
};

__global__ __launch_bounds__(kActGradThreads) void act_grad_kernel(const ActGradArgs a) {
    __shared__ float sums[2][4][512];
    const Piece pc = find_piece<true>(a.g, kActRows, (int)blockIdx.x);
    if (pc.group < 0) return;
    const bool glu = a.act == kActSwiglu;
    const int64_t width = glu ? 2 * a.n : a.n;
    const int lane = lane_id(), wave = threadIdx.x / kWave;
    const int64_t c = (int64_t)blockIdx.y * 512 + lane * 8;
    const int have = (int)(a.n - c < 8 ? a.n - c : 8);
    const int rows = pc.rows < kActRows ? (int)pc.rows : kActRows;
    const bool wide = (a.n & 7) == 0;
    float s0[8], s1[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) s0[q] = s1[q] = 0.0f;
    // columns past the width, up to the row pitch of d, are zeros: the products read them
    const int64_t pad_end = a.ldd;
    constexpr int U = 2;  // rows of a wave on their way at a time
    for (int i0 = wave; i0 < rows; i0 += 4 * U) {
        float gs[U][8], zs[U][8], us[U][8];
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int i = i0 + 4 * k;
            const int64_t row = pc.row0 + i;
            const int n = i < rows ? have : 0;
#pragma unroll
            for (int q = 0; q < 8; ++q) zs[k][q] = us[k][q] = 0.0f;
            load_run<8>(a.grad + row * a.n + c, n, wide, gs[k]);
            if (a.act) load_run<8>(a.pre + row * width + c, n, wide, zs[k]);
            if (glu) load_run<8>(a.pre + row * width + a.n + c, n, wide, us[k]);
        }
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int i = i0 + 4 * k;
            if (i >= rows) break;
            const int64_t row = pc.row0 + i;
            float d0[8], d1[8];
            const float(&g)[8] = gs[k];
            const float(&z)[8] = zs[k];
            const float(&u)[8] = us[k];
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                if (glu) {
                    const float s = sigmoid_f(z[q]);
                    d0[q] = g[q] * u[q] * (s + z[q] * s * (1.0f - s));
                    d1[q] = g[q] * z[q] * s;
                } else {
                    d0[q] = a.act ? g[q] * act_slope(z[q], a.act) : g[q];
                    d1[q] = 0.0f;
                }
                if (q < have) {
                    s0[q] += d0[q];
                    s1[q] += d1[q];
                } else {
                    d0[q] = d1[q] = 0.0f;
                }
            }
            if (a.d) {
                uint16_t* o = a.d + row * a.ldd;
                if (!glu) {  // the pad of a row lies behind its last column
                    const int room = (int)(pad_end - c < 8 ? pad_end - c : 8);
                    store_run<8>(o, c, d0, room, false, true);
                } else {
                    store_run<8>(o, c, d0, have, false, wide);
                    store_run<8>(o, a.n + c, d1, have, false, wide);
                    if (have > 0 && c + 8 >= a.n)
                        for (int64_t p = width; p < pad_end; ++p) o[p] = 0;
                }
            }
        }
    }
    if (!a.partial) return;
#pragma unroll
    for (int q = 0; q < 8; ++q) {
        sums[0][wave][lane * 8 + q] = s0[q];
        sums[1][wave][lane * 8 + q] = s1[q];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 512; i += 256) {
        const int64_t cc = (int64_t)blockIdx.y * 512 + i;
        if (cc >= a.n) continue;
        float* p = a.partial + (int64_t)blockIdx.x * width;
        p[cc] = ((sums[0][0][i] + sums[0][1][i]) + sums[0][2][i]) + sums[0][3][i];
        if (glu) p[a.n + cc] = ((sums[1][0][i] + sums[1][1][i]) + sums[1][2][i]) + sums[1][3][i];
    }
}

// grad_b[e][c]: the partial rows of e's pieces. A block takes 64 columns; its
// four waves add every fourth piece in order, and their sums in order.
// `pieces`: how many act_grad_kernel had room for (offsets that overlap ask for more).
__global__ __launch_bounds__(256) void bias_join_kernel(const Groups g, const float* partial, int64_t width,
                                                        int pieces, uint16_t* out) {
    __shared__ float sums[4][kWave];
    const int e = blockIdx.y, lane = lane_id(), wave = threadIdx.x / kWave;
    int before = 0, mine = 0;  // pieces of the groups before e, pieces of e
    if (!g.offset && !g.count && g.groups == 1) {
        mine = (int)((g.total + kActRows - 1) / kActRows);
    } else {
        for (int e0 = 0; e0 <= e; e0 += kWave) {
            const int i = e0 + lane;
            int64_t b, n = 0;
            if (i <= e) group_rows(g, i, &b, &n);
            const int p = (int)((n + kActRows - 1) / kActRows);
            if (i == e) mine = p;
            int sum = i < e ? p : 0;
#pragma unroll
            for (int d = 32; d; d >>= 1) sum += __shfl_xor(sum, d, kWave);
            before += sum;
        }
        mine = __shfl(mine, e & (kWave - 1), kWave);
    }
    before = before < 0 || before > pieces ? pieces : before;
    mine = mine > pieces - before ? pieces - before : mine;
    const int64_t c = (int64_t)blockIdx.x * kWave + lane;
    float s = 0.0f;
    if (c < width) {
        const float* p = partial + (int64_t)before * width + c;
        int i = wave;
        for (; i + 12 < mine; i += 16) {
            float x[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) x[u] = p[(int64_t)(i + 4 * u) * width];
#pragma unroll
            for (int u = 0; u < 4; ++u) s += x[u];
        }
        for (; i < mine; i += 4) s += p[(int64_t)i * width];
    }
    sums[wave][lane] = s;
    __syncthreads();
    if (wave == 0 && c < width)
        out[(int64_t)e * width + c] =
            (uint16_t)pack_bf16x2(((sums[0][lane] + sums[1][lane]) + sums[2][lane]) + sums[3][lane], 0.0f);
}

int64_t act_grad_blocks(const Groups& g, bool grouped) { return worst_pieces(g, kActRows, grouped); }

size_t act_grad_workspace_bytes(int64_t total, int groups, int64_t width, bool bias_grad) {
    if (!bias_grad) return 0;
    const int64_t pieces = total / kActRows + (groups < total ? groups : total) + 1;
    return (size_t)pieces * width * 4;
}

hipError_t launch_act_grad(const void* grad_out, const void* preact, int act, int64_t n, const Groups& g, bool grouped,
                           void* d, int64_t ldd, void* bias_grad, float* partial, hipStream_t stream) {
    ActGradArgs a;
    a.grad = static_cast<const uint16_t*>(grad_out);
    a.pre = static_cast<const uint16_t*>(preact);
    a.act = act;
    a.n = n;
    a.ldd = ldd;
    a.g = g;
    a.d = static_cast<uint16_t*>(d);
    a.partial = bias_grad ? partial : nullptr;
    const int64_t width = act == kActSwiglu ? 2 * n : n;
    const int64_t pieces = act_grad_blocks(g, grouped);
    if (pieces > 0) {
        hipLaunchKernelGGL(act_grad_kernel, dim3((unsigned)pieces, (unsigned)((n + 511) / 512)), dim3(kActGradThreads), 0, stream, a);
        hipError_t err = hipGetLastError();
        if (err != hipSuccess) return err;
    }
    if (bias_grad)
        hipLaunchKernelGGL(bias_join_kernel, dim3((unsigned)((width + kWave - 1) / kWave), (unsigned)g.groups), dim3(256), 0,
                           stream, g, partial, width, (int)pieces, static_cast<uint16_t*>(bias_grad));
    return hipGetLastError();
}

hipError_t preload_act_grad() {
    hipFuncAttributes at;
    return hipFuncGetAttributes(&at, reinterpret_cast<const void*>(&bias_join_kernel));
}

}  // namespace cgd
