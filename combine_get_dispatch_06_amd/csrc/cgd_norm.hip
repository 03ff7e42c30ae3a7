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
// once; a row's sums go over its lanes within the vector unit and, where a row has more
// than a wave, over its waves through LDS.
#include "cgd_gemm.h"
#include "cgd_layer_launch.h"

namespace cgd {

namespace {

// The lanes that hold a row: LANES neighbours (16, 32, 64) of a block of 256, or
// (0) a whole block of `threads`, a multiple of 64.
constexpr int kMaxWaves = 16;

// The value of the lane N places on, around a row of 16 lanes: within the vector unit,
// where a shuffle through LDS is some ten times as late.
template <int N>
__device__ __forceinline__ float turned16(float v) {
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x120 + N, 0xF, 0xF, true));
}
__device__ __forceinline__ float sum16(float v) {  // the same bits in all 16 lanes: addition commutes
    v += turned16<8>(v);
    v += turned16<4>(v);
    v += turned16<2>(v);
    return v + turned16<1>(v);
}
__device__ __forceinline__ float max16(float v) {
    v = fmaxf(v, turned16<8>(v));
    v = fmaxf(v, turned16<4>(v));
    v = fmaxf(v, turned16<2>(v));
    return fmaxf(v, turned16<1>(v));
}
__device__ __forceinline__ float of_lane(float v, int lane) { return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), lane)); }

// Sums of N values over a row; every lane of it gets them. `slot`: LDS, for blocks.
template <int LANES, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], int threads, float (*slot)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
        v[i] = sum16(v[i]);
        if constexpr (LANES == 32) v[i] += __shfl_xor(v[i], 16, kWave);
        if constexpr (LANES == 0 || LANES == 64) v[i] = (of_lane(v[i], 0) + of_lane(v[i], 16)) + (of_lane(v[i], 32) + of_lane(v[i], 48));
    }
    if constexpr (LANES == 0) {
        const int wave = threadIdx.x / kWave, waves = threads / kWave;
        if (lane_id() == 0)
#pragma unroll
            for (int i = 0; i < N; ++i) slot[wave][i] = v[i];
        sync_lds();
        const int from = lane_id() & (kMaxWaves - 1);
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = of_lane(sum16(from < waves ? slot[from][i] : 0.0f), 0);
    }
}

__device__ __forceinline__ void unpack8(const uint4& q, float (&v)[8]) {
    v[0] = bf16_lo(q.x), v[1] = bf16_hi(q.x), v[2] = bf16_lo(q.y), v[3] = bf16_hi(q.y);
    v[4] = bf16_lo(q.z), v[5] = bf16_hi(q.z), v[6] = bf16_lo(q.w), v[7] = bf16_hi(q.w);
}
__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
    return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
}

// FAR: what the call touches does not fit the Infinity Cache, so nothing of it is worth
// keeping there: non-temporal accesses. 4096 x 7168 with residual and FP8 (265 MB)
// 46.7 us against 54, its gradient (235 MB) 42.6 against 48.8; 131040 x 128 (67 MB) 13.6
// against 11.8. That is the call alone. With ordinary stores (and the same loads) it takes
// 48.5 for 47.5, with 8192 rows 85.6 for 90.2, and what reads y next is faster: norm, gate and
// dispatch of 4096 rows 142 for 152 (8192: 270 for 267), bf16 norm and gate of 8192 121 for 134.
constexpr int64_t kFarBytes = int64_t(160) << 20;
template <bool FAR>
__device__ __forceinline__ uint4 take(const uint4* p) {
    if constexpr (FAR) return load_nt(p);
    return *p;
}
template <bool FAR, typename T>
__device__ __forceinline__ void put(T* p, const T& v) {
    if constexpr (FAR)
        store_nt(p, v);
    else
        *p = v;
}

__device__ __forceinline__ void weight8(const void* w, int f32, int v, float (&out)[8]) {
    if (f32) {
        const float4 a = static_cast<const float4*>(w)[2 * v], b = static_cast<const float4*>(w)[2 * v + 1];
        out[0] = a.x, out[1] = a.y, out[2] = a.z, out[3] = a.w;
        out[4] = b.x, out[5] = b.y, out[6] = b.z, out[7] = b.w;
    } else {
        unpack8(static_cast<const uint4*>(w)[v], out);
    }
}

// A row whose mean of squares (with eps) is below kFaint has lost bits of its squares, or
// all of them. It is taken again, kLift times as large: every bf16 value is a normal
// number then, and so are the squares. That is done behind what every row goes through,
// with its inputs loaded anew; where the sums are known it would keep apart what overlaps
// otherwise (131040 x 128 1.3 us more, the gradient of 8000 x 4096 2). To look for such
// rows shows in few widths: 1 to 2 us of the gradient of 10000 x 3200 (42) and 30000 x 1032 (53).
constexpr float kFaint = 0x1p-100f, kLift = 0x1p100f;

// V 16-byte vectors a lane, R rows one after the other (their loads together).
template <int LANES, int V, int R, bool FAR>
__global__ __launch_bounds__(LANES ? 256 : 1024) void norm_kernel(const NormArgs a, int threads) {
    __shared__ float slot[LANES ? 1 : 2][kMaxWaves][1];
    const int nvec = a.width / 8;
    constexpr int GROUPS = LANES ? 256 / LANES : 1;
    const int step = LANES ? LANES : threads;
    const int l = LANES ? threadIdx.x % (LANES ? LANES : 1) : threadIdx.x;
    const int64_t row0 = (int64_t)blockIdx.x * (GROUPS * R) + (LANES ? threadIdx.x / (LANES ? LANES : 1) : 0);
    uint4 xs[R][V], rs[R][V];
#pragma unroll
    for (int k = 0; k < R; ++k) {
        const int64_t row = row0 + k * GROUPS, base = row * nvec;
#pragma unroll
        for (int u = 0; u < V; ++u) {
            const int v = l + u * step;
            xs[k][u] = rs[k][u] = make_uint4(0, 0, 0, 0);
            if (v < nvec && row < a.rows) {
                xs[k][u] = take<FAR>(reinterpret_cast<const uint4*>(a.x) + base + v);
                if (a.residual) rs[k][u] = take<FAR>(reinterpret_cast<const uint4*>(a.residual) + base + v);
            }
        }
    }
    float w[V][8];
#pragma unroll
    for (int u = 0; u < V; ++u) weight8(a.weight, a.weight_f32, l + u * step < nvec ? l + u * step : 0, w[u]);
    // vector u of the row's outputs, from its values s
    auto give = [&](int64_t base, int u, const float(&s)[8], float r, bool in) {
        const int v = l + u * step;
        float y[8];
        float m = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            y[i] = s[i] * r * w[u][i];
            m = fmaxf(m, fabsf(y[i]));
        }
        if (in && a.y) put<FAR>(reinterpret_cast<uint4*>(a.y) + base + v, pack8(y));
        if (a.codes) {  // 16 lanes hold a block of 128: all of them are in the row or none
            const Fp8Scale sc = fp8_block_scale(max16(m), a.format);
            if (in) {
                uint2 q;
                q.x = pack_e4m3x4(y[0] * sc.mul, y[1] * sc.mul, y[2] * sc.mul, y[3] * sc.mul);
                q.y = pack_e4m3x4(y[4] * sc.mul, y[5] * sc.mul, y[6] * sc.mul, y[7] * sc.mul);
                put<FAR>(reinterpret_cast<uint2*>(a.codes) + base + v, q);
                if ((v & 15) == 0) {
                    const int64_t at = (base + v) / 16;
                    if (a.format == 2)
                        static_cast<uint8_t*>(a.scales)[at] = (uint8_t)sc.ue8m0;
                    else
                        static_cast<float*>(a.scales)[at] = sc.scale;
                }
            }
        }
    };
    bool faint[R];
#pragma unroll
    for (int k = 0; k < R; ++k) {
        const int64_t row = row0 + k * GROUPS, base = row * nvec;
        float s[V][8];
        float ss[1] = {0.0f};
#pragma unroll
        for (int u = 0; u < V; ++u) {
            float r[8];
            unpack8(xs[k][u], s[u]);
            unpack8(rs[k][u], r);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (a.residual) s[u][i] += r[i];
                ss[0] = __builtin_fmaf(s[u][i], s[u][i], ss[0]);
            }
        }
        row_sums<LANES>(ss, threads, slot[0]);
        const float mean = ss[0] / (float)a.width + a.eps;
        const float r = rsqrtf(mean);
        faint[k] = mean < kFaint && row < a.rows;
#pragma unroll
        for (int u = 0; u < V; ++u) {
            const int v = l + u * step;
            const bool in = v < nvec && row < a.rows && !faint[k];
            if (in && a.sum) put<FAR>(reinterpret_cast<uint4*>(a.sum) + base + v, pack8(s[u]));
            give(base, u, s[u], r, in);
        }
    }
#pragma unroll
    for (int k = 0; k < R; ++k) {
        if (!faint[k]) continue;  // (the same for all lanes of the row)
        const int64_t base = (row0 + k * GROUPS) * nvec;
        float s[V][8];
        float ss[1] = {0.0f};
#pragma unroll
        for (int u = 0; u < V; ++u) {
            const int v = l + u * step;
            uint4 x4 = make_uint4(0, 0, 0, 0), r4 = x4;
            if (v < nvec) {
                x4 = reinterpret_cast<const uint4*>(a.x)[base + v];
                if (a.residual) r4 = reinterpret_cast<const uint4*>(a.residual)[base + v];
            }
            float r[8];
            unpack8(x4, s[u]);
            unpack8(r4, r);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (a.residual) s[u][i] += r[i];
            if (v < nvec && a.sum) reinterpret_cast<uint4*>(a.sum)[base + v] = pack8(s[u]);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                s[u][i] *= kLift;
                ss[0] = __builtin_fmaf(s[u][i], s[u][i], ss[0]);
            }
        }
        row_sums<LANES>(ss, threads, slot[LANES ? 0 : 1]);
        const float r = rsqrtf(ss[0] / (float)a.width + a.eps * kLift * kLift);
#pragma unroll
        for (int u = 0; u < V; ++u) give(base, u, s[u], r, l + u * step < nvec);
    }
}

template <int LANES, int V, int R = 1>
hipError_t norm_rows(const NormArgs& all, int threads, hipStream_t stream) {
    const int rows = LANES ? 256 / (LANES ? LANES : 1) * R : 1;
    const int64_t most = kMaxWorkItems / threads * rows;
    const bool far = all.rows * all.width * (all.residual ? 8 : 4) > kFarBytes;  // (FP8 outputs: as if bf16)
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
        const dim3 grid((unsigned)((a.rows + rows - 1) / rows)), block((unsigned)threads);
        // one vector a lane and one row at a time is for few rows, which are never far
        if (far && (V > 1 || R > 1))
            hipLaunchKernelGGL((norm_kernel<LANES, V, R, (V > 1 || R > 1)>), grid, block, 0, stream, a, threads);
        else
            hipLaunchKernelGGL((norm_kernel<LANES, V, R, false>), grid, block, 0, stream, a, threads);
    }
    return hipGetLastError();
}

// Whether sums of a row have lost bits, or all of them, or are more than fp32 holds: then
// its gradient is worked out by itself, from values that are some power of two larger or
// smaller.
__device__ __forceinline__ bool is_lost(float square, float dot) {
    return !(square >= kFaint && square < __builtin_inff() && fabsf(dot) < __builtin_inff());
}

// Gradient. A block takes every gridDim.x-th group of rows and keeps the weight's gradient of its columns in registers: one row of sums a
// block. Two blocks share a CU, so that one loads while the other adds up: 45 us for
// 4095 x 7168 where one with its next row on the way took 52.
template <int LANES, int V, bool FAR>
__global__ __launch_bounds__(LANES ? 256 : 1024, LANES ? 1 : V > 1 ? 4 : 8) void norm_grad_kernel(const NormGradArgs a, int threads) {
    constexpr int GROUPS = LANES ? 256 / LANES : 1;
    constexpr bool KEPT = V < 4;  // room for the weights in registers: four vectors spill (1000 x 32768: 126 us for 62)
    __shared__ float slot[2][kMaxWaves][2];
    const int nvec = a.width / 8;
    const int step = LANES ? LANES : threads;
    const int l = LANES ? threadIdx.x % (LANES ? LANES : 1) : threadIdx.x;
    float w[KEPT ? V : 1][8], dw[V][8];
    // the weights of vector u of the lane: kept, or loaded again
    auto weights = [&](int u, int from) -> const float(&)[8] {
        if constexpr (KEPT) return w[u];
        weight8(a.weight, a.weight_f32, from + u * step < nvec ? from + u * step : 0, w[0]);
        return w[0];
    };
#pragma unroll
    for (int u = 0; u < V; ++u) {
        if constexpr (KEPT) weight8(a.weight, a.weight_f32, l + u * step < nvec ? l + u * step : 0, w[u]);
#pragma unroll
        for (int i = 0; i < 8; ++i) dw[u][i] = 0.0f;
    }
    int turn = 0;
    bool some = false;  // rows that are lost
    const float mean = 1.0f / (float)a.width;
    int64_t row0 = (int64_t)blockIdx.x * GROUPS;
    const int mine = LANES ? threadIdx.x / (LANES ? LANES : 1) : 0;
    for (; row0 < a.rows; row0 += (int64_t)gridDim.x * GROUPS) {
        const int64_t row = row0 + mine;
        const bool there = row < a.rows;
        const int64_t base = row * nvec;
        uint4 x4[V], g4[V], d4[V];
        const int first = KEPT ? l : afresh(l);
#pragma unroll
        for (int u = 0; u < V; ++u) {
            const int v = first + u * step;
            x4[u] = g4[u] = d4[u] = make_uint4(0, 0, 0, 0);
            if (there && v < nvec) {
                x4[u] = take<FAR>(reinterpret_cast<const uint4*>(a.x) + base + v);
                g4[u] = take<FAR>(reinterpret_cast<const uint4*>(a.grad) + base + v);
                if (KEPT && a.grad_sum) d4[u] = take<FAR>(reinterpret_cast<const uint4*>(a.grad_sum) + base + v);
            }
        }
        const int once = KEPT ? l : afresh(l);
        float sums[2] = {0.0f, 0.0f};  // of s^2, of g s
#pragma unroll
        for (int u = 0; u < V; ++u) {
            float x[8], g[8];
            unpack8(x4[u], x);
            unpack8(g4[u], g);
            const float(&wu)[8] = weights(u, once);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                sums[0] = __builtin_fmaf(x[i], x[i], sums[0]);
                sums[1] = __builtin_fmaf(g[i] * wu[i], x[i], sums[1]);
            }
        }
        // two sets of slots: a wave may be one sum ahead of another's reads, not two
        row_sums<LANES>(sums, threads, slot[turn]);
        turn ^= 1;
        const float square = __builtin_fmaf(sums[0], mean, a.eps);
        const bool lost = is_lost(square, sums[1]) && there;
        some |= lost;
        const float r = rsqrtf(square);
        const float c = sums[1] * r * r * mean;  // times s: h mean(g h)
        const bool kept = there && !lost;  // (r of no row may be infinite)
        const int twice = KEPT ? l : afresh(l);
#pragma unroll
        for (int u = 0; u < V; ++u) {
            const int v = twice + u * step;
            float x[8], g[8], d[8];
            unpack8(x4[u], x);
            unpack8(g4[u], g);
            if (!KEPT && a.grad_sum && there && v < nvec) d4[u] = take<FAR>(reinterpret_cast<const uint4*>(a.grad_sum) + base + v);
            unpack8(d4[u], d);
            const float(&wu)[8] = weights(u, twice);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (kept) dw[u][i] = __builtin_fmaf(g[i] * r, x[i], dw[u][i]);
                const float t = r * (g[i] * wu[i] - x[i] * c);
                d[i] = a.grad_sum ? d[i] + t : t;
            }
            if (a.grad_x && kept && v < nvec) reinterpret_cast<uint4*>(a.grad_x)[base + v] = pack8(d);
        }
    }
    // the lost rows, found by the same sums once more: the same operations, so the same rows
    if (ballot(some) != 0) {
        for (row0 = (int64_t)blockIdx.x * GROUPS; row0 < a.rows; row0 += (int64_t)gridDim.x * GROUPS) {
            const int64_t row = row0 + mine, base = row * nvec;
            const bool there = row < a.rows;
            auto vector = [&](const uint16_t* from, int v, float factor, float(&out)[8]) {
                unpack8(from && there && v < nvec ? reinterpret_cast<const uint4*>(from)[base + v] : make_uint4(0, 0, 0, 0), out);
#pragma unroll
                for (int i = 0; i < 8; ++i) out[i] *= factor;
            };
            auto add_up = [&](float lift, float(&sums)[2]) {
                sums[0] = sums[1] = 0.0f;
#pragma unroll
                for (int u = 0; u < V; ++u) {
                    const int from = afresh(l), v = from + u * step;
                    float x[8], g[8];
                    vector(a.x, v, lift, x);
                    vector(a.grad, v, 1.0f, g);
                    const float(&wu)[8] = weights(u, from);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        sums[0] = __builtin_fmaf(x[i], x[i], sums[0]);
                        sums[1] = __builtin_fmaf(g[i] * wu[i], x[i], sums[1]);
                    }
                    __builtin_amdgcn_sched_barrier(0);
                }
                row_sums<LANES>(sums, threads, slot[turn]);
                turn ^= 1;
            };
            float sums[2];
            add_up(1.0f, sums);
            float square = __builtin_fmaf(sums[0], mean, a.eps);
            if (!is_lost(square, sums[1]) || !there) continue;  // (the same for all lanes of the row)
            const float lift = square < kFaint ? kLift : square < __builtin_inff() ? 0x1p-40f : 0x1p-112f;
            add_up(lift, sums);
            square = sums[0] * mean + a.eps * lift * lift;
            const float r = rsqrtf(square), c = sums[1] * r * mean;  // mean(g h)
            // of the row as it is, r is r * lift: in two steps where that may be infinite
            const float down = r * fminf(lift, 1.0f), up = fmaxf(lift, 1.0f);
#pragma unroll
            for (int u = 0; u < V; ++u) {
                const int from = afresh(l), v = from + u * step;
                float x[8], g[8], d[8];
                vector(a.x, v, lift, x);
                vector(a.grad, v, 1.0f, g);
                vector(a.grad_sum, v, 1.0f, d);
                const float(&wu)[8] = weights(u, from);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float h = x[i] * r;
                    dw[u][i] = __builtin_fmaf(g[i], h, dw[u][i]);
                    const float t = down * (g[i] * wu[i] - h * c) * up;
                    d[i] = a.grad_sum ? d[i] + t : t;
                }
                if (a.grad_x && v < nvec) reinterpret_cast<uint4*>(a.grad_x)[base + v] = pack8(d);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    }
    if (!a.partial) return;
    float* const out = a.partial + (int64_t)blockIdx.x * a.width;
    if constexpr (LANES > 0) {  // the block's groups of lanes, in order
        __shared__ float part[256][9];
#pragma unroll
        for (int u = 0; u < V; ++u) {
            __syncthreads();
#pragma unroll
            for (int i = 0; i < 8; ++i) part[threadIdx.x][i] = dw[u][i];
            __syncthreads();
            for (int c = threadIdx.x; c < LANES * 8; c += 256) {
                float s = 0.0f;
#pragma unroll
                for (int k = 0; k < GROUPS; ++k) s += part[k * LANES + c / 8][c % 8];
                if (c + u * LANES * 8 < a.width) out[c + u * LANES * 8] = s;
            }
        }
    } else {
#pragma unroll
        for (int u = 0; u < V; ++u) {
            const int v = l + u * step;
            if (v >= nvec) continue;
            reinterpret_cast<float4*>(out)[2 * v] = make_float4(dw[u][0], dw[u][1], dw[u][2], dw[u][3]);
            reinterpret_cast<float4*>(out)[2 * v + 1] = make_float4(dw[u][4], dw[u][5], dw[u][6], dw[u][7]);
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

template <int LANES, int V>
void norm_grad_rows(const NormGradArgs& a, int64_t blocks, int threads, hipStream_t stream) {
    if (a.rows * a.width * (a.grad_sum ? 8 : 6) > kFarBytes)
        hipLaunchKernelGGL((norm_grad_kernel<LANES, V, true>), dim3((unsigned)blocks), dim3((unsigned)threads), 0, stream, a, threads);
    else
        hipLaunchKernelGGL((norm_grad_kernel<LANES, V, false>), dim3((unsigned)blocks), dim3((unsigned)threads), 0, stream, a, threads);
}

// Threads of a block that holds a row with V vectors a lane.
int row_threads(int width, int v) { return (width / 8 + kWave * v - 1) / (kWave * v) * kWave; }

constexpr int kRowsTogether = 2;  // of small widths, where there are many
// Vectors a lane of a row that has a block. Few rows get as many threads as they have
// vectors; otherwise two vectors leave fewest lanes without one (4096 x 7168: 47 us;
// four 53), and the gradient has room for one in 64 registers.
int forward_vectors(int64_t rows, int width) { return width <= 8192 ? (rows <= 512 ? 1 : 2) : width <= 16384 && rows <= 512 ? 2 : 4; }
int gradient_vectors(int width) { return width <= 8192 ? 1 : width <= 16384 ? 2 : 4; }

}  // namespace

hipError_t launch_norm(const NormArgs& a, hipStream_t stream) {
    if (a.rows == 0) return hipSuccess;
    const int w = a.width;
    // Several rows a block; many rows: two at a time. us with one and two: 66000 x 128 with a residual
    // 12.3 and 11.1, 131040 x 128 13.2 and 13.0, with a residual 21.7 and 20.2, 33000 x 512 with one 22.0 and
    // 20.6; but 262144 x 128 with a residual 39.6 and 43.3, and to FP8 33000 x 512 13.1 and 14.6.
    if (w <= 512) {
        const int lanes = w <= 128 ? 16 : w <= 256 ? 32 : 64;
        const bool many = a.rows * lanes >= int64_t(256) * 2048 * kRowsTogether;
        if (lanes == 16) return many ? norm_rows<16, 1, kRowsTogether>(a, 256, stream) : norm_rows<16, 1>(a, 256, stream);
        if (lanes == 32) return many ? norm_rows<32, 1, kRowsTogether>(a, 256, stream) : norm_rows<32, 1>(a, 256, stream);
        return many ? norm_rows<64, 1, kRowsTogether>(a, 256, stream) : norm_rows<64, 1>(a, 256, stream);
    }
    if (w <= 1024) return norm_rows<64, 2>(a, 256, stream);
    const int v = forward_vectors(a.rows, w);
    const int threads = row_threads(w, v);
    if (v == 1) return norm_rows<0, 1>(a, threads, stream);
    if (v == 2) return norm_rows<0, 2>(a, threads, stream);
    return norm_rows<0, 4>(a, threads, stream);
}

// Each block writes a row of sums for the weight's gradient, so only as many as keep the
// CUs busy: 1024 threads a CU, two blocks (16000 x 2048: 41 us with four blocks a CU, 49
// with two, 46 with eight; 8000 x 4096: 39 with two, 42 with four), and one where a lane
// has several vectors (2000 x 16384: 45 us, 50 with two). Rows for a few turns are shared
// out evenly (300 x 16384: 15.3 us for 20.4).
int64_t norm_grad_blocks(int64_t rows, int width) {
    const int per = width <= 128 ? 16 : width <= 256 ? 8 : width <= 1024 ? 4 : 1;  // rows at a time
    const int64_t groups = (rows + per - 1) / per;
    const int v = gradient_vectors(width), threads = row_threads(width, v);
    const int64_t most = width <= 1024 ? 1024 : 256 * (v > 1 ? 1 : threads > 512 ? 2 : 1024 / threads);
    const int64_t turns = (groups + most - 1) / most;
    return turns > 0 && turns <= 4 ? (groups + turns - 1) / turns : groups < most ? groups : most;
}

hipError_t launch_norm_grad(const NormGradArgs& a, hipStream_t stream) {
    const int w = a.width;
    const int64_t blocks = norm_grad_blocks(a.rows, w);
    if (blocks > 0) {
        const int v = gradient_vectors(w);
        if (w <= 128)
            norm_grad_rows<16, 1>(a, blocks, 256, stream);
        else if (w <= 256)
            norm_grad_rows<32, 1>(a, blocks, 256, stream);
        else if (w <= 512)
            norm_grad_rows<64, 1>(a, blocks, 256, stream);
        else if (w <= 1024)
            norm_grad_rows<64, 2>(a, blocks, 256, stream);
        else if (v == 1)
            norm_grad_rows<0, 1>(a, blocks, row_threads(w, 1), stream);
        else if (v == 2)
            norm_grad_rows<0, 2>(a, blocks, row_threads(w, 2), stream);
        else
            norm_grad_rows<0, 4>(a, blocks, row_threads(w, 4), stream);
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
