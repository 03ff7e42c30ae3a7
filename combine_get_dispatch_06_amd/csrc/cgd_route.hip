// Router: scores -> the experts of each token and their weights, and back.
//
//   l  = logit (NaN counts as -inf, +inf as the largest finite fp32)
//   s  = softmax(l) or sigmoid(l)
//   c  = s + bias; without a bias, and with no groups or groups judged by their
//        best expert alone, c = l, which orders the same way
//   groups of E / G experts: value = sum of the group's `group_top` largest c;
//        the topk_groups best groups stay
//   the K largest c of those, descending; ties go to the lowest index
//   w  = scale * s, or scale * s / (sum of s over the chosen) when renormalised
// An expert with l = -inf, or c = -inf or NaN, is never chosen; slots left
// over get index -1 and weight 0, which layout, dispatch and combine skip.
//
// One wave per token; lane i holds experts i, i + 64, ... Choosing by rounds of
// a wave-wide maximum costs K reductions one after another, so the wave finds a
// threshold instead: the largest value that at least K of the 64 lane maxima
// reach (binary search with ballots). Everything that reaches it (a few more
// than K) is gathered, one candidate per lane, and each candidate counts the
// candidates ahead of it: that count is its place. More than 64 candidates
// (long ties) take the rounds.
// Values next to each other are told apart exactly: c is compared in 64 bits
// wherever a score enters it (the fp32 used for the threshold is rounded from
// it, and rounding keeps the order), logits as they are.
#include "cgd_device.h"
#include "cgd_experts_launch.h"

namespace cgd {

constexpr int kRouteWaves = 4;
constexpr int kRouteMaxGroups = 64;

// fp32 -> unsigned with the same order; 0 is below every value
__device__ __forceinline__ uint32_t order_key(float v) {
    const uint32_t b = __float_as_uint(v);
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
    for (int d = 32; d; d >>= 1) v = fmaxf(v, __shfl_xor(v, d, kWave));
    return v;
}
// LDS writes of this wave's lanes before its reads that follow
__device__ __forceinline__ void wave_fence() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}
template <typename T>
__device__ __forceinline__ T wave_sum(T v) {
#pragma unroll
    for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d, kWave);
    return v;
}
__device__ __forceinline__ uint32_t wave_umax(uint32_t v) {
#pragma unroll
    for (int d = 32; d; d >>= 1) {
        const uint32_t o = __shfl_xor(v, d, kWave);
        v = o > v ? o : v;
    }
    return v;
}
__device__ __forceinline__ uint64_t wave_umax64(uint64_t v) {
#pragma unroll
    for (int d = 32; d; d >>= 1) {
        const uint64_t o = __shfl_xor((unsigned long long)v, d, kWave);
        v = o > v ? o : v;
    }
    return v;
}

__device__ __forceinline__ float load_logit(const void* p, bool bf16, int64_t i) {
    float v = bf16 ? __uint_as_float((uint32_t) static_cast<const uint16_t*>(p)[i] << 16) : static_cast<const float*>(p)[i];
    if (!(v == v)) v = -INFINITY;
    return v > 3.402823466e38f ? 3.402823466e38f : v;
}

// 64-bit doubles as unsigned with the same order (-0 counts as +0)
__device__ __forceinline__ uint64_t order_key64(double v) {
    const uint64_t b = (uint64_t)__double_as_longlong(v + 0.0);
    return (b >> 63) ? ~b : (b | 0x8000000000000000ull);
}

// WIDE: choices in 64 bits. PER: experts per lane.
template <bool WIDE, int PER>
__global__ __launch_bounds__(kRouteWaves* kWave) void route_kernel(const RouteArgs a) {
    __shared__ uint64_t cand_key[kRouteWaves][kWave];
    __shared__ int cand_id[kRouteWaves][kWave];
    __shared__ double all[WIDE ? kRouteWaves : 1][WIDE ? PER * kWave : 1];
    const int lane = lane_id();
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int64_t t = (int64_t)blockIdx.x * kRouteWaves + wave;
    if (t >= a.T) return;  // waves are independent: no block barrier below

    float l[PER];
    float top = -INFINITY;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        const int e = lane + j * kWave;
        l[j] = e < a.E ? load_logit(a.logits, a.logits_bf16, t * a.E + e) : -INFINITY;
        top = fmaxf(top, l[j]);
    }
    top = wave_max(top);
    const bool none = top == -INFINITY;

    // choice values
    double c[WIDE ? PER : 1];
    double norm = 1.0;  // softmax denominator
    if (WIDE) {
        if (!a.sigmoid) {
            double s = 0.0;
#pragma unroll
            for (int j = 0; j < PER; ++j) {
                c[j] = none ? 0.0 : exp((double)l[j] - (double)top);
                s += c[j];
            }
            norm = wave_sum(s);
        }
        const bool by_logit = !a.bias && a.group_top == 1;
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const int e = lane + j * kWave;
            double v = by_logit ? (double)l[j] : a.sigmoid ? 1.0 / (1.0 + exp(-(double)l[j])) : c[j] / norm;
            if (a.bias && e < a.E) v += (double)a.bias[e];
            if (!(v == v) || l[j] == -INFINITY) v = -INFINITY;
            c[j] = v;
        }
    } else if (!a.sigmoid && !a.renormalize) {
        float s = 0.0f;
#pragma unroll
        for (int j = 0; j < PER; ++j) s += none ? 0.0f : expf(l[j] - top);
        norm = (double)wave_sum(s);
    }

    // groups
    uint64_t keep = ~0ull;
    const int per_group = a.E / a.groups;
    if (a.groups > 1 && a.topk_groups < a.groups) {
        double v = -INFINITY;
        if (WIDE) {
#pragma unroll
            for (int j = 0; j < PER; ++j) all[wave][lane + j * kWave] = c[j];
        }
        wave_fence();
        if (WIDE) {
            if (lane < a.groups) {
                double b1 = -INFINITY, b2 = -INFINITY;
                for (int i = 0; i < per_group; ++i) {
                    const double x = all[wave][lane * per_group + i];
                    b2 = fmax(b2, fmin(b1, x));
                    b1 = fmax(b1, x);
                }
                v = b1;
                if (a.group_top == 2 && b2 > -INFINITY) v += b2;
            }
        }
        const uint64_t key = lane < a.groups && v > -INFINITY ? order_key64(v) : 0ull;
        int ahead = 0;
        for (int i = 0; i < a.groups; ++i) {
            const uint64_t o = ((uint64_t)__builtin_amdgcn_readlane((int)(uint32_t)(key >> 32), i) << 32) |
                               (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)key, i);
            ahead += (o > key || (o == key && i < lane)) ? 1 : 0;
        }
        keep = ballot(lane < a.groups && ahead < a.topk_groups);
    }

    // threshold
    uint32_t k32[PER];
    uint32_t mine = 0;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        const int e = lane + j * kWave;
        bool ok = e < a.E && l[j] > -INFINITY;
        if (WIDE) ok = ok && c[j] > -INFINITY;
        if (a.groups > 1 && ok) ok = (keep >> (e / per_group)) & 1;
        const float v = WIDE ? (float)c[j] + 0.0f : l[j] + 0.0f;
        k32[j] = ok ? order_key(v) : 0u;
        mine = k32[j] > mine ? k32[j] : mine;
    }
    uint32_t lo = 1u;
    if (a.E > kWave && __popcll(ballot(mine >= 1u)) > a.K) {
        // invariant: at least K lanes reach lo, fewer than K reach hi
        uint32_t hi = wave_umax(mine);
        if (__popcll(ballot(mine >= hi)) >= a.K) {
            lo = hi;
        } else {
            while (hi - lo > 1) {
                const uint32_t mid = lo + (hi - lo) / 2;
                const int n = __popcll(ballot(mine >= mid));
                if (n >= a.K) {
                    lo = mid;
                    if (n <= a.K + 4) break;
                } else {
                    hi = mid;
                }
            }
        }
    }
    int found = 0;
#pragma unroll
    for (int j = 0; j < PER; ++j) found += __popcll(ballot(k32[j] >= lo));

    // candidates -> places
    int id = -1, place = 1 << 20;
    if (found <= kWave) {
        int at = 0;
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const uint64_t m = ballot(k32[j] >= lo);
            if (k32[j] >= lo) {
                const int p = at + __popcll(m & lanemask_lt());
                cand_key[wave][p] = WIDE ? order_key64(c[j]) : (uint64_t)k32[j];
                cand_id[wave][p] = lane + j * kWave;
            }
            at += __popcll(m);
        }
        wave_fence();
        uint64_t key = 0;
        if (lane < found) {
            key = cand_key[wave][lane];
            id = cand_id[wave][lane];
        }
        int ahead = 0;
        for (int i = 0; i < found; ++i) {
            const uint32_t oh = __builtin_amdgcn_readlane((int)(uint32_t)(key >> 32), i);
            const uint32_t ol = __builtin_amdgcn_readlane((int)(uint32_t)key, i);
            const int oi = __builtin_amdgcn_readlane(id, i);
            const uint64_t o = ((uint64_t)oh << 32) | ol;
            ahead += (o > key || (o == key && oi < id)) ? 1 : 0;
        }
        if (lane < found) place = ahead;
    } else {
        // rounds: the best value, then among its holders the lowest index
        for (int k = 0; k < a.K; ++k) {
            uint64_t best = 0;
#pragma unroll
            for (int j = 0; j < PER; ++j) {
                const uint64_t key = k32[j] ? (WIDE ? order_key64(c[j]) : (uint64_t)k32[j]) : 0ull;
                best = key > best ? key : best;
            }
            best = wave_umax64(best);
            if (best == 0) break;
            uint32_t first = 0;  // largest of ~index: the lowest index
#pragma unroll
            for (int j = 0; j < PER; ++j) {
                const uint64_t key = k32[j] ? (WIDE ? order_key64(c[j]) : (uint64_t)k32[j]) : 0ull;
                const uint32_t inv = ~(uint32_t)(lane + j * kWave);
                if (key == best && inv > first) first = inv;
            }
            const int e = (int)~wave_umax(first);
#pragma unroll
            for (int j = 0; j < PER; ++j)
                if (lane + j * kWave == e) k32[j] = 0u;
            if (lane == k) {
                id = e;
                place = k;
            }
        }
    }

    // weights of the chosen
    const bool chosen = id >= 0 && place < a.K;
    double s = 0.0;
    if (chosen) {
        const float x = load_logit(a.logits, a.logits_bf16, t * a.E + id);
        if (a.sigmoid)
            s = 1.0 / (1.0 + exp(-(double)x));
        else
            s = WIDE ? exp((double)x - (double)top) / norm : (double)expf(x - top) / norm;
    }
    if (a.renormalize) {
        const double total = wave_sum(s);
        s = total > 0.0 ? s / total : 0.0;
    }
    if (chosen) {
        a.topk_idx[t * a.K + place] = id;
        a.topk_weights[t * a.K + place] = (float)(s * (double)a.scale);
    }
    const int n = __popcll(ballot(chosen));
    if (lane >= n && lane < a.K) {
        a.topk_idx[t * a.K + lane] = -1;
        a.topk_weights[t * a.K + lane] = 0.0f;
    }
}

// Gradient of the weights with respect to the logits:
//   softmax:               dl_e = scale * p_e * (G_e - sum_i G_i p_i), G_e = sum of g over e's slots
//   softmax, renormalised: the same over the chosen alone (p renormalised)
//   sigmoid:               dl_e = scale * G_e * s_e (1 - s_e)
//   sigmoid, renormalised: dl_e = scale * sum over e's slots (g - sum_j g_j s_j / S) / S * s_e (1 - s_e), S = sum_j s_j
// One wave per token, one pass. An expert that appears in several slots of a
// token collects them in slot order; values outside [0, E) are no slot.
template <int PER>
__global__ __launch_bounds__(kRouteWaves* kWave) void route_grad_kernel(const RouteGradArgs a) {
    __shared__ float slot_grad[kRouteWaves][PER * kWave];
    const int lane = lane_id();
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int64_t t = (int64_t)blockIdx.x * kRouteWaves + wave;
    if (t >= a.T) return;
    float l[PER];
    float top = -INFINITY;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        const int e = lane + j * kWave;
        l[j] = e < a.E ? load_logit(a.logits, a.logits_bf16, t * a.E + e) : -INFINITY;
        top = fmaxf(top, l[j]);
        slot_grad[wave][e] = 0.0f;
    }
    int id = -1;
    float g = 0.0f, x = -INFINITY;
    if (lane < a.K) {
        const int64_t i = a.topk_idx[t * a.K + lane];
        if (i >= 0 && i < a.E) {
            id = (int)i;
            g = a.grad_weights[t * a.K + lane] * a.scale;
            x = load_logit(a.logits, a.logits_bf16, t * a.E + id);
        }
    }
    top = wave_max(top);
    const bool none = top == -INFINITY;

    // score of the slot's expert, and the denominators
    float ps, inv = 1.0f;
    if (a.sigmoid) {
        ps = id >= 0 ? 1.0f / (1.0f + expf(-x)) : 0.0f;
    } else {
        ps = id >= 0 && !none ? expf(x - top) : 0.0f;
    }
    float p[PER];
    if (a.sigmoid) {
#pragma unroll
        for (int j = 0; j < PER; ++j) p[j] = 1.0f / (1.0f + expf(-l[j]));
    } else {
        float sum = 0.0f;
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            p[j] = none ? 0.0f : expf(l[j] - top);
            sum += p[j];
        }
        sum = wave_sum(sum);
        inv = sum > 0.0f ? 1.0f / sum : 0.0f;
#pragma unroll
        for (int j = 0; j < PER; ++j) p[j] *= inv;
        ps *= inv;
    }
    if (a.renormalize) {
        // a chosen share of the chosen total: its gradient in the scores first
        const float total = wave_sum(ps);
        const float it = total > 0.0f ? 1.0f / total : 0.0f;
        const float dot = wave_sum(g * ps) * it;
        g = id >= 0 ? (g - dot) * it : 0.0f;
    }
    // one sum for each expert, in slot order, written by its first slot
    float sum = 0.0f;
    bool first = id >= 0;
    for (int k = 0; k < a.K; ++k) {
        const int oi = __builtin_amdgcn_readlane(id, k);
        const float og = __uint_as_float(__builtin_amdgcn_readlane((int)__float_as_uint(g), k));
        if (oi == id) {
            sum += og;
            if (k < lane) first = false;
        }
    }
    wave_fence();
    if (first) slot_grad[wave][id] = sum;
    wave_fence();
    const float dot = a.sigmoid ? 0.0f : wave_sum(id >= 0 ? g * ps : 0.0f);
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        const int e = lane + j * kWave;
        if (e >= a.E) continue;
        const float G = slot_grad[wave][e];
        const float d = a.sigmoid ? G * p[j] * (1.0f - p[j]) : p[j] * (G - dot);
        if (a.logits_bf16)
            static_cast<uint16_t*>(a.grad_logits)[t * a.E + e] = (uint16_t)pack_bf16x2(d, 0.0f);
        else
            static_cast<float*>(a.grad_logits)[t * a.E + e] = d;
    }
}

template <bool WIDE>
static void route_launch(const RouteArgs& a, hipStream_t stream) {
    const dim3 grid((unsigned)((a.T + kRouteWaves - 1) / kRouteWaves)), block(kRouteWaves * kWave);
    if (a.E <= 64)
        hipLaunchKernelGGL((route_kernel<WIDE, 1>), grid, block, 0, stream, a);
    else if (a.E <= 128)
        hipLaunchKernelGGL((route_kernel<WIDE, 2>), grid, block, 0, stream, a);
    else if (a.E <= 256)
        hipLaunchKernelGGL((route_kernel<WIDE, 4>), grid, block, 0, stream, a);
    else
        hipLaunchKernelGGL((route_kernel<WIDE, 8>), grid, block, 0, stream, a);
}

hipError_t launch_route(const RouteArgs& a, hipStream_t stream) {
    if (a.T == 0) return hipSuccess;
    if (a.bias || a.groups > 1)
        route_launch<true>(a, stream);
    else
        route_launch<false>(a, stream);
    return hipGetLastError();
}

hipError_t launch_route_grad(const RouteGradArgs& a, hipStream_t stream) {
    if (a.T == 0) return hipSuccess;
    const dim3 grid((unsigned)((a.T + kRouteWaves - 1) / kRouteWaves)), block(kRouteWaves * kWave);
    if (a.E <= 64)
        hipLaunchKernelGGL((route_grad_kernel<1>), grid, block, 0, stream, a);
    else if (a.E <= 128)
        hipLaunchKernelGGL((route_grad_kernel<2>), grid, block, 0, stream, a);
    else if (a.E <= 256)
        hipLaunchKernelGGL((route_grad_kernel<4>), grid, block, 0, stream, a);
    else
        hipLaunchKernelGGL((route_grad_kernel<8>), grid, block, 0, stream, a);
    return hipGetLastError();
}

hipError_t preload_route() {
    hipFuncAttributes at;
    return hipFuncGetAttributes(&at, reinterpret_cast<const void*>(&route_grad_kernel<8>));
}

}  // namespace cgd
