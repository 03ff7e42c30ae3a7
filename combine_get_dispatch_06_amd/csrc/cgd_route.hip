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
constexpr float kZeroScore = 745.0f;  // exp of less than its negative is zero in 64 bits

// fp32 -> unsigned with the same order; kNone is -inf, and there is nothing below it
constexpr uint32_t kNone = 0x007FFFFFu;
__device__ __forceinline__ uint32_t order_key(float v) {
    const uint32_t b = __float_as_uint(v);
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

__device__ __forceinline__ float from_key(uint32_t k) {
    return __uint_as_float((k & 0x80000000u) ? k & 0x7FFFFFFFu : ~k);
}

// Reductions over the wave, by lane moves within the vector unit: shifts by 1, 2,
// 4 and 8 within rows of 16 lanes, then each row's last lane to the rows behind.
// Lanes that a move does not reach get 0, which changes neither a sum nor a
// maximum of unsigned values, so that move and operation are one instruction.
// Lane 63 ends up with all 64.
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t moved(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xF, ROWS == 0xF);
}
template <typename F>
__device__ __forceinline__ uint32_t wave_reduce(uint32_t v, F f) {
    v = f(v, moved<0x111, 0xF>(v));
    v = f(v, moved<0x112, 0xF>(v));
    v = f(v, moved<0x114, 0xF>(v));
    v = f(v, moved<0x118, 0xF>(v));
    v = f(v, moved<0x142, 0xA>(v));  // rows 1 and 3 from the row before
    v = f(v, moved<0x143, 0xC>(v));  // rows 2 and 3 from row 1
    return (uint32_t)__builtin_amdgcn_readlane((int)v, kWave - 1);
}
__device__ __forceinline__ uint32_t wave_umax(uint32_t v) {
    return wave_reduce(v, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
}
__device__ __forceinline__ uint32_t wave_umin(uint32_t v) { return ~wave_umax(~v); }
__device__ __forceinline__ uint32_t wave_usum(uint32_t v) {
    return wave_reduce(v, [](uint32_t a, uint32_t b) { return a + b; });
}
__device__ __forceinline__ float wave_max(float v) { return from_key(wave_umax(order_key(v))); }
__device__ __forceinline__ float wave_sum(float v) {
    return __uint_as_float(wave_reduce(__float_as_uint(v), [](uint32_t a, uint32_t b) {
        return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
    }));
}
__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
    for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d, kWave);
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

// LDS writes of this wave's lanes before its reads that follow
__device__ __forceinline__ void wave_fence() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// A logit as fp32, cleaned: NaN counts as -inf, +inf as the largest finite value.
__device__ __forceinline__ float clean(float v) {
    return fminf(fmaxf(v, -INFINITY), 3.402823466e38f);  // fmaxf gives the other operand for NaN
}
template <bool BF16>
__device__ __forceinline__ float raw_logit(const void* p, int64_t i) {
    return BF16 ? __uint_as_float((uint32_t) static_cast<const uint16_t*>(p)[i] << 16) : static_cast<const float*>(p)[i];
}
template <bool BF16>
__device__ __forceinline__ float load_logit(const void* p, int64_t i) {
    return clean(raw_logit<BF16>(p, i));
}
// A lane's logits of token t, still uncleaned (nothing waits for them here).
template <bool BF16, int PER>
__device__ __forceinline__ void fetch_logits(const void* p, int64_t t, int64_t T, int E, float (&v)[PER]) {
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        const int e = lane_id() + j * kWave;
        v[j] = e < E && t < T ? raw_logit<BF16>(p, t * E + e) : -INFINITY;
    }
}

// 64-bit doubles as unsigned with the same order (-0 counts as +0)
__device__ __forceinline__ uint64_t order_key64(double v) {
    const uint64_t b = (uint64_t)__double_as_longlong(v + 0.0);
    return (b >> 63) ? ~b : (b | 0x8000000000000000ull);
}

// Bound by vector instructions (some 340 a token) and their latency, so 28 waves of
// a CU that each wait for their own token hide it: fewer waves that take tokens in
// turn with the next one's logits on their way hold twice the registers and measured
// 39 us against 35 at the time; 31 us now (top-16 of 512, 32768 tokens in fp32: 2.4
// TB/s, memory alone would take 11). 128 tokens of 256 experts with groups: 7.6 us, of
// which an empty launch is 2; the rest is one token's latency (the groups' scan, one lane
// a group, reads LDS with bank conflicts in half of its cycles).
// WIDE: choices in 64 bits. PER: experts per lane.
template <bool WIDE, bool BF16, int PER>
__global__ __launch_bounds__(kRouteWaves* kWave) void route_kernel(const RouteArgs a) {
    __shared__ uint64_t cand_key[kRouteWaves][kWave];
    __shared__ int cand_id[kRouteWaves][kWave];
    __shared__ float cand_x[kRouteWaves][kWave];
    __shared__ double all[WIDE ? kRouteWaves : 1][WIDE ? PER * kWave : 1];
    const int lane = lane_id();
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int64_t t = (int64_t)blockIdx.x * kRouteWaves + wave;
    if (t >= a.T) return;  // waves are independent: no block barrier below
    float l[PER];
    fetch_logits<BF16>(a.logits, t, a.T, a.E, l);
    float top = -INFINITY;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        l[j] = clean(l[j]);
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
    const int per_group = WIDE ? a.E / a.groups : 1;
    if (WIDE && a.groups > 1 && a.topk_groups < a.groups) {
        double v = -INFINITY;
        if (WIDE) {
#pragma unroll
            for (int j = 0; j < PER; ++j) all[wave][lane + j * kWave] = c[j];
        }
        wave_fence();
        if (WIDE) {
            if (lane < a.groups) {
                double b1 = -INFINITY, b2 = -INFINITY;
                int i = 0;
                for (; i + 8 <= per_group; i += 8) {  // eight reads on their way at a time
                    double x[8];
#pragma unroll
                    for (int u = 0; u < 8; ++u) x[u] = all[wave][lane * per_group + i + u];
#pragma unroll
                    for (int u = 0; u < 8; ++u) {
                        b2 = fmax(b2, fmin(b1, x[u]));
                        b1 = fmax(b1, x[u]);
                    }
                }
                for (; i < per_group; ++i) {
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
        float v = WIDE ? (float)c[j] + 0.0f : l[j] + 0.0f;
        if (WIDE && a.groups > 1 && e < a.E && !((keep >> (e / per_group)) & 1)) v = -INFINITY;
        k32[j] = order_key(v);  // -inf: kNone
        mine = k32[j] > mine ? k32[j] : mine;
    }
    uint32_t lo = kNone + 1u;
    if (a.E > kWave && __popcll(ballot(mine > kNone)) > a.K) {
        // invariant: at least K lanes reach lo, fewer than K reach hi
        const uint32_t least = wave_umin(mine);
        lo = least > lo ? least : lo;
        uint32_t hi = WIDE ? wave_umax(mine) : order_key(top + 0.0f);
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
    float x = -INFINITY;  // the candidate's logit
    if (found <= kWave) {
        int at = 0;
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const uint64_t m = ballot(k32[j] >= lo);
            if (k32[j] >= lo) {
                const int p = at + __builtin_amdgcn_mbcnt_hi((uint32_t)(m >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)m, 0u));
                cand_x[wave][p] = l[j];
                if (WIDE) {
                    cand_key[wave][p] = order_key64(c[j]);
                    cand_id[wave][p] = lane + j * kWave;
                } else {
                    cand_key[wave][p] = ((uint64_t)k32[j] << 32) | (uint32_t)(lane + j * kWave);
                }
            }
            at += __popcll(m);
        }
        wave_fence();
        uint64_t key = 0;
        if (lane < found) {
            key = cand_key[wave][lane];
            id = WIDE ? cand_id[wave][lane] : (int)(uint32_t)key;
            if (!WIDE) key >>= 32;
            x = cand_x[wave][lane];
        }
        // the candidates are in ascending order of index: of equal values the one
        // in a lower lane is ahead
        uint32_t ahead = 0;
        if (WIDE) {
            for (int i = 0; i < found; ++i) {
                const uint64_t o = ((uint64_t)__builtin_amdgcn_readlane((int)(uint32_t)(key >> 32), i) << 32) |
                                   (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)key, i);
                ahead += o > key ? 1u : 0u;
            }
        } else {
            const uint32_t k = (uint32_t)key;
            for (int i = 0; i < found; ++i) ahead += (uint32_t)__builtin_amdgcn_readlane((int)k, i) > k ? 1u : 0u;
        }
        // without equal values the places are 0 .. found - 1
        if (wave_usum(lane < found ? ahead : 0u) != (uint32_t)(found * (found - 1) / 2)) {
            for (int i = 0; i < found; ++i) {
                const uint64_t o = ((uint64_t)__builtin_amdgcn_readlane((int)(uint32_t)(key >> 32), i) << 32) |
                                   (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)key, i);
                ahead += o == key && i < lane ? 1u : 0u;
            }
        }
        if (lane < found) place = (int)ahead;
    } else {
        // rounds: the best value, then among its holders the lowest index
        for (int k = 0; k < a.K; ++k) {
            uint64_t best = 0;
#pragma unroll
            for (int j = 0; j < PER; ++j) {
                const uint64_t key = k32[j] > kNone ? (WIDE ? order_key64(c[j]) : (uint64_t)k32[j]) : 0ull;
                best = key > best ? key : best;
            }
            best = wave_umax64(best);
            if (best == 0) break;
            uint32_t first = 0;  // largest of ~index: the lowest index
#pragma unroll
            for (int j = 0; j < PER; ++j) {
                const uint64_t key = k32[j] > kNone ? (WIDE ? order_key64(c[j]) : (uint64_t)k32[j]) : 0ull;
                const uint32_t inv = ~(uint32_t)(lane + j * kWave);
                if (key == best && inv > first) first = inv;
            }
            const int e = (int)~wave_umax(first);
#pragma unroll
            for (int j = 0; j < PER; ++j)
                if (lane + j * kWave == e) k32[j] = kNone;
            if (lane == k) {
                id = e;
                place = k;
                x = load_logit<BF16>(a.logits, t * a.E + e);
            }
        }
    }

    // Weights of the chosen, in fp32: off by 5.3e-8 of their size (root mean square), of
    // which the rounding of the result is 2.5e-8; exponentials in 64 bits are for the choice.
    const bool chosen = id >= 0 && place < a.K;
    float s = 0.0f;
    // Renormalised softmax needs no denominator: it cancels. Its exponentials are relative
    // to the largest chosen logit, which a bias or groups can leave far below the token's
    // largest (without them that one is chosen): relative to that one they would lose their
    // bits from 87 below on and be zero at 104. A token whose chosen scores are all zero in
    // 64 bits, too, has no shares.
    const bool shares = a.renormalize && !a.sigmoid;
    const float ref = WIDE && shares ? wave_max(chosen ? x : -INFINITY) : top;
    if (chosen) {
        s = a.sigmoid ? 1.0f / (1.0f + expf(-x)) : expf(x - ref);
        if (shares)
            s = top - ref > kZeroScore ? 0.0f : s;
        else if (!a.sigmoid)
            s /= (float)norm;
    }
    if (a.renormalize) {
        if (a.sigmoid && wave_max(s) < 1e-30f) {  // scores this small: all of them scaled up by the same factor
            const float best = wave_max(chosen ? x : -INFINITY);
            s = chosen && best > -kZeroScore ? expf(x - best) : 0.0f;
        }
        const float total = wave_sum(s);
        s = total > 0.0f ? s / total : 0.0f;
    }
    if (chosen) {
        a.topk_idx[t * a.K + place] = id;
        a.topk_weights[t * a.K + place] = s * a.scale;
    }
    const int n = __popcll(ballot(chosen));
    if (lane >= n && lane < a.K) {
        a.topk_idx[t * a.K + lane] = -1;
        a.topk_weights[t * a.K + lane] = 0.0f;
    }
}

// Gradient of the weights with respect to the logits:
//   softmax:               dl_e = scale * p_e * (G_e - sum_i G_i p_i), G_e = sum of g over e's slots
//   sigmoid:               dl_e = scale * G_e * s_e (1 - s_e)
//   renormalised, with shares w = s / (sum of s over the slots):
//                          dl_e = scale * w_e * sum over e's slots (g - sum_j g_j w_j), times (1 - s_e) for sigmoid
// One wave per token, one pass. An expert that appears in several slots of a
// token collects them in slot order; values outside [0, E) are no slot. Bound by
// latency: 7.2 us for 8191 tokens of 256 experts in bf16 (9.2 MB, 1.4 us of memory).
template <bool BF16, int PER>
__global__ __launch_bounds__(kRouteWaves* kWave) void route_grad_kernel(const RouteGradArgs a) {
    __shared__ float slot_grad[kRouteWaves][PER * kWave];
    const int lane = lane_id();
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int64_t t = (int64_t)blockIdx.x * kRouteWaves + wave;
    if (t >= a.T) return;
    float l[PER], slot_g = 0.0f;
    int64_t slot_i = -1;
    fetch_logits<BF16>(a.logits, t, a.T, a.E, l);
    if (lane < a.K) {
        slot_i = a.topk_idx[t * a.K + lane];
        slot_g = a.grad_weights[t * a.K + lane];
    }
    float top = -INFINITY;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        const int e = lane + j * kWave;
        l[j] = clean(l[j]);
        top = fmaxf(top, l[j]);
        slot_grad[wave][e] = l[j];  // for the slots to read, then their gradients
    }
    wave_fence();
    int id = -1;
    float g = 0.0f, x = -INFINITY;
    if (slot_i >= 0 && slot_i < a.E) {
        id = (int)slot_i;
        g = slot_g * a.scale;
        x = slot_grad[wave][id];
    }
    wave_fence();
#pragma unroll
    for (int j = 0; j < PER; ++j) slot_grad[wave][lane + j * kWave] = 0.0f;
    top = wave_max(top);

    // p: the score of each expert; ps: that of the slot's. Renormalised: the share
    // of the chosen total instead, from exponentials relative to the largest
    // chosen logit (softmax; sigmoid where all chosen scores are tiny).
    float p[PER], ps = 0.0f;
    float ref = top, inv = 1.0f;
    bool by_exp = !a.sigmoid;
    if (a.renormalize) {
        ref = wave_max(x);
        by_exp = by_exp || ref < -60.0f;
    }
    // scores that are zero in 64 bits, too, have no gradient (as in the forward direction)
    const bool none = ref == -INFINITY || (a.sigmoid ? ref < -kZeroScore : top - ref > kZeroScore);
    if (!none && id >= 0) ps = by_exp ? expf(x - ref) : 1.0f / (1.0f + expf(-x));
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        // (renormalised, experts above the largest chosen one get no gradient: kept finite)
        p[j] = none ? 0.0f : by_exp ? expf(fminf(l[j] - ref, 0.0f)) : 1.0f / (1.0f + expf(-l[j]));
        sum += p[j];
    }
    if (a.renormalize)
        sum = wave_sum(ps);
    else
        sum = a.sigmoid ? 1.0f : wave_sum(sum);
    inv = sum > 0.0f ? 1.0f / sum : 0.0f;
#pragma unroll
    for (int j = 0; j < PER; ++j) p[j] *= inv;
    ps *= inv;
    if (a.renormalize) {
        const float dot = wave_sum(g * ps);
        g = id >= 0 ? g - dot : 0.0f;
    }
    // one sum for each expert, in slot order, written by its first slot
    float slots = 0.0f;
    bool first = id >= 0;
    for (int k = 0; k < a.K; ++k) {
        const int oi = __builtin_amdgcn_readlane(id, k);
        const float og = __uint_as_float(__builtin_amdgcn_readlane((int)__float_as_uint(g), k));
        if (oi == id) {
            slots += og;
            if (k < lane) first = false;
        }
    }
    wave_fence();
    if (first) slot_grad[wave][id] = slots;
    wave_fence();
    const float dot = a.sigmoid || a.renormalize ? 0.0f : wave_sum(id >= 0 ? g * ps : 0.0f);
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        const int e = lane + j * kWave;
        if (e >= a.E) continue;
        float d = p[j] * (slot_grad[wave][e] - dot);
        if (a.sigmoid) d *= 1.0f / (1.0f + expf(l[j]));  // 1 - s
        if (BF16)
            static_cast<uint16_t*>(a.grad_logits)[t * a.E + e] = (uint16_t)pack_bf16x2(d, 0.0f);
        else
            static_cast<float*>(a.grad_logits)[t * a.E + e] = d;
    }
}

static dim3 route_grid(int64_t T) { return dim3((unsigned)((T + kRouteWaves - 1) / kRouteWaves)); }
// Tokens of one launch: its work-items, 64 for each token, stay below 2^32.
constexpr int64_t kRouteTokens = int64_t(1) << 25;

static const void* logits_from(const void* p, int64_t at, int bf16) { return static_cast<const char*>(p) + at * (bf16 ? 2 : 4); }

template <bool WIDE, bool BF16>
static void route_launch(const RouteArgs& a, hipStream_t stream) {
    const dim3 grid = route_grid(a.T), block(kRouteWaves * kWave);
    if (a.E <= 64)
        hipLaunchKernelGGL((route_kernel<WIDE, BF16, 1>), grid, block, 0, stream, a);
    else if (a.E <= 128)
        hipLaunchKernelGGL((route_kernel<WIDE, BF16, 2>), grid, block, 0, stream, a);
    else if (a.E <= 256)
        hipLaunchKernelGGL((route_kernel<WIDE, BF16, 4>), grid, block, 0, stream, a);
    else
        hipLaunchKernelGGL((route_kernel<WIDE, BF16, 8>), grid, block, 0, stream, a);
}

hipError_t launch_route(const RouteArgs& all, hipStream_t stream) {
    for (int64_t t = 0; t < all.T; t += kRouteTokens) {
        RouteArgs a = all;
        a.T = all.T - t < kRouteTokens ? all.T - t : kRouteTokens;
        a.logits = logits_from(all.logits, t * a.E, a.logits_bf16);
        a.topk_idx += t * a.K;
        a.topk_weights += t * a.K;
        if (a.bias || a.groups > 1)
            a.logits_bf16 ? route_launch<true, true>(a, stream) : route_launch<true, false>(a, stream);
        else
            a.logits_bf16 ? route_launch<false, true>(a, stream) : route_launch<false, false>(a, stream);
        const hipError_t err = hipGetLastError();
        if (err != hipSuccess) return err;
    }
    return hipSuccess;
}

template <bool BF16>
static void route_grad_launch(const RouteGradArgs& a, hipStream_t stream) {
    const dim3 grid = route_grid(a.T), block(kRouteWaves * kWave);
    if (a.E <= 64)
        hipLaunchKernelGGL((route_grad_kernel<BF16, 1>), grid, block, 0, stream, a);
    else if (a.E <= 128)
        hipLaunchKernelGGL((route_grad_kernel<BF16, 2>), grid, block, 0, stream, a);
    else if (a.E <= 256)
        hipLaunchKernelGGL((route_grad_kernel<BF16, 4>), grid, block, 0, stream, a);
    else
        hipLaunchKernelGGL((route_grad_kernel<BF16, 8>), grid, block, 0, stream, a);
}

hipError_t launch_route_grad(const RouteGradArgs& all, hipStream_t stream) {
    for (int64_t t = 0; t < all.T; t += kRouteTokens) {
        RouteGradArgs a = all;
        a.T = all.T - t < kRouteTokens ? all.T - t : kRouteTokens;
        a.logits = logits_from(all.logits, t * a.E, a.logits_bf16);
        a.grad_logits = const_cast<void*>(logits_from(all.grad_logits, t * a.E, a.logits_bf16));
        a.topk_idx += t * a.K;
        a.grad_weights += t * a.K;
        a.logits_bf16 ? route_grad_launch<true>(a, stream) : route_grad_launch<false>(a, stream);
        const hipError_t err = hipGetLastError();
        if (err != hipSuccess) return err;
    }
    return hipSuccess;
}

hipError_t preload_route() {
    hipFuncAttributes at;
    return hipFuncGetAttributes(&at, reinterpret_cast<const void*>(&route_grad_kernel<false, 8>));
}

}  // namespace cgd
