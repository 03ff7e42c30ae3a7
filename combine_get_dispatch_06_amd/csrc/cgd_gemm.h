// Tiled matrix products on the gfx950 matrix cores, shared by the dense and
// the grouped entry points and by both directions.
//
//   out[m, n] = sum_k Q[m, k] * P[n, k]
//
// Q is the row operand (tokens; output channels of a weight gradient), P the
// column operand (weights; input channels of a weight gradient). Each is
// either "k-contiguous" (rows of k) or "transposed" (rows of m or n, one per
// k): forward products read both k-contiguous, the input gradient reads its
// weights transposed, the weight gradient reads both transposed. Nothing is
// laid out again in memory: transposed tiles are turned by the LDS
// transposing read while they are loaded into registers.
//
// One block makes one BM x BN tile of the output. Tiles of 128 bytes of k
// (64 bf16, 128 FP8) go from global memory straight into LDS, 16 bytes per
// lane, kStages deep; each wave multiplies its (BM/WM) x (BN/WN) part with
// 16x16 matrix instructions, sums in fp32 registers. The first matrix operand
// is P, so a lane ends up with runs of consecutive output columns of one row.
//
// Bounds: every global read goes through a buffer descriptor that ends where
// the rows of the tile end (reads past it return zero), and lanes past the end
// of the reduction are pointed past the descriptor; stores are predicated.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "cgd_device.h"
#include "cgd_experts_launch.h"

namespace cgd {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4_t __attribute__((ext_vector_type(4)));
typedef short short4_t __attribute__((ext_vector_type(4)));
typedef short short8_t __attribute__((ext_vector_type(8)));
typedef float float4_t __attribute__((ext_vector_type(4)));
typedef int int4_t __attribute__((ext_vector_type(4)));
typedef int int8_t_ __attribute__((ext_vector_type(8)));

#define CGD_LDS(T) __attribute__((address_space(3))) T

__device__ __forceinline__ uint32_t lds_address(const void* p) {
    return (uint32_t)(uintptr_t)(const CGD_LDS(char)*)p;
}

// A raw buffer descriptor over `bytes` bytes at `base` (held in scalar
// registers): loads at or past `bytes` return zero.
struct Buffer {
    uint64_t base;
    uint32_t bytes;
    __device__ __forceinline__ int4_t words() const {
        int4_t r;
        r.x = __builtin_amdgcn_readfirstlane((int)(uint32_t)base);
        r.y = __builtin_amdgcn_readfirstlane((int)(uint32_t)(base >> 32) & 0xFFFF);
        r.z = __builtin_amdgcn_readfirstlane((int)bytes);
        r.w = 0x00020000;
        return r;
    }
};
constexpr uint32_t kPastEnd = 0x80000000u;  // an offset past every descriptor (those end below 2^31)

// 16 bytes per lane from buffer offset `off` to LDS address lds + 16 * lane.
// The load has no register result; the waits for it are written out where a
// stage is needed (wait_stage).
__device__ __forceinline__ void load_to_lds16(const int4_t& buf, uint32_t off, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(lds), "v"(off), "s"(buf)
                 : "memory", "m0");
}
// 4 bytes (fp32) or 1 byte (widened to 4) per lane to lds + 4 * lane.
__device__ __forceinline__ void load_to_lds4(const int4_t& buf, uint32_t off, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, 0 offen lds" ::"s"(lds), "v"(off), "s"(buf)
                 : "memory", "m0");
}
__device__ __forceinline__ void load_to_lds1(const int4_t& buf, uint32_t off, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_ubyte %1, %2, 0 offen lds" ::"s"(lds), "v"(off), "s"(buf)
                 : "memory", "m0");
}
// At most N of this wave's loads still on their way, none of its LDS reads.
template <int N>
__device__ __forceinline__ void wait_loads() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(N) : "memory");
}
__device__ __forceinline__ void block_barrier() { asm volatile("s_barrier" ::: "memory"); }

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ int64_t uniform64(int64_t v) {
    const uint32_t lo = __builtin_amdgcn_readfirstlane((int)(uint32_t)v);
    const uint32_t hi = __builtin_amdgcn_readfirstlane((int)(uint32_t)((uint64_t)v >> 32));
    return (int64_t)(((uint64_t)hi << 32) | lo);
}

// First row and number of rows of group e, whatever the device data say:
// always inside [0, total].
__device__ __forceinline__ void group_rows(const Groups& g, int e, int64_t* begin, int64_t* rows) {
    int64_t b, n;
    if (g.offset) {
        b = g.offset[e];
        n = g.offset[e + 1];
        b = b < 0 ? 0 : (b > g.total ? g.total : b);
        n = n > g.total ? g.total : n;
        n -= b;
    } else {
        b = (int64_t)e * g.capacity;
        n = g.capacity;
    }
    if (g.count) {
        const int64_t c = g.count[e];
        n = c < n ? c : n;
    }
    *begin = b;
    *rows = n < 0 ? 0 : n;
}

// Which group and which piece of BM rows the flattened piece `want` is, and
// how many pieces there are in all. Every wave works it out for itself, 64
// groups at a time (one load round for each 64 groups, a scan over lanes).
struct Piece {
    int group;
    int64_t row0;  // first row of the piece
    int64_t rows;  // rows of the group from row0 on
    int total;     // pieces in all groups
};
template <bool FIND>
__device__ __forceinline__ Piece find_piece(const Groups& g, int bm, int want) {
    Piece r;
    r.group = -1;
    r.row0 = r.rows = 0;
    r.total = 0;
    if (!g.offset && !g.count && g.groups == 1) {  // one dense product: nothing to read
        r.total = (int)((g.total + bm - 1) / bm);
        r.group = want < r.total ? 0 : -1;
        r.row0 = (int64_t)want * bm;
        r.rows = g.total - r.row0;
        return r;
    }
    const int lane = lane_id();
    int before = 0;
    for (int e0 = 0; e0 < g.groups; e0 += kWave) {
        const int e = e0 + lane;
        int64_t b = 0, n = 0;
        if (e < g.groups) group_rows(g, e, &b, &n);
        const int mine = (int)((n + bm - 1) / bm);
        int upto = mine;  // inclusive scan over the lanes
#pragma unroll
        for (int d = 1; d < kWave; d <<= 1) {
            const int o = __shfl_up(upto, d, kWave);
            if (lane >= d) upto += o;
        }
        if (FIND && r.group < 0) {
            const int first = before + upto - mine;
            const uint64_t hit = ballot(mine > 0 && want >= first && want < first + mine);
            if (hit) {
                const int l = __ffsll((unsigned long long)hit) - 1;
                const int f = __builtin_amdgcn_readlane(first, l);
                const int64_t off = (int64_t)(want - f) * bm;
                const uint32_t blo = __builtin_amdgcn_readlane((int)(uint32_t)b, l);
                const uint32_t bhi = __builtin_amdgcn_readlane((int)(uint32_t)((uint64_t)b >> 32), l);
                const uint32_t nlo = __builtin_amdgcn_readlane((int)(uint32_t)n, l);
                const uint32_t nhi = __builtin_amdgcn_readlane((int)(uint32_t)((uint64_t)n >> 32), l);
                r.group = e0 + l;
                r.row0 = (int64_t)(((uint64_t)bhi << 32) | blo) + off;
                r.rows = (int64_t)(((uint64_t)nhi << 32) | nlo) - off;
            }
        }
        before += __builtin_amdgcn_readlane(upto, kWave - 1);
    }
    r.total = before;
    return r;
}

// ---- activations, in fp32 -------------------------------------------------
__device__ __forceinline__ float sigmoid_f(float v) { return 1.0f / (1.0f + __expf(-v)); }
__device__ __forceinline__ float silu_f(float v) { return v * sigmoid_f(v); }
__device__ __forceinline__ float gelu_f(float v) { return 0.5f * v * (1.0f + erff(v * 0.70710678118654752f)); }
__device__ __forceinline__ float act_f(float v, int act) {
    if (act == kActRelu) return v < 0.0f ? 0.0f : v;  // NaN passes through
    if (act == kActSilu) return silu_f(v);
    if (act == kActGelu) return gelu_f(v);
    return v;
}

__device__ __forceinline__ float bf16_at(const uint16_t* p) { return __uint_as_float((uint32_t)*p << 16); }

// Stores N (4 or 8) consecutive values of one output row from column c on, as
// bf16 or fp32, in 8- or 16-byte pieces where the row allows it (`wide`).
template <int N>
__device__ __forceinline__ void store_run(void* out, int64_t at, const float* v, int have, bool f32, bool wide) {
    if (have <= 0) return;
    if (f32) {
        float* o = static_cast<float*>(out) + at;
        if (wide && have >= N) {
#pragma unroll
            for (int i = 0; i < N; i += 4) *reinterpret_cast<float4_t*>(o + i) = float4_t{v[i], v[i + 1], v[i + 2], v[i + 3]};
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (i < have) o[i] = v[i];
        }
        return;
    }
    uint16_t* o = static_cast<uint16_t*>(out) + at;
    uint32_t w[N / 2];
#pragma unroll
    for (int i = 0; i < N; i += 2) w[i / 2] = pack_bf16x2(v[i], v[i + 1]);
    if (wide && have >= N) {
        if (N == 8)
            *reinterpret_cast<uint4*>(o) = make_uint4(w[0], w[1], w[N / 2 - 2], w[N / 2 - 1]);
        else
            *reinterpret_cast<uint2*>(o) = make_uint2(w[0], w[1]);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (i < have) o[i] = (uint16_t)(w[i / 2] >> (16 * (i & 1)));
    }
}

// Loads up to N consecutive bf16 values as fp32 (zero past `have`).
template <int N>
__device__ __forceinline__ void load_run(const uint16_t* p, int have, bool wide, float* v) {
    if (wide && have >= N) {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            const uint2 q = *reinterpret_cast<const uint2*>(p + i);
            v[i] = bf16_lo(q.x);
            v[i + 1] = bf16_hi(q.x);
            v[i + 2] = bf16_lo(q.y);
            v[i + 3] = bf16_hi(q.y);
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = i < have ? bf16_at(p + i) : 0.0f;
    }
}

// The 128-byte LDS rows of a k-contiguous tile hold their 16-byte pieces in an
// order that depends on the row: piece c of row r is at c ^ key(r), so that the
// 16 rows a matrix instruction takes are spread over the banks. The rows of one
// instruction are 16 consecutive rows of Q, and for P the rows
// (i / 4) * RUN + i % 4 (RUN consecutive columns per lane): key depends on i only.
template <int RUN>
__device__ __forceinline__ int row_key(int row) {
    return (row & 3) | (((row / RUN) & 1) << 2);
}

// Kernel arguments: see GemmArgs in cgd_experts_launch.h.
template <int BM, int BN, int WM, int WN, int ST, bool QT, bool PT, bool FP8>
__global__ __launch_bounds__(WM* WN* kWave, 2) void gemm_kernel(const GemmArgs a) {
    constexpr int NW = WM * WN;              // waves
    constexpr int TM = BM / WM, TN = BN / WN;  // a wave's part
    constexpr int MT = TM / 16, NT = TN / 16, NH = NT / 2;
    constexpr int RUN = 4 * NH;              // consecutive columns per lane
    constexpr int BK = FP8 ? 128 : 64;       // 128 bytes of k
    constexpr int QB = BM * 128, PB = BN * 128;
    // scales of a stage: one per row, the weights', and a place that is never read
    constexpr int SROWS = BM < 64 ? 64 : BM;
    constexpr int SB = FP8 ? SROWS * 4 + 512 : 0;
    constexpr int STAGE = QB + PB + SB;
    constexpr int QL = BM / 8 / NW, PL = BN / 8 / NW;  // 1-KB loads per wave
    constexpr int SL = FP8 ? 1 : 0;
    constexpr int LOADS = QL + PL + SL;
    static_assert(QL >= 1 && PL >= 2 && NT % 2 == 0 && MT >= 1, "tile too small for its waves");
    static_assert(!FP8 || (!QT && !PT), "FP8 tiles are k-contiguous");
    static_assert(!FP8 || SROWS / 64 + 1 <= NW, "one wave loads 64 row scales, one the weights'");
    __shared__ __attribute__((aligned(1024))) char smem[ST * STAGE];

    const int lane = lane_id();
    const int wave = uniform(threadIdx.x / kWave);
    const int wm = wave / WN, wn = wave % WN;
    const int li = lane & 15, lg = lane >> 4;

    // ---- which tile -------------------------------------------------------
    // Blocks go to the 8 XCDs in turn; each XCD takes one run of consecutive
    // tiles, and within a run 4 row tiles share a column of tiles, so that the
    // tiles in flight on an XCD share operands in its L2.
    const int half_n = a.glu ? BN / 2 : BN;  // output columns of a tile
    const int ntn = (int)((a.n + half_n - 1) / half_n);
    int group, split = 0;
    int64_t m0, rows, k0 = 0, klen;
    int tn;
    int64_t qrow0, prow0 = 0;
    if (!QT) {
        Piece pc = find_piece<false>(a.g, BM, 0);
        const int nsplit = a.splits;
        const int tiles = pc.total * ntn * nsplit;
        const int per = (tiles + 7) / 8;
        const int t0 = (int)(blockIdx.x & 7) * per + (int)(blockIdx.x >> 3);
        if ((int)(blockIdx.x >> 3) >= per || t0 >= tiles) return;
        int t = t0;
        split = t / (pc.total * ntn);
        t -= split * (pc.total * ntn);
        constexpr int GM = 4;
        const int sr = t / (GM * ntn);
        const int gm = pc.total - sr * GM < GM ? pc.total - sr * GM : GM;
        const int in = t - sr * GM * ntn;
        tn = in / gm;
        pc = find_piece<true>(a.g, BM, sr * GM + in % gm);
        if (pc.group < 0) return;
        group = uniform(pc.group);
        qrow0 = uniform64(pc.row0);
        rows = uniform64(pc.rows);
        m0 = 0;
        k0 = (int64_t)split * a.ksplit;
        klen = a.k - k0 < a.ksplit ? a.k - k0 : a.ksplit;
    } else {
        // weight gradient: a fixed grid of tiles, the reduction over a group's rows
        const int ntm = (int)((a.m + BM - 1) / BM);
        const int per_group = ntm * ntn;
        const int tiles = per_group * a.g.groups;
        const int per = (tiles + 7) / 8;
        const int t = (int)(blockIdx.x & 7) * per + (int)(blockIdx.x >> 3);
        if ((int)(blockIdx.x >> 3) >= per || t >= tiles) return;
        group = t / per_group;
        const int in0 = t - group * per_group;
        constexpr int GM = 4;
        const int sr = in0 / (GM * ntn);
        const int gm = ntm - sr * GM < GM ? ntm - sr * GM : GM;
        const int in = in0 - sr * GM * ntn;
        tn = in / gm;
        m0 = (int64_t)(sr * GM + in % gm) * BM;
        int64_t b, n;
        if (!a.g.offset && !a.g.count && a.g.groups == 1) {
            b = 0;
            n = a.g.total;
        } else {
            group_rows(a.g, group, &b, &n);
        }
        qrow0 = prow0 = uniform64(b);
        klen = uniform64(n);
        rows = a.m - m0;
    }
    const int64_t n0 = (int64_t)tn * half_n;
    const int nk = uniform((int)((klen + BK - 1) / BK));

    // ---- where the operands are --------------------------------------------
    // Q: k-contiguous: rows qrow0 .. ; transposed: columns m0 .. of rows qrow0 ..
    Buffer qb, pb0, pb1;
    uint32_t qv[QL], pv[PL];
    const int64_t ES = FP8 ? 1 : 2;
    int64_t q_left = 0, p_left = 0;  // transposed operands: rows of k left
    if (!QT) {
        qb.base = (uint64_t)a.q + (uint64_t)(qrow0 * a.ldq + k0 * ES);
        const int64_t r = rows < BM ? rows : BM;
        qb.bytes = (uint32_t)(r * a.ldq - k0 * ES);
#pragma unroll
        for (int j = 0; j < QL; ++j) {
            const int row = (j * NW + wave) * 8 + lane / 8;
            qv[j] = (uint32_t)(row * (int)a.ldq + (((lane & 7) ^ row_key<4>(row)) << 4));
        }
    } else {
        constexpr int RPI = 512 / BM;  // k rows per 1-KB load
        qb.base = (uint64_t)a.q + (uint64_t)(qrow0 * a.ldq + m0 * 2);
        q_left = klen;
        qb.bytes = (uint32_t)((q_left < 64 ? q_left : 64) * a.ldq - m0 * 2);
        if (q_left <= 0) qb.bytes = 0;
#pragma unroll
        for (int j = 0; j < QL; ++j) {
            const int kr = (j * NW + wave) * RPI + lane / (64 / RPI);
            const int s = lane & (64 / RPI - 1);
            qv[j] = (uint32_t)(kr * (int)a.ldq + ((s ^ ((kr & 3) << 1)) << 4));
        }
    }
    if (!PT) {
        const uint64_t pbase = (uint64_t)a.p + (uint64_t)((int64_t)group * a.p_group);
        const int64_t second = a.glu ? a.n + n0 : n0 + BN / 2;  // first weight row of the tile's upper half
        const int64_t r0 = a.n - n0 < BN / 2 ? a.n - n0 : BN / 2;
        int64_t r1 = a.glu ? r0 : a.n - second;
        r1 = r1 < 0 ? 0 : (r1 > BN / 2 ? BN / 2 : r1);
        pb0.base = pbase + (uint64_t)(n0 * a.ldp + k0 * ES);
        pb0.bytes = (uint32_t)(r0 * a.ldp - k0 * ES);
        pb1.base = pbase + (uint64_t)(second * a.ldp + k0 * ES);
        pb1.bytes = r1 > 0 ? (uint32_t)(r1 * a.ldp - k0 * ES) : 0u;
#pragma unroll
        for (int j = 0; j < PL; ++j) {
            const int row = ((j % (PL / 2)) * NW + wave) * 8 + lane / 8;
            pv[j] = (uint32_t)(row * (int)a.ldp + (((lane & 7) ^ row_key<RUN>(row)) << 4));
        }
    } else {
        constexpr int RPI = 512 / BN;
        pb0.base = (uint64_t)a.p + (uint64_t)((int64_t)group * a.p_group + (prow0 + k0) * a.ldp + n0 * 2);
        p_left = klen;
        pb0.bytes = (uint32_t)((p_left < 64 ? p_left : 64) * a.ldp - n0 * 2);
        if (p_left <= 0) pb0.bytes = 0;
        pb1 = pb0;
#pragma unroll
        for (int j = 0; j < PL; ++j) {
            const int kr = (j * NW + wave) * RPI + lane / (64 / RPI);
            const int s = lane & (64 / RPI - 1);
            pv[j] = (uint32_t)(kr * (int)a.ldp + ((s ^ ((kr & 3) << 2)) << 4));
        }
    }
    // FP8 scales: wave w < BM/64 brings those of rows 64 w .., the last wave
    // those of the two weight blocks the tile's halves lie in (lanes 0 and 1:
    // the halves are at most 128 wide and start at multiples of their width,
    // and SwiGLU's up rows start at a multiple of 128).
    Buffer sb;
    uint32_t sv = kPastEnd;
    int64_t s_step = 0;
    bool s_byte = false;
    if (FP8) {
        const int kb0 = (int)(k0 / 128);
        if (wave == NW - 1) {
            sb.base = (uint64_t)a.ps + (uint64_t)((int64_t)group * a.ps_group * 4);
            sb.bytes = (uint32_t)(a.ps_group * 4);
            const int64_t second = a.glu ? a.n + n0 : n0 + BN / 2;
            const int64_t row = lane == 0 ? n0 : second;
            const int64_t blk = row / 128;
            if (lane < 2 && row < a.n * (a.glu ? 2 : 1)) sv = (uint32_t)((blk * a.ps_row + kb0) * 4);
            s_step = 4;
        } else {
            const int row = wave * 64 + lane;
            const int sbytes = a.qs_byte ? 1 : 4;
            sb.base = (uint64_t)a.qs + (uint64_t)((qrow0 * a.qs_row + kb0 * a.qs_blk) * sbytes);
            sb.bytes = 0x7FFFFFF0u;
            if (row < BM && row < rows) sv = (uint32_t)(row * a.qs_row * sbytes);
            s_step = a.qs_blk * sbytes;
            s_byte = a.qs_byte;
        }
    }

    const uint32_t lds0 = uniform((int)lds_address(smem));
    const int64_t q_step = QT ? 64 * a.ldq : 128, p_step = PT ? 64 * a.ldp : 128;
    int64_t k_left = klen;  // of the next stage to load

    auto load_stage = [&](int buf) {
        const uint32_t l = lds0 + (uint32_t)(buf * STAGE);
        const bool tail = k_left < BK;
        const int left = (int)(tail ? k_left : BK);
        const int4_t qw = qb.words(), pw0 = pb0.words(), pw1 = pb1.words();
#pragma unroll
        for (int j = 0; j < QL; ++j) {
            uint32_t v = qv[j];
            if (!QT && tail) {
                const int row = (j * NW + wave) * 8 + lane / 8;
                const int c = (lane & 7) ^ row_key<4>(row);
                v = c * (FP8 ? 16 : 8) < left ? v : kPastEnd;
            }
            load_to_lds16(qw, v, l + (j * NW + wave) * 1024);
        }
#pragma unroll
        for (int j = 0; j < PL; ++j) {
            uint32_t v = pv[j];
            if (!PT && tail) {
                const int row = ((j % (PL / 2)) * NW + wave) * 8 + lane / 8;
                const int c = (lane & 7) ^ row_key<RUN>(row);
                v = c * (FP8 ? 16 : 8) < left ? v : kPastEnd;
            }
            load_to_lds16(!PT && j >= PL / 2 ? pw1 : pw0, v, l + QB + (j * NW + wave) * 1024);
        }
        if (FP8) {
            const int4_t sw = sb.words();
            // waves with neither rows nor the weights' scales load zeros into the
            // unread place: every wave has the same count of loads to wait for
            const uint32_t dst = l + QB + PB + (wave == NW - 1 ? SROWS * 4 : wave * 64 < SROWS ? wave * 256 : SROWS * 4 + 256);
            if (s_byte)
                load_to_lds1(sw, sv, dst);
            else
                load_to_lds4(sw, sv, dst);
            sb.base += s_step;
            if (wave == NW - 1) sb.bytes = sb.bytes > 4 ? sb.bytes - 4 : 0;
        }
        qb.base += q_step;
        pb0.base += p_step;
        pb1.base += p_step;
        if (QT) {
            q_left -= 64;
            const int64_t r = q_left < 0 ? 0 : (q_left < 64 ? q_left : 64);
            qb.bytes = r > 0 ? (uint32_t)(r * a.ldq - m0 * 2) : 0u;
        } else {
            qb.bytes = qb.bytes > 128 ? qb.bytes - 128 : 0;
        }
        if (PT) {
            p_left -= 64;
            const int64_t r = p_left < 0 ? 0 : (p_left < 64 ? p_left : 64);
            pb0.bytes = r > 0 ? (uint32_t)(r * a.ldp - n0 * 2) : 0u;
        } else {
            pb0.bytes = pb0.bytes > 128 ? pb0.bytes - 128 : 0;
            pb1.bytes = pb1.bytes > 128 ? pb1.bytes - 128 : 0;
        }
        k_left -= BK;
    };

    float4_t acc[MT][NT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j] = float4_t{0.f, 0.f, 0.f, 0.f};

    // ---- LDS addresses of a lane's fragments -------------------------------
    const CGD_LDS(char)* sm = (const CGD_LDS(char)*)smem;
    // k-contiguous: piece (ks * 4 + lg) of the row, for ks = 0, 1
    int qa[4], pa[2];
    if (!QT) {
        const int row = wm * TM + li;
        qa[0] = row * 128 + ((lg ^ row_key<4>(row)) << 4);
        qa[1] = row * 128 + (((4 + lg) ^ row_key<4>(row)) << 4);
        qa[2] = qa[3] = 0;
    } else {
        // four columns of k row lg * 8 + li / 4; column piece of 16-row tile mt
        const int kr = lg * 8 + (li >> 2);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int col = wm * TM + u * 16 + (li & 3) * 4;
            qa[u] = kr * (BM * 2) + (((col >> 3) ^ ((kr & 3) << 1)) << 4) + (col & 7) * 2;
        }
    }
    if (!PT) {
        const int row = wn * (TN / 2) + (li >> 2) * RUN + (li & 3);
        pa[0] = QB + row * 128 + ((lg ^ row_key<RUN>(row)) << 4);
        pa[1] = QB + row * 128 + (((4 + lg) ^ row_key<RUN>(row)) << 4);
    } else {
        pa[0] = pa[1] = 0;
    }
    auto q_frag = [&](int base, int ks, int mt) -> bf16x8_t {
        if (!QT) return *(const CGD_LDS(bf16x8_t)*)(sm + base + qa[ks] + mt * 2048);
        const int at = base + qa[mt & 3] + (mt >> 2) * 128 + ks * 32 * (BM * 2);
        const short4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((CGD_LDS(short4_t)*)(sm + at));
        const short4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((CGD_LDS(short4_t)*)(sm + at + 4 * (BM * 2)));
        return __builtin_bit_cast(bf16x8_t, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    };
    auto p_frag = [&](int base, int ks, int nt) -> bf16x8_t {
        const int h = nt / NH, t = nt % NH;
        if (!PT) return *(const CGD_LDS(bf16x8_t)*)(sm + base + pa[ks] + h * (BN / 2) * 128 + t * 512);
        const int kr = lg * 8 + (li >> 2);
        const int col = h * (BN / 2) + wn * (TN / 2) + (li & 3) * RUN + t * 4;
        const int at = base + QB + kr * (BN * 2) + (((col >> 3) ^ ((kr & 3) << 2)) << 4) + (col & 7) * 2 + ks * 32 * (BN * 2);
        const short4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((CGD_LDS(short4_t)*)(sm + at));
        const short4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((CGD_LDS(short4_t)*)(sm + at + 4 * (BN * 2)));
        return __builtin_bit_cast(bf16x8_t, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    };

    // ---- main loop ----------------------------------------------------------
#pragma unroll
    for (int s = 0; s < ST - 1; ++s)
        if (s < nk) load_stage(s);
    int buf = 0, next = ST - 1;
    for (int kt = 0; kt < nk; ++kt) {
        // stage kt has landed once at most the loads of the stages after it are
        // still on their way; past the barrier it has for every wave, and the
        // stage read in the last step may be overwritten
        if (ST > 2 && kt + ST - 2 < nk)
            wait_loads<(ST - 2) * LOADS>();
        else
            wait_loads<0>();
        block_barrier();
        if (kt + ST - 1 < nk) load_stage(next);
        const int base = buf * STAGE;
        if constexpr (!FP8) {
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
                bf16x8_t qf[MT], pf[NT];
#pragma unroll
                for (int j = 0; j < NT; ++j) pf[j] = p_frag(base, ks, j);
#pragma unroll
                for (int i = 0; i < MT; ++i) qf[i] = q_frag(base, ks, i);
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                    for (int j = 0; j < NT; ++j)
                        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(pf[j], qf[i], acc[i][j], 0, 0, 0);
            }
        } else {
            const CGD_LDS(float)* sc = (const CGD_LDS(float)*)(sm + base + QB + PB);
            const float w0 = sc[SROWS], w1 = sc[SROWS + 1];
            int8_t_ pf[NT];
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const int4_t lo = __builtin_bit_cast(int4_t, p_frag(base, 0, j)), hi = __builtin_bit_cast(int4_t, p_frag(base, 1, j));
                pf[j] = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
            }
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                const int4_t lo = __builtin_bit_cast(int4_t, q_frag(base, 0, i)), hi = __builtin_bit_cast(int4_t, q_frag(base, 1, i));
                const int8_t_ qf = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
                float s = sc[wm * TM + i * 16 + li];
                if (a.qs_byte) {
                    const uint32_t e = __float_as_uint(s);
                    s = __uint_as_float(e ? e << 23 : 0x00400000u);
                }
                const float s0 = s * w0, s1 = s * w1;
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    const float4_t z = {0.f, 0.f, 0.f, 0.f};
                    const float4_t d = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(pf[j], qf, z, 0, 0, 0, 127, 0, 127);
                    const float f = j < NH ? s0 : s1;
#pragma unroll
                    for (int r = 0; r < 4; ++r) acc[i][j][r] = fmaf(d[r], f, acc[i][j][r]);
                }
            }
        }
        buf = buf + 1 == ST ? 0 : buf + 1;
        next = next + 1 == ST ? 0 : next + 1;
    }

    // ---- epilogue -----------------------------------------------------------
    // A lane holds, for each 16-row tile, one row and RUN consecutive columns
    // in the lower half of the tile and RUN in the upper half.
    const int64_t lim = rows < BM ? rows : BM;
    const int64_t c0 = n0 + wn * (TN / 2) + lg * RUN;                                   // lower half's columns
    const int64_t c1 = (a.glu ? a.n : (int64_t)BN / 2) + c0;                            // upper half's (weight rows)
    const int have0 = (int)(a.n - c0 < RUN ? a.n - c0 : RUN);
    const int64_t end1 = a.glu ? 2 * a.n : a.n;
    const int have1 = a.glu ? have0 : (int)(end1 - c1 < RUN ? end1 - c1 : RUN);
    float bias0[RUN], bias1[RUN];
#pragma unroll
    for (int r = 0; r < RUN; ++r) bias0[r] = bias1[r] = 0.0f;
    if (a.bias && a.splits == 1) {
        const uint16_t* b = static_cast<const uint16_t*>(a.bias) + (int64_t)group * end1;
        load_run<RUN>(b + c0, have0, false, bias0);
        load_run<RUN>(b + c1, have1, false, bias1);
    }
    const int64_t orow0 = QT ? (int64_t)group * a.m + m0 : qrow0;
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        const int64_t r = wm * TM + i * 16 + li;
        if (r >= lim) continue;
        float v0[RUN], v1[RUN];
#pragma unroll
        for (int t = 0; t < NH; ++t)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                v0[t * 4 + q] = acc[i][t][q];
                v1[t * 4 + q] = acc[i][NH + t][q];
            }
        const int64_t row = orow0 + r;
        if (a.splits > 1) {  // partial sums, joined by join_kernel
            const int64_t at = ((int64_t)split * a.g.total + row) * end1;
            store_run<RUN>(a.partial, at + c0, v0, have0, true, (end1 & 3) == 0);
            store_run<RUN>(a.partial, at + c1, v1, have1, true, (end1 & 3) == 0 && (!a.glu || (a.n & 3) == 0));
            continue;
        }
#pragma unroll
        for (int q = 0; q < RUN; ++q) {
            v0[q] += bias0[q];
            v1[q] += bias1[q];
        }
        if (a.preact) {
            store_run<RUN>(a.preact, row * end1 + c0, v0, have0, false, (end1 & 7) == 0);
            store_run<RUN>(a.preact, row * end1 + c1, v1, have1, false, (end1 & 7) == 0 && (!a.glu || (a.n & 7) == 0));
        }
        if (a.glu) {
#pragma unroll
            for (int q = 0; q < RUN; ++q) v0[q] = silu_f(v0[q]) * v1[q];
        } else if (a.act) {
#pragma unroll
            for (int q = 0; q < RUN; ++q) {
                v0[q] = act_f(v0[q], a.act);
                v1[q] = act_f(v1[q], a.act);
            }
        }
        if (a.residual) {
            const uint16_t* res = static_cast<const uint16_t*>(a.residual) + row * a.n;
            float z[RUN];
            load_run<RUN>(res + c0, have0, (a.n & 7) == 0, z);
#pragma unroll
            for (int q = 0; q < RUN; ++q) v0[q] += z[q];
            if (!a.glu) {
                load_run<RUN>(res + c1, have1, (a.n & 7) == 0, z);
#pragma unroll
                for (int q = 0; q < RUN; ++q) v1[q] += z[q];
            }
        }
        const bool wide = a.out_f32 ? (a.n & 3) == 0 : (a.n & 7) == 0;
        store_run<RUN>(a.out, row * a.n + c0, v0, have0, a.out_f32, wide);
        if (!a.glu) store_run<RUN>(a.out, row * a.n + c1, v1, have1, a.out_f32, wide);
    }
}

}  // namespace cgd
