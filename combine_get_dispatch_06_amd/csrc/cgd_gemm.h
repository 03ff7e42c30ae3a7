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
// A block makes BM x BN tiles of the output. Pieces of 128 bytes of k (64 bf16,
// 128 FP8; 64 bytes in the smaller gradient tiles) go from global memory straight
// into LDS, 16 bytes per lane, some stages ahead; each wave multiplies its
// (BM/WM) x (BN/WN) part with 16x16 matrix instructions, sums in fp32 registers.
// The first matrix operand is P, so a lane ends up with runs of consecutive
// output columns of one row.
//
// Three main loops:
//   256 x 256 on four waves (ST = 0): a CU to itself, 256 sums per lane in the
//     accumulation registers, three slots of Q and two of P in LDS. Operands are
//     read from LDS half a stage ahead. 32768 x 4096 x 7168 in 1.33-1.40 ms (1.37-1.45
//     PFLOP/s); loads half as deep measured 6 % more, 32x32 matrix instructions
//     more, too (twice the traffic of sums for a product). The chip's power bounds it:
//     the clock falls to 1.75 GHz with the matrix units 73 % busy and waves waiting a
//     tenth of the time. Reductions of 8 stages a tile (weight gradients of 32 groups of
//     512 rows) keep them a third busy: a tile's start and epilogue are not covered.
//   192 x 256 on eight waves (FP8): a CU to itself, two slots of P and three of Q.
//     Every 128 of k the products are scaled and added by the vector unit, 96
//     times four values a lane for 24 matrix instructions. Matrix units 60 % busy, a
//     wave waits a third of the time: 6144 x 8192 x 8192 in 0.37 ms (2.2 PFLOP/s).
//     (The general epilogue spills a few registers, outside the loop.)
//   smaller tiles: two or more blocks to a CU, ST stages; those of gradients
//     (RB = 64) read LDS a stage ahead of the matrix instructions: 32.4 us against
//     35.3 with 128-byte stages (4096 x 1024 x 512, both gradients). Few rows are
//     bound by the weights' latency and rate: 16 experts of 64 rows, 7168 ->
//     2 x 2048 in 180 us (5.2 TB/s), by the groups' sizes up to 250.
//
// Bounds: every global read goes through a buffer descriptor, and each lane's
// offset is inside its operand or kPastEnd, behind every descriptor's end, where
// reads return zero and touch no memory: lanes whose row or piece of k does not
// exist. Stores are predicated.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "cgd_device.h"
#include "cgd_experts_launch.h"

namespace cgd {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef short short4_t __attribute__((ext_vector_type(4)));
typedef float float4_t __attribute__((ext_vector_type(4)));
typedef int int4_t __attribute__((ext_vector_type(4)));
typedef int int8_t_ __attribute__((ext_vector_type(8)));

#define CGD_LDS(T) __attribute__((address_space(3))) T

__device__ __forceinline__ uint32_t lds_address(const void* p) {
    return (uint32_t)(uintptr_t)(const CGD_LDS(char)*)p;
}

// A raw buffer descriptor from `base` on. Reads at kPastEnd return zero without
// touching memory; every lane offset is either inside the operand or kPastEnd.
__device__ __forceinline__ int4_t buffer_from(uint64_t base) {
    int4_t r;
    r.x = __builtin_amdgcn_readfirstlane((int)(uint32_t)base);
    r.y = __builtin_amdgcn_readfirstlane((int)(uint32_t)(base >> 32));  // addresses end below 2^48
    r.z = 0x7FFFFFF0;
    r.w = 0x00020000;
    return r;
}
__device__ __forceinline__ void advance(int4_t& buf, int64_t bytes) {
    const uint64_t b = (((uint64_t)(uint32_t)buf.y << 32) | (uint32_t)buf.x) + (uint64_t)bytes;
    buf.x = (int)(uint32_t)b;
    buf.y = (int)(uint32_t)(b >> 32);
}
constexpr uint32_t kPastEnd = 0x80000000u;  // past every descriptor's end

// 16 bytes per lane from buffer offset `off` to LDS address lds + AT + 16 * lane.
// The load has no register result; the waits for it are written out where a
// stage is needed (wait_loads).
template <int AT>
__device__ __forceinline__ void load_to_lds16(const int4_t& buf, uint32_t off, uint32_t lds) {
    asm volatile("s_add_u32 m0, %0, %3\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(lds), "v"(off),
                 "s"(buf), "n"(AT)
                 : "memory", "m0", "scc");
}
// The same in two parts, with at least one instruction that is not theirs in
// between (the address register needs one wait state): nothing else in these
// kernels uses that register.
template <int AT>
__device__ __forceinline__ void aim_load(uint32_t lds) {
    asm volatile("s_add_u32 m0, %0, %1" ::"s"(lds), "n"(AT) : "memory", "m0", "scc");
}
__device__ __forceinline__ void aimed_load(const int4_t& buf, uint32_t off) {
    asm volatile("buffer_load_dwordx4 %0, %1, 0 offen lds" ::"v"(off), "s"(buf) : "memory");
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

// LDS writes of the block's waves before the reads that follow, and the other way round
__device__ __forceinline__ void block_sync() {
    wait_loads<0>();
    block_barrier();
}

// The same for LDS accesses alone: loads from memory stay on their way.
__device__ __forceinline__ void sync_lds() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// The same value, worked out anew where it is used: what follows from it is not
// kept in registers over the main loop for the next tile.
__device__ __forceinline__ int afresh(int v) {
    asm volatile("" : "+v"(v));
    return v;
}

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

template <int V>
struct Const {
    static constexpr int value = V;
};

// 8 values of k for one row of a transposed tile, from k rows at `p` and `next` bytes on
__device__ __forceinline__ bf16x8_t turned(const CGD_LDS(char)* p, int next) {
    const short4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((CGD_LDS(short4_t)*)p);
    const short4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((CGD_LDS(short4_t)*)(p + next));
    return __builtin_bit_cast(bf16x8_t, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}

// f(Const<0>), ..., f(Const<N - 1>)
template <int N, int I = 0, typename F>
__device__ __forceinline__ void each(F&& f) {
    if constexpr (I < N) {
        f(Const<I>());
        each<N, I + 1>(f);
    }
}

// ---- activations, in fp32 -------------------------------------------------
__device__ __forceinline__ float sigmoid_f(float v) { return 1.0f / (1.0f + __expf(-v)); }
__device__ __forceinline__ float silu_f(float v) { return v * sigmoid_f(v); }
// the normal distribution, by erfc: 1 + erf cancels for negative v (4 % off at -5)
__device__ __forceinline__ float normal_cdf(float v) { return 0.5f * erfcf(v * -0.70710678118654752f); }
__device__ __forceinline__ float gelu_f(float v) { return v * normal_cdf(v); }
__device__ __forceinline__ float act_f(float v, int act) {
    if (act == kActRelu) return v < 0.0f ? 0.0f : v;  // NaN passes through
    if (act == kActSilu) return silu_f(v);
    if (act == kActGelu) return gelu_f(v);
    return v;
}

__device__ __forceinline__ float bf16_at(const uint16_t* p) { return __uint_as_float((uint32_t)*p << 16); }

// c += p q^T (16 x 16, 32 of k) with c in accumulation registers. The compiler,
// given the choice, keeps part of 256 sums in the others and moves them over
// and back in every step; written out, and held where they are ahead of the main
// loop (keep()), they stay. Results may be read after settle(), and no vector
// instruction may write an operand or a sum within two wait states ahead: the
// compiler does not see a matrix instruction here, so both are checked on the
// generated code (tests/test_products_code.py, tests/test_products_operands.py).
__device__ __forceinline__ void multiply(float4_t& c, const bf16x8_t& p, const bf16x8_t& q) {
    asm("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(c) : "v"(p), "v"(q));
}
// Waits until the last matrix instructions have written their results (the
// compiler does not see them in multiply(), so it inserts no waits of its own).
__device__ __forceinline__ void keep(float4_t& c) { asm volatile("" : "+a"(c)); }  // there until here
__device__ __forceinline__ void settle() { asm volatile("s_nop 15\n\ts_nop 15" ::: "memory"); }

// d = p q over 128 of k, not accumulated. It keeps its place among the volatile
// statements; result_here(d) has to stand between it and the first use of d, with
// three others or settle() before that. After a use it keeps that in its place.
__device__ __forceinline__ void product_fp8(float4_t& d, const int8_t_& p, const int8_t_& q) {
    asm volatile("v_mfma_f32_16x16x128_f8f6f4 %0, %1, %2, 0" : "=&v"(d) : "v"(p), "v"(q));
}
__device__ __forceinline__ void result_here(float4_t& d) { asm volatile("" : "+v"(d)); }

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

// 8 values to (bf16 or fp32), or bf16 values added from, columns `apart` apart:
// in whole 16-byte pieces where they are consecutive, the row is aligned
// (apart == 1) and all are there.
__device__ __forceinline__ void store_spaced(void* out, int64_t at, const float* v, int have, int apart, bool f32) {
    if (apart == 1 && have == 8) {
        store_run<8>(out, at, v, 8, f32, true);
    } else if (f32) {
#pragma unroll
        for (int q = 0; q < 8; ++q)
            if (q < have) static_cast<float*>(out)[at + q * apart] = v[q];
    } else {
#pragma unroll
        for (int q = 0; q < 8; ++q)
            if (q < have) static_cast<uint16_t*>(out)[at + q * apart] = (uint16_t)pack_bf16x2(v[q], 0.0f);
    }
}
__device__ __forceinline__ void add_spaced(const uint16_t* p, float* v, int have, int apart) {
    if (apart == 1 && have == 8) {
        const uint4 w = *reinterpret_cast<const uint4*>(p);
        const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int q = 0; q < 8; q += 2) {
            v[q] += bf16_lo(x[q / 2]);
            v[q + 1] += bf16_hi(x[q / 2]);
        }
        return;
    }
#pragma unroll
    for (int q = 0; q < 8; ++q)
        if (q < have) v[q] += bf16_at(p + q * apart);
}

// Loads up to N consecutive bf16 values as fp32 (zero past `have`).
template <int N>
__device__ __forceinline__ void load_run(const uint16_t* p, int have, bool wide, float* v) {
    if (wide && have >= N) {
        uint32_t w[N / 2];
        if constexpr (N == 8) {
            const uint4 q = *reinterpret_cast<const uint4*>(p);
            w[0] = q.x, w[1] = q.y, w[2] = q.z, w[3] = q.w;
        } else {
            const uint2 q = *reinterpret_cast<const uint2*>(p);
            w[0] = q.x, w[1] = q.y;
        }
#pragma unroll
        for (int i = 0; i < N; i += 2) {
            v[i] = bf16_lo(w[i / 2]);
            v[i + 1] = bf16_hi(w[i / 2]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = i < have ? bf16_at(p + i) : 0.0f;
    }
}

// The LDS rows (RB = 128 or 64 bytes) of a k-contiguous tile hold their 16-byte
// pieces in an order that depends on the row: piece c of row r is at c ^ key(r),
// so that the 16 rows a matrix instruction takes are spread over all banks (no
// conflict counted). The rows of one instruction are 16 consecutive rows of Q,
// and for P the rows (i / 4) * RUN + i % 4 (RUN consecutive columns per lane):
// key depends on i only.
template <int RB, int RUN>
__device__ __forceinline__ int row_key(int row) {
    return RB == 64 ? -(row / RUN) & 3 : (row & 3) | (((row / RUN) & 1) << 2);
}
// The same for transposed tiles (rows of one k): the LDS transposing read takes
// 32 bytes from each of 8 rows at a time (rows 0-3 and 8-11, ...).
__device__ __forceinline__ int k_key(int kr) { return ((kr & 3) << 1) | (kr & 8); }

// Kernel arguments: see GemmArgs in cgd_experts_launch.h.
template <int BM, int BN, int WM, int WN, int ST, int RB, bool QT, bool PT, bool FP8>
__global__ __launch_bounds__(WM* WN* kWave, ST ? 2 : 1) void gemm_kernel(const GemmArgs a) {
    constexpr int NW = WM * WN;              // waves
    constexpr int TM = BM / WM, TN = BN / WN;  // a wave's part
    constexpr int MT = TM / 16, NT = TN / 16, NH = NT / 2;
    constexpr int RUN = 4 * NH;              // consecutive columns per lane
    constexpr int BK = FP8 ? RB : RB / 2;    // RB bytes of k in a stage
    constexpr int QB = BM * RB, PB = BN * RB;
    constexpr int RPL = 1024 / RB;           // tile rows in one 1-KB load, CPR 16-byte pieces in each
    constexpr int CPR = RB / 16;
    // scales of a stage: one per row, the weights', and a place that is never read
    constexpr int SROWS = BM < 64 ? 64 : BM;
    constexpr int SB = FP8 ? SROWS * 4 + 512 : 0;
    constexpr int STAGE = QB + PB + SB;
    constexpr int QL = QB / 1024 / NW, PL = PB / 1024 / NW;  // 1-KB loads per wave
    constexpr int SL = FP8 ? 1 : 0;
    constexpr int LOADS = QL + PL + SL;
    static_assert(QL >= 1 && PL >= 2 && NT % 2 == 0 && MT >= 1, "tile too small for its waves");
    static_assert(!FP8 || (!QT && !PT && RB == 128), "FP8 tiles are k-contiguous");
    static_assert(RB == 128 || RB == 64, "a stage holds 128 or 64 bytes of k");
    static_assert(PT || (NW * RPL % ((RB == 64 ? 4 : 2) * RUN) == 0 && (BN / 2) % ((RB == 64 ? 4 : 2) * RUN) == 0), "a lane's piece of k is the same in all its loads");
    static_assert(!FP8 || SROWS / 64 + 1 <= NW, "one wave loads 64 row scales, one the weights'");
    // The epilogue's rows go through LDS PASSES times, IPP 16-row tiles of each wave at a time.
    constexpr int PASSES = ST == 0 ? 4 : MT > 4 ? MT : MT > 2 ? 2 : 1, IPP = MT / PASSES;
    constexpr int ROWS = WM * IPP * 16;
    // Tiles with a CU to themselves: one block for each CU takes them in turn.
    constexpr bool ALONE = ST == 0 || BM * BN > 192 * 128;
    // LDS: ST stages of both operands; or (ST = 0) two of P and three of Q, all
    // 160 KB, the epilogue's rows in two of Q's; or (FP8) two of P, three of Q and
    // of the scales, the epilogue's rows in the last of Q's and behind it.
    constexpr int STAGED = ST == 0 ? 2 * PB + QB : ALONE ? 2 * (PB + QB) + 3 * SB : 0;
    constexpr int LDS_BYTES = ST == 0 ? 3 * QB + 2 * PB : ALONE ? STAGED + ROWS * BN * 4 : ST * STAGE;
    static_assert(!ALONE || (ST > 0 ? ROWS * BN * 4 >= QB : true), "the last of Q's slots");
    __shared__ __attribute__((aligned(1024))) char smem[LDS_BYTES];

    const int lane = lane_id();
    const int wave = uniform(threadIdx.x / kWave);
    const int wm = wave / WN, wn = wave % WN;
    const int li = lane & 15, lg = lane >> 4;

    // ---- which tile -------------------------------------------------------
    // Blocks go to the 8 XCDs in turn; each XCD takes one run of consecutive
    // tiles, and within a run 4 row tiles share a column of tiles, so that the
    // tiles in flight on an XCD share operands in its L2. A block takes every
    // gridDim / 8th tile of its XCD's run. A tile of a weight gradient takes as long as
    // its group has rows, so an XCD's run may hold long groups alone: there the XCDs take
    // 16 tiles in turn (4 or 64 measured up to 20 % more). That costs shared operands, so it
    // pays with few groups, an XCD's run lying within one or two, or with long runs. Both
    // gradients in us, in runs and in turn, groups' rows spread by e^0.1 / by e^0.6:
    //   2 to 15 groups, runs of 64 tiles and more:   10 of 700 rows, 2048 x 2048   149 131 / 159 133
    //     (4 of 1500, 2048 x 4096  234 201 / 237 209;   15 of 512, 2048 x 2048     204 207 / 213 208)
    //     shorter runs:  4 of 1024, 2048 x 2048  113 111 / 115 113; 12 of 512, 1024 x 1280 62 79 / 66 83
    //   16 groups and more, runs of 256 and more:    32 of 512, 2048 x 3200        540 543 / 611 539
    //     (32 of 512, 4096 x 4096  1250 1313 / 1379 1281)
    //     shorter runs: 16 of 512, 2048 x 2048   206 222 / 222 224; 24 of 400, the same 235 250 / 262 260
    constexpr int GM = 4;
    const int half_n = a.glu ? BN / 2 : BN;  // output columns of a tile
    const int ntn = (int)((a.n + half_n - 1) / half_n);
    const int ntm = QT ? (int)((a.m + BM - 1) / BM) : uniform(find_piece<false>(a.g, BM, 0).total);
    const int tiles = ntm * ntn * a.splits * (QT ? a.g.groups : 1);
    const int run_len = (tiles + 7) / 8;
    const bool shared_out = QT && ALONE && a.g.groups > 1 && run_len >= (a.g.groups < 16 ? 64 : 256);
    struct Tile {
        int group, split;
        int64_t m0, rows;    // weight gradient: first output row; rows of the tile that exist (may exceed BM)
        int64_t row0;        // first row of x (of d and x: of the reduction)
        int64_t n0, k0, klen;
    };
    auto locate = [&](int seq, Tile* t) -> bool {
        const int xcd = (int)(blockIdx.x & 7);
        const int id = shared_out ? ((seq / 16 * 8 + xcd) * 16) + seq % 16 : xcd * run_len + seq;
        if ((!shared_out && seq >= run_len) || id >= tiles) return false;
        t->split = id / (ntm * ntn);
        const int in0 = id - t->split * (ntm * ntn);
        const int sr = in0 / (GM * ntn);
        const int gm = ntm - sr * GM < GM ? ntm - sr * GM : GM;
        const int in = in0 - sr * GM * ntn;
        const int tm = sr * GM + in % gm;
        t->n0 = (int64_t)uniform(in / gm) * half_n;
        if (!QT) {
            const Piece pc = find_piece<true>(a.g, BM, tm);
            if (pc.group < 0) return false;
            t->group = uniform(pc.group);
            t->row0 = uniform64(pc.row0);
            t->rows = uniform64(pc.rows);
            t->m0 = 0;
            t->k0 = uniform64((int64_t)t->split * a.ksplit);
            t->klen = uniform64(a.k - t->k0 < a.ksplit ? a.k - t->k0 : a.ksplit);
        } else {  // the reduction goes over a group's rows
            t->group = uniform(t->split / a.splits);
            t->split = uniform(t->split - t->group * a.splits);
            int64_t b = 0, n = a.g.total;
            if (a.g.offset || a.g.count || a.g.groups > 1) group_rows(a.g, t->group, &b, &n);
            const int64_t piece = ((n + BK - 1) / BK + a.splits - 1) / a.splits * BK, first = t->split * piece;
            t->row0 = uniform64(b + (first < n ? first : n));
            t->klen = uniform64(first >= n ? 0 : n - first < piece ? n - first : piece);
            t->k0 = 0;
            t->m0 = (int64_t)uniform(tm) * BM;
            t->rows = a.m - t->m0;
        }
        return true;
    };
    int seq = (int)(blockIdx.x >> 3);
    Tile cur;
    if (!locate(seq, &cur)) return;

    // ---- where the operands are --------------------------------------------
    // Q: k-contiguous: rows row0 .. ; transposed: columns m0 .. of rows row0 ..
    // A lane that has nothing to load in any stage (rows or columns past the
    // tile's) keeps kPastEnd; k is checked stage by stage against k_left.
    int4_t qd, pd0, pd1, sd;
    uint32_t qv[QL], pv[PL], sv = kPastEnd;
    int qk[QT ? QL : 1], pk[PT ? PL : 1];  // where in the stage's k a lane's loads are
    int kq_left, kp_left;                  // k left from the next stage of each on
    constexpr int ES = FP8 ? 1 : 2;
    const int ldq = (int)a.ldq, ldp = (int)a.ldp;
    const int64_t q_step = QT ? BK * a.ldq : RB, p_step = PT ? BK * a.ldp : RB;
    int64_t s_step = 0;
    const bool s_byte = FP8 && a.qs_byte && wave != NW - 1;

    // From the last stage on (a whole one included, once it is past) lanes whose
    // piece of k lies behind the end load nothing.
    auto mask_q = [&]() {
        if (kq_left >= BK) return;
#pragma unroll
        for (int i = 0; i < QL; ++i) qv[i] = qk[QT ? i : 0] < kq_left ? qv[i] : kPastEnd;
        if (FP8) sv = kq_left > 0 ? sv : kPastEnd;
    };
    auto mask_p = [&]() {
        if (kp_left >= BK) return;
#pragma unroll
        for (int j = 0; j < PL; ++j) pv[j] = pk[PT ? j : 0] < kp_left ? pv[j] : kPastEnd;
    };
    auto aim = [&](const Tile& t) {
        const int lane = afresh(threadIdx.x) & (kWave - 1);
        if (!QT) {
            qd = buffer_from((uint64_t)a.q + (uint64_t)(t.row0 * a.ldq + t.k0 * ES));
            qk[0] = ((lane & (CPR - 1)) ^ row_key<RB, 4>(wave * RPL + lane / CPR)) * (16 / ES);
#pragma unroll
            for (int j = 0; j < QL; ++j) {
                const int row = (j * NW + wave) * RPL + lane / CPR;
                qv[j] = row < t.rows ? (uint32_t)(row * ldq + qk[0] * ES) : kPastEnd;
            }
        } else {
            constexpr int RPI = 512 / BM;  // k rows per 1-KB load
            qd = buffer_from((uint64_t)a.q + (uint64_t)(t.row0 * a.ldq + t.m0 * 2));
#pragma unroll
            for (int j = 0; j < QL; ++j) {
                qk[j] = (j * NW + wave) * RPI + lane / (64 / RPI);
                const int c = ((lane & (64 / RPI - 1)) ^ k_key(qk[j])) * 16;
                qv[j] = t.m0 * 2 + c < a.ldq ? (uint32_t)(qk[j] * ldq + c) : kPastEnd;
            }
        }
        if (!PT) {
            const uint64_t base = (uint64_t)a.p + (uint64_t)((int64_t)t.group * a.p_group + t.k0 * ES);
            const int64_t second = a.glu ? a.n + t.n0 : t.n0 + BN / 2;  // first weight row of the tile's upper half
            const int64_t left0 = a.n - t.n0, left1 = a.glu ? left0 : a.n - second;
            pd0 = buffer_from(base + (uint64_t)(t.n0 * a.ldp));
            pd1 = buffer_from(base + (uint64_t)(second * a.ldp));
            pk[0] = ((lane & (CPR - 1)) ^ row_key<RB, RUN>(wave * RPL + lane / CPR)) * (16 / ES);
#pragma unroll
            for (int j = 0; j < PL; ++j) {
                const int row = ((j % (PL / 2)) * NW + wave) * RPL + lane / CPR;
                pv[j] = row < (j < PL / 2 ? left0 : left1) ? (uint32_t)(row * ldp + pk[0] * ES) : kPastEnd;
            }
        } else {
            constexpr int RPI = 512 / BN;
            pd0 = pd1 = buffer_from((uint64_t)a.p + (uint64_t)((int64_t)t.group * a.p_group + (QT ? t.row0 * a.ldp : 0) + t.n0 * 2));
#pragma unroll
            for (int j = 0; j < PL; ++j) {
                pk[j] = (j * NW + wave) * RPI + lane / (64 / RPI);
                const int c = ((lane & (64 / RPI - 1)) ^ k_key(pk[j])) * 16;
                pv[j] = t.n0 * 2 + c < a.ldp ? (uint32_t)(pk[j] * ldp + c) : kPastEnd;
            }
        }
        // FP8 scales: wave w < BM/64 brings those of rows 64 w .., the last wave
        // those of the two weight blocks the tile's halves lie in (lanes 0 and 1:
        // the halves are at most 128 wide and start at multiples of their width,
        // and SwiGLU's up rows start at a multiple of 128).
        if (FP8) {
            const int64_t kb0 = t.k0 / 128;
            uint64_t sb = 0;
            sv = kPastEnd;
            if (wave == NW - 1) {
                sb = (uint64_t)a.ps + (uint64_t)(((int64_t)t.group * a.ps_group + kb0) * 4);
                const int64_t second = a.glu ? a.n + t.n0 : t.n0 + BN / 2;
                const int64_t row = lane == 0 ? t.n0 : second;
                if (lane < 2 && row < a.n * (a.glu ? 2 : 1)) sv = (uint32_t)(row / 128 * a.ps_row * 4);
                s_step = 4;
            } else {
                const int row = wave * 64 + lane;
                const int size = a.qs_byte ? 1 : 4;
                sb = (uint64_t)a.qs + (uint64_t)((t.row0 * a.qs_row + kb0 * a.qs_blk) * size);
                if (row < BM && row < t.rows) sv = (uint32_t)(row * a.qs_row * size);
                s_step = a.qs_blk * size;
            }
            sd = buffer_from(sb);
        }
        kq_left = kp_left = uniform((int)t.klen);
        mask_q();
        mask_p();
    };

    const uint32_t lds0 = uniform((int)lds_address(smem)) + wave * 1024;
    // Load `I` of the next stage of Q (of P, of the scales); l: this wave's
    // place in the stage's slot (its loads go NW KB apart).
    auto load_q = [&](auto I, uint32_t l) { load_to_lds16<decltype(I)::value * NW * 1024>(qd, qv[decltype(I)::value], l); };
    auto load_p = [&](auto J, uint32_t l) {
        constexpr int j = decltype(J)::value;
        load_to_lds16<j * NW * 1024>(!PT && j >= PL / 2 ? pd1 : pd0, pv[j], l);
    };
    auto load_s = [&](uint32_t l) {
        // waves with neither rows nor the weights' scales load zeros into the
        // unread place: every wave has the same count of loads to wait for
        const uint32_t dst = l - wave * 1024 + (wave == NW - 1 ? SROWS * 4 : wave * 64 < SROWS ? wave * 256 : SROWS * 4 + 256);
        if (s_byte)
            load_to_lds1(sd, sv, dst);
        else
            load_to_lds4(sd, sv, dst);
    };
    auto next_q = [&]() {
        advance(qd, q_step);
        if (FP8) advance(sd, s_step);
        kq_left -= BK;
        mask_q();
    };
    auto next_p = [&]() {
        advance(pd0, p_step);
        if (!PT) advance(pd1, p_step);
        kp_left -= BK;
        mask_p();
    };
    auto load_piece = [&](auto I, int buf) {
        constexpr int i = decltype(I)::value;
        const uint32_t l = lds0 + (uint32_t)(buf * STAGE);
        if constexpr (i < QL)
            load_q(I, l);
        else if constexpr (i < QL + PL)
            load_p(Const<i - QL>(), l + QB);
        else
            load_s(l + QB + PB);
    };
    auto load_stage = [&](int buf) {
        each<LOADS>([&](auto I) { load_piece(I, buf); });
        next_q();
        next_p();
    };

    float4_t acc[MT][NT];
    // A lane holds one row of each 16-row tile i and 4 consecutive columns of
    // each column piece j: j < NH in the lower half of the tile, the others the
    // same columns of the upper half.
    auto column = [&](int j, int lg) -> int {  // within its half
        return wn * (TN / 2) + (PT ? j % NH * 16 + lg * 4 : lg * RUN + j % NH * 4);
    };
    auto clear_sums = [&](const Tile& t) {  // to the bias
        const int lg = (afresh(threadIdx.x) & (kWave - 1)) >> 4;
        float4_t z[NT];
#pragma unroll
        for (int j = 0; j < NT; ++j) z[j] = float4_t{0.f, 0.f, 0.f, 0.f};
        if (!PT && a.bias && a.splits == 1) {
            const uint16_t* b = static_cast<const uint16_t*>(a.bias) + (int64_t)t.group * (a.glu ? 2 * a.n : a.n);
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const int64_t c = t.n0 + column(j, lg) + (j >= NH && !a.glu ? BN / 2 : 0);
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    if (c + q < a.n) z[j][q] = bf16_at(b + (j >= NH && a.glu ? a.n : 0) + c + q);
            }
        }
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int j = 0; j < NT; ++j) acc[i][j] = z[j];
    };

    // ---- LDS addresses of a lane's fragments -------------------------------
    const CGD_LDS(char)* sm = (const CGD_LDS(char)*)smem;
    // k-contiguous: piece (ks * 4 + lg) of the row, for ks = 0, 1
    int qa[QT ? MT : 2], pa[PT ? NT : 2];
    if (!QT) {
        const int row = wm * TM + li;
        qa[0] = row * RB + ((lg ^ row_key<RB, 4>(row)) << 4);
        qa[1] = row * RB + (((4 + lg) ^ row_key<RB, 4>(row)) << 4);
    } else {
        // four columns of 16-row tile u from k row lg * 8 + li / 4
        const int kr = lg * 8 + (li >> 2);
#pragma unroll
        for (int u = 0; u < MT; ++u) {
            const int col = wm * TM + u * 16 + (li & 3) * 4;
            qa[u] = kr * (BM * 2) + (((col >> 3) ^ k_key(kr)) << 4) + (col & 7) * 2;
        }
    }
    if (!PT) {
        const int row = wn * (TN / 2) + (li >> 2) * RUN + (li & 3);
        pa[0] = row * RB + ((lg ^ row_key<RB, RUN>(row)) << 4);
        pa[1] = row * RB + (((4 + lg) ^ row_key<RB, RUN>(row)) << 4);
    } else {
        const int kr = lg * 8 + (li >> 2);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const int col = t / NH * (BN / 2) + wn * (TN / 2) + t % NH * 16 + (li & 3) * 4;
            pa[t] = kr * (BN * 2) + (((col >> 3) ^ k_key(kr)) << 4) + (col & 7) * 2;
        }
    }
    auto q_frag = [&](int base, int ks, int mt) -> bf16x8_t {
        if (!QT) return *(const CGD_LDS(bf16x8_t)*)(sm + base + qa[ks] + mt * 16 * RB);
        const int at = base + qa[mt] + ks * 32 * (BM * 2);
        return turned(sm + at, 4 * (BM * 2));
    };
    auto p_frag = [&](int base, int ks, int nt) -> bf16x8_t {
        const int h = nt / NH, t = nt % NH;
        if (!PT) return *(const CGD_LDS(bf16x8_t)*)(sm + base + pa[ks] + h * (BN / 2) * RB + t * 4 * RB);
        const int at = base + pa[nt] + ks * 32 * (BN * 2);
        return turned(sm + at, 4 * (BN * 2));
    };

    // ---- loads ahead of the main loop ----------------------------------------
    auto qslot = [&](int slot) { return 2 * PB + slot * QB + (FP8 && slot == 2 ? 3 * SB : 0); };
    // (four-wave tiles: all that does not go where the epilogue works; then the rest)
    constexpr int S_AT = 2 * PB + 2 * QB;  // the scales' slots
    auto start = [&](const Tile& t) {
        aim(t);
        if constexpr (FP8 && ALONE) {
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                each<PL>([&](auto I) { load_p(I, lds0 + s * PB); });
                next_p();
                each<QL>([&](auto I) { load_q(I, lds0 + qslot(s)); });
                load_s(lds0 + S_AT + s * SB);
                next_q();
            }
        } else if constexpr (ST == 0) {
            each<PL>([&](auto I) { load_p(I, lds0); });
            next_p();
            each<QL>([&](auto I) { load_q(I, lds0 + qslot(0)); });
            next_q();
            each<PL>([&](auto I) { load_p(I, lds0 + PB); });
            next_p();
        } else if constexpr (RB == 64) {
#pragma unroll
            for (int s = 0; s < ST; ++s) load_stage(s);
        } else {
#pragma unroll
            for (int s = 0; s < ST - 1; ++s)
                if (s * BK < t.klen) load_stage(s);
        }
    };
    auto start_rest = [&]() {
        if constexpr (ST == 0) {
#pragma unroll
            for (int s = 1; s < 3; ++s) {
                each<QL>([&](auto I) { load_q(I, lds0 + qslot(s)); });
                next_q();
            }
        }
    };

    // ---- main loop ----------------------------------------------------------
    auto multiply_tile = [&](const int nk) {
        if constexpr (FP8 && ALONE) {
            // A step is 128 of k: MT rows of NT products from zero, each added with its
            // scales one row later, just before the same place's next product (vector
            // and matrix instructions of two waves share a SIMD). A row's operand and
            // scale are read one row ahead, P's operands of the next step in the course
            // of this one, so nothing waits for LDS behind the barrier; the barrier of a
            // step stands before the last row of the step before, whose operands are in
            // registers by then. P has one step's time to arrive, Q two.
            int8_t_ pf[2][NT], qf[2];
            float4_t d[NT];
            uint32_t sx[2] = {0, 0};  // as they are in memory
            float w0 = 0.f, w1 = 0.f;
            auto whole = [&](const CGD_LDS(char)* at, int a0, int a1, int off) -> int8_t_ {
                const int4_t lo = *(const CGD_LDS(int4_t)*)(at + a0 + off), hi = *(const CGD_LDS(int4_t)*)(at + a1 + off);
                return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
            };
            auto read_p = [&](int base, int j) {
                return whole(sm + base, pa[0], pa[1], j / NH * (BN / 2) * RB + j % NH * 4 * RB);
            };
            auto read_q = [&](int base, int i) { return whole(sm + base, qa[0], qa[1], i * 16 * RB); };
            const int sa = afresh(S_AT + (wm * TM + li) * 4);
            auto read_s = [&](int at, int i) { return *(const CGD_LDS(uint32_t)*)(sm + at + i * 64); };
            const int sh = a.qs_byte ? 23 : 0;
            const uint32_t least = a.qs_byte ? 0x00400000u : 0u;  // (UE8M0: 2^-127)
            float f0, f1;
            auto scale = [&](auto I) {  // both of row I's
                const uint32_t v = sx[decltype(I)::value & 1] << sh;
                const float x = __uint_as_float(v > least ? v : least);
                f0 = x * w0;
                f1 = x * w1;
            };
            auto add = [&](auto I, int j) {  // row I's product j, NT - 1 others after it
                constexpr int i = decltype(I)::value;
                result_here(d[j]);
#pragma unroll
                for (int r = 0; r < 4; ++r) acc[i][j][r] = fmaf(d[j][r], j < NH ? f0 : f1, acc[i][j][r]);
                result_here(acc[i][j]);
            };
            auto row = [&](auto I, auto SET) {  // row I's products, the sums of the row before
                constexpr int i = decltype(I)::value, set = decltype(SET)::value;
                using Before = Const<i == 0 ? MT - 1 : i - 1>;
                scale(Before());
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    add(Before(), j);
                    product_fp8(d[j], pf[set][j], qf[i & 1]);
                }
            };
            static_assert(!(FP8 && ALONE) || (MT == 6 && NT == 4 && QL == 3 && PL == 4), "the schedule below");
            wait_loads<2 * (QL + 1) + PL>();
            block_barrier();
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                pf[0][j] = read_p(0, j);
                pf[1][j] = int8_t_{};  // the first step adds two rows of zeros
                d[j] = float4_t{0.f, 0.f, 0.f, 0.f};
            }
            qf[1] = int8_t_{};
            int slot = 0, ahead = 2;  // Q's slots of this step and of the one after the next
            auto step = [&](auto SET) {
                constexpr int set = decltype(SET)::value;
                // Q and the scales of this step and P of the next have landed; every wave has
                // read the last one's Q and this one's P
                wait_loads<QL + 1>();
                sync_lds();
                const int qbase = qslot(slot), s_at = sa + slot * SB;
                each<PL>([&](auto I) { load_p(I, lds0 + set * PB); });
                next_p();
                qf[0] = read_q(qbase, 0);
                const uint32_t first = read_s(s_at, 0);
                const CGD_LDS(float)* ws = (const CGD_LDS(float)*)(sm + S_AT + slot * SB + SROWS * 4);
                const float nw0 = ws[0], nw1 = ws[1];
                row(Const<MT - 1>(), Const<1 - set>());
                sx[0] = first;
                __builtin_amdgcn_sched_barrier(0);
                each<MT - 1>([&](auto I) {
                    constexpr int i = decltype(I)::value;
                    qf[(i + 1) & 1] = read_q(qbase, i + 1);
                    const uint32_t ns = read_s(s_at, i + 1);
                    if constexpr (i < NT) pf[1 - set][i] = read_p((1 - set) * PB, i);
                    row(I, SET);
                    if constexpr (i == 0) w0 = nw0, w1 = nw1;
                    sx[(i + 1) & 1] = ns;
                    if constexpr (i < QL) load_q(I, lds0 + qslot(ahead));
                    if constexpr (i == QL) load_s(lds0 + S_AT + ahead * SB);
                    __builtin_amdgcn_sched_barrier(0);
                });
                next_q();
                slot = slot == 2 ? 0 : slot + 1;
                ahead = ahead == 2 ? 0 : ahead + 1;
            };
            int kt = 0;
            for (; kt + 1 < nk; kt += 2) {
                step(Const<0>());
                step(Const<1>());
            }
            if (kt < nk) {
                step(Const<0>());
                row(Const<MT - 1>(), Const<0>());
                settle();  // in both branches: what they give is moved together behind them
            } else {
                row(Const<MT - 1>(), Const<1>());
                settle();
            }
            scale(Const<MT - 1>());
#pragma unroll
            for (int j = 0; j < NT; ++j) add(Const<MT - 1>(), j);
        } else if constexpr (ST == 0) {
            // Few, large waves: the 64 products of half a stage (32 of k) run on
            // operands that were read from LDS during the half before, with one LDS
            // read, load or address slipped behind a product each, so that one wave
            // per SIMD keeps its matrix unit fed. Half way through stage k every
            // wave has read all of it: after the barrier there the loads of P's
            // stage k + 2 (needed a stage later, so they go first) and Q's stage
            // k + 3 (needed two stages later) take its place. Three slots for Q
            // (activations, which come from HBM and are shared by fewer tiles in
            // flight) and two for P measured 1350 us at 32768 x 4096 x 7168, the
            // other way round 1425. Loads past the end are issued all the same
            // (they touch no memory), which keeps the count of loads to wait for
            // the same in every step. 32 x 32 products need half the instructions
            // but measured slower (more traffic of sums for the same power).
            static_assert(ST || (QL == 8 && PL == 8 && MT == 8 && NT == 8), "the schedule below is for 64 products in half a stage");
            int q_read = 0;  // Q's slot of stage kt
            bf16x8_t qf[2][MT], pf[2][NT];
            // fragment n of the next half stage: P's first, all of which its first row needs
            auto fetch = [&](auto N, auto SET, int ks, int qbase, int pbase) {
                constexpr int n = decltype(N)::value, set = decltype(SET)::value;
                if constexpr (n < NT)
                    pf[set][n] = p_frag(pbase, ks, n);
                else
                    qf[set][n - NT] = q_frag(qbase, ks, n - NT);
            };
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int j = 0; j < NT; ++j) keep(acc[i][j]);  // where they stay (see multiply())
            wait_loads<PL + 2 * QL>();
            block_barrier();
            each<MT + NT>([&](auto N) { fetch(N, Const<0>(), 0, qslot(0), 0); });
            for (int kt = 0;;) {  // at least one stage: an empty reduction multiplies zeros
                const int pbase = (kt & 1) * PB, qbase = qslot(q_read);
                q_read = q_read == 2 ? 0 : q_read + 1;
                const int pnext = PB - pbase, qnext = qslot(q_read);
                const uint32_t fq = lds0 + qbase, fp = lds0 + pbase;
                __builtin_amdgcn_sched_barrier(0);
                each<64>([&](auto G) {
                    constexpr int g = decltype(G)::value, i = g / 8, j = g % 8;
                    multiply(acc[i][j], pf[0][j], qf[0][i]);
                    __builtin_amdgcn_sched_barrier(0);
                    if constexpr (g % 3 == 0 && g < 48) fetch(Const<g / 3>(), Const<1>(), 1, qbase, pbase);
                    __builtin_amdgcn_sched_barrier(0);
                });
                // Q's and P's stage kt + 1 have landed; Q's kt + 2 may still be on its way
                wait_loads<QL>();
                block_barrier();
                each<64>([&](auto G) {
                    constexpr int g = decltype(G)::value, i = g / 8, j = g % 8;
                    multiply(acc[i][j], pf[1][j], qf[1][i]);
                    __builtin_amdgcn_sched_barrier(0);
                    if constexpr (g < 16) {
                        if constexpr (g % 2 == 0)
                            aim_load<g / 2 * NW * 1024>(fp);
                        else
                            aimed_load(!PT && g / 2 >= PL / 2 ? pd1 : pd0, pv[g / 2]);
                    } else if constexpr (g < 48) {
                        constexpr int n = (g - 16) / 2;
                        if constexpr (g % 2 == 0)
                            fetch(Const<n>(), Const<0>(), 0, qnext, pnext);
                        else if constexpr (n % 2 == 0)
                            aim_load<n / 2 * NW * 1024>(fq);
                        else
                            aimed_load(qd, qv[n / 2]);
                    } else if constexpr (g == 50) {
                        next_q();
                    } else if constexpr (g == 54) {
                        next_p();
                    }
                    __builtin_amdgcn_sched_barrier(0);
                });
                if (++kt >= nk) {
                    settle();  // on the way out, before the sums are touched
                    break;
                }
            }
        } else if constexpr (RB == 64) {
            // Operands are read from LDS one stage ahead into the other of two
            // register sets, so the matrix instructions of a stage wait for
            // nothing; ST stages are on their way or being read. Loads past the
            // end are issued all the same (they touch no memory), which keeps the
            // count of loads to wait for the same in every step.
            bf16x8_t qf[2][MT], pf[2][NT];
            wait_loads<(ST - 1) * LOADS>();
            block_barrier();
#pragma unroll
            for (int j = 0; j < NT; ++j) pf[0][j] = p_frag(QB, 0, j);
#pragma unroll
            for (int i = 0; i < MT; ++i) qf[0][i] = q_frag(0, 0, i);
            int slot = 0;  // of stage kt
            auto step = [&](auto set) {
                constexpr int S = decltype(set)::value;
                // stage kt + 1 has landed for every wave, and every wave has read stage kt
                wait_loads<(ST - 2) * LOADS>();
                block_barrier();
                const int refill = slot;
                slot = slot + 1 == ST ? 0 : slot + 1;
                const int base = slot * STAGE;
                __builtin_amdgcn_sched_barrier(0);
                // row by row: LDS reads for the next stage, matrix instructions of
                // this one, a load of the stage that takes the freed slot
                each<MT>([&](auto I) {
                    constexpr int i = decltype(I)::value;
#pragma unroll
                    for (int j = i * NT / MT; j < (i + 1) * NT / MT; ++j) pf[1 - S][j] = p_frag(base + QB, 0, j);
                    qf[1 - S][i] = q_frag(base, 0, i);
#pragma unroll
                    for (int j = 0; j < NT; ++j)
                        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(pf[S][j], qf[S][i], acc[i][j], 0, 0, 0);
                    if constexpr (i < LOADS) load_piece(I, refill);
                    if constexpr (i == MT - 1) {
                        next_q();
                        next_p();
                    }
                    __builtin_amdgcn_sched_barrier(0);
                });
                static_assert(LOADS <= MT, "one load for each row of the wave's tile");
            };
            int kt = 0;
            for (; kt + 1 < nk; kt += 2) {
                step(Const<0>());
                step(Const<1>());
            }
            if (kt < nk) step(Const<0>());
        } else {
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
                    for (int j = 0; j < NT; ++j) pf[j] = p_frag(base + QB, ks, j);
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
                    const int4_t lo = __builtin_bit_cast(int4_t, p_frag(base + QB, 0, j)), hi = __builtin_bit_cast(int4_t, p_frag(base + QB, 1, j));
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
        }
    };

    // ---- epilogue -----------------------------------------------------------
    // The sums go through LDS, some 16-row tiles of each wave at a time, so that
    // what follows is a short loop over rows (written out over the registers it
    // is code that is fetched once for each tile, which took longer than the
    // work), with 8 columns of the tile's lower half and the same 8 of its upper
    // half per lane and lanes along a row. Four-wave tiles use two of Q's slots
    // for it, so that the next tile's first loads can travel meanwhile.
    constexpr int RUNS = BN / 16;        // lanes along a row
    constexpr int STEP = NW * kWave / RUNS, ITER = ROWS / STEP;
    static_assert(MT % PASSES == 0 && ROWS % STEP == 0 && ROWS * BN * 4 + STAGED <= LDS_BYTES, "rows of a pass fit");
    const bool wide_n = (a.n & 7) == 0;
    const int64_t np = (a.n + 7) / 8 * 8;  // columns of a partial sum's row: padded to whole stores
    auto finish = [&](const Tile& t) {
        const int tid = afresh(threadIdx.x), lane = tid & (kWave - 1), li = lane & 15, lg = lane >> 4;
        CGD_LDS(float)* st = (CGD_LDS(float)*)(smem + STAGED);
        // 16-byte unit u of row r lies at u ^ key(r): 16 rows' units are spread over the banks
        auto key = [](int r) { return (r & 15) ^ ((~r & 4) << 1); };
        auto put = [&](auto H) {
            constexpr int i0 = decltype(H)::value * IPP;
#pragma unroll
            for (int i = 0; i < IPP; ++i)
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    if (ST == 0) keep(acc[i0 + i][j]);
                    const int r = (wm * IPP + i) * 16 + li, u = (j / NH * (BN / 2) + column(j, lg)) / 4;
                    *(CGD_LDS(float4_t)*)(st + r * BN + (u ^ key(r)) * 4) = acc[i0 + i][j];
                }
        };
        const int64_t out0 = QT ? (int64_t)t.group * a.m + t.m0 : t.row0;
        const int64_t width = a.glu ? 2 * a.n : a.n;
        const int64_t second = a.glu ? a.n : (int64_t)BN / 2;  // from the lower half's columns to the upper half's
        const int run = tid % RUNS;
        // where the loop below can store whole 16-byte pieces
        const bool whole = a.splits > 1 ||
                           (t.n0 + half_n <= a.n && !a.act &&
                            (wide_n || (a.out_f32 && (a.n & 3) == 0 && !a.preact && !a.residual)));
        each<PASSES>([&](auto H) {  // written out: with a variable index the sums would live in memory
            constexpr int h = decltype(H)::value;
            sync_lds();
            put(H);
            sync_lds();
            auto tile_row = [&](int lr) { return lr / (IPP * 16) * TM + h * (IPP * 16) + lr % (IPP * 16); };
            if (whole) {
                const int64_t c0 = t.n0 + run * 8, c1 = second + c0;
                float v0[ITER][8], v1[ITER][8];
#pragma unroll
                for (int k = 0; k < ITER; ++k) {
                    const int lr = tid / RUNS + k * STEP;
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        const float4_t x = *(const CGD_LDS(float4_t)*)(st + lr * BN + ((run * 2 + q) ^ key(lr)) * 4);
                        const float4_t y = *(const CGD_LDS(float4_t)*)(st + lr * BN + ((BN / 8 + run * 2 + q) ^ key(lr)) * 4);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            v0[k][q * 4 + e] = x[e];
                            v1[k][q * 4 + e] = y[e];
                        }
                    }
                }
#pragma unroll
                for (int k = 0; k < ITER; ++k) {
                    const int r = tile_row(tid / RUNS + k * STEP);
                    if (r >= t.rows) continue;
                    const int64_t row = out0 + r;
                    if (a.splits > 1) {  // partial sums, joined by join_kernel
                        float* p = a.partial + (t.split * (QT ? a.g.groups * a.m : a.g.total) + row) * (a.glu ? 2 * np : np);
                        if (c0 < np) store_run<8>(p, c0, v0[k], 8, true, true);
                        const int64_t d1 = a.glu ? np + c0 : c1;
                        if (a.glu ? c0 < np : c1 < np) store_run<8>(p, d1, v1[k], 8, true, true);
                        continue;
                    }
                    if (a.preact) {
                        store_run<8>(a.preact, row * width + c0, v0[k], 8, false, true);
                        store_run<8>(a.preact, row * width + c1, v1[k], 8, false, true);
                    }
                    if (a.glu) {
#pragma unroll
                        for (int q = 0; q < 8; ++q) v0[k][q] = silu_f(v0[k][q]) * v1[k][q];
                    }
                    if (a.residual) {
                        const uint16_t* res = static_cast<const uint16_t*>(a.residual) + row * a.n;
                        add_spaced(res + c0, v0[k], 8, 1);
                        if (!a.glu) add_spaced(res + c1, v1[k], 8, 1);
                    }
                    store_run<8>(a.out, row * a.n + c0, v0[k], 8, a.out_f32, true);
                    if (!a.glu) store_run<8>(a.out, row * a.n + c1, v1[k], 8, a.out_f32, true);
                }
                return;
            }
            // everything else (an activation, a tile that sticks out to the right,
            // rows that are not a multiple of 16 bytes): single values are stored
            // RUNS columns apart, so that lanes store next to each other
            const int first = wide_n ? run * 8 : run, apart = wide_n ? 1 : RUNS;
            const int64_t c0 = t.n0 + first, c1 = second + c0;
            const int64_t left0 = a.n - c0, left1 = a.glu ? left0 : a.n - c1;
            const int have0 = left0 <= 0 ? 0 : left0 > 7 * apart ? 8 : (int)((left0 + apart - 1) / apart);
            const int have1 = left1 <= 0 ? 0 : left1 > 7 * apart ? 8 : (int)((left1 + apart - 1) / apart);
#pragma unroll 1
            for (int lr = tid / RUNS; lr < ROWS; lr += STEP) {
                const int r = tile_row(lr);
                if (r >= t.rows) continue;
                float v0[8], v1[8];
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    const int c = first + q * apart;
                    v0[q] = st[lr * BN + ((c / 4) ^ key(lr)) * 4 + c % 4];
                    v1[q] = st[lr * BN + ((BN / 8 + c / 4) ^ key(lr)) * 4 + c % 4];
                }
                const int64_t row = out0 + r;
                if (a.preact) {
                    store_spaced(a.preact, row * width + c0, v0, have0, apart, false);
                    store_spaced(a.preact, row * width + c1, v1, have1, apart, false);
                }
                if (a.glu) {
#pragma unroll
                    for (int q = 0; q < 8; ++q) v0[q] = silu_f(v0[q]) * v1[q];
                } else if (a.act) {
#pragma unroll
                    for (int q = 0; q < 8; ++q) {
                        v0[q] = act_f(v0[q], a.act);
                        v1[q] = act_f(v1[q], a.act);
                    }
                }
                if (a.residual) {
                    const uint16_t* res = static_cast<const uint16_t*>(a.residual) + row * a.n;
                    add_spaced(res + c0, v0, have0, apart);
                    if (!a.glu) add_spaced(res + c1, v1, have1, apart);
                }
                store_spaced(a.out, row * a.n + c0, v0, have0, apart, a.out_f32);
                if (!a.glu) store_spaced(a.out, row * a.n + c1, v1, have1, apart, a.out_f32);
            }
        });
    };

    // Tiles with a CU to themselves, inside the output, whose sums are stored as they
    // are or with a residual, need no LDS: a lane has RUN (8 or 16) neighbouring
    // columns of a row in either half, or (P transposed) four pieces of 4 that the
    // four lanes of a row exchange. Through LDS the same took 4 us a tile longer, with
    // nothing to cover it: 4096 x 2048 -> 7168 with a residual 137 us against 125.
    auto finish_plain = [&](const Tile& t) {
        static_assert(!ALONE || (RUN == 16 || (RUN == 8 && !PT)), "runs of whole stores");
        const int lane = afresh(threadIdx.x) & (kWave - 1), li = lane & 15, lg = lane >> 4;
        const int64_t out0 = (QT ? (int64_t)t.group * a.m + t.m0 : t.row0) + wm * TM + li;
        const int64_t c0 = t.n0 + wn * (TN / 2) + lg * RUN;
        const int64_t left = t.rows - wm * TM - li;  // of the lane's rows
        each<MT>([&](auto I) {
            constexpr int i = decltype(I)::value;
            const int64_t at = (out0 + i * 16) * a.n + c0;
            uint4 w[2][NH / 2] = {};
            if (!PT && a.residual && i * 16 < left) {
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int q = 0; q < NH / 2; ++q)
                        w[h][q] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.residual) + at + h * (BN / 2) + q * 8);
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t v[2 * NH];
#pragma unroll
                for (int j = 0; j < NH; ++j) {
                    if (ST == 0) keep(acc[i][h * NH + j]);
                    float4_t x = acc[i][h * NH + j];
                    if (!PT) {
                        const uint32_t lo = j & 1 ? w[h][j / 2].z : w[h][j / 2].x, hi = j & 1 ? w[h][j / 2].w : w[h][j / 2].y;
                        if (a.residual) x += float4_t{bf16_lo(lo), bf16_hi(lo), bf16_lo(hi), bf16_hi(hi)};
                    }
                    v[2 * j] = pack_bf16x2(x[0], x[1]);
                    v[2 * j + 1] = pack_bf16x2(x[2], x[3]);
                }
                if constexpr (PT) {  // piece j of lane row g <-> piece g of lane row j
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const auto p = __builtin_amdgcn_permlane32_swap(v[q], v[q + 4], false, false);
                        v[q] = p[0];
                        v[q + 4] = p[1];
                    }
#pragma unroll
                    for (int q = 0; q < 2; ++q)
#pragma unroll
                        for (int e = 0; e < 8; e += 4) {
                            const auto p = __builtin_amdgcn_permlane16_swap(v[e + q], v[e + q + 2], false, false);
                            v[e + q] = p[0];
                            v[e + q + 2] = p[1];
                        }
                }
                if (i * 16 < left) {
                    uint16_t* o = static_cast<uint16_t*>(a.out) + at + h * (BN / 2);
#pragma unroll
                    for (int q = 0; q < NH / 2; ++q)
                        *reinterpret_cast<uint4*>(o + q * 8) = uint4{v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
                }
            }
        });
    };

    // ---- the block's tiles ----------------------------------------------------
    start(cur);
    start_rest();
    for (;;) {
        Tile next;
        seq += (int)(gridDim.x >> 3);
        const bool more = ALONE && locate(seq, &next);
        clear_sums(cur);
        multiply_tile(uniform((int)((cur.klen + BK - 1) / BK)));
        block_sync();  // every wave is done with LDS, and no load is on its way there
        if (more) start(next);
        if constexpr (ALONE) {
            if (a.splits == 1 && !a.act && !a.glu && !a.preact && !a.out_f32 && wide_n && cur.n0 + BN <= a.n)
                finish_plain(cur);
            else
                finish(cur);
        } else {
            finish(cur);
        }
        if (!more) return;
        sync_lds();
        start_rest();
        cur = next;
    }
}

}  // namespace cgd
