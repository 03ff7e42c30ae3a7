// Forward products in bf16, the choice of tiles, and the kernel that joins a
// split reduction.
#include "cgd_gemm_launch.h"

namespace cgd {

// Tile shapes: 256 x 256 (FP8: 192 x 256, which leaves LDS for the epilogue) once
// there is one for most CUs; 128 x 128 below that, two blocks to a CU; 32 x 128
// for a dense product of up to 128 rows, where a tall tile leaves fewer blocks to
// share the weights' read (4096 x 4096 for 64 rows: 13.6 us against 16.8). Grouped
// products of few rows keep the tall tile: every group's weights are read anyway,
// and a group that does not fit one tile reads them twice (16 experts, 64 rows
// each on average, 7168 -> 2 x 2048: 176 us against 206 with 64 rows a tile).
// Where one tile for each group just fills the blocks that run at once (two for a CU:
// room for fewer than an eighth as many second tiles), the first groups above 128 rows
// start another round: groups that may be uneven take 192 x 128 there. us with 128 and
// 192 rows a tile, mean of five draws; the groups' shares are spread by e^0.5, e^0.2:
//     rows a group              56               64               80               112
//     16 x 7168 -> 2 x 2048     175 181 165 172  214 189 168 176  271 199 175 184  291 259 291 201
//     32 x 2048 -> 2 x 1024      84  78  73  75   88  79  73  76   97  90  74  77   94 103  98  77
//     15 x 7168 -> 2 x 2048     170 176 158 166  190 184 162 171  248 194 171 179  282 257 281 196
//   more room, 128 rows:
//     14 x 7168 -> 2 x 2048     163 171 152 161  164 178 157 166  169 188 166 174  273 196 253 191
//     24 x 4096 -> 2 x 2048     196 203 192 201  195 204 195 204  196 205 200 207  237 215 203 204
//     8 x 4096 -> 4096           82  97  80  93   84  98  81  96   91  99  83  99
// (128 rows a group: the first two lines 295 301 300 205 and 95 103 96 82.) Packed
// buffers say how long a group can be; FP8 has no tile of this shape.
// A reduction is split where even so there were fewer than 512 blocks (two for a CU).
constexpr int kRoundBlocks = 512;
static const int kTileRows[4] = {256, 128, 32, 192}, kTileColumns[4] = {256, 128, 128, 128};

GemmPlan plan_forward(int64_t n, int glu, int64_t k, bool fp8, const Groups& g, bool grouped) {
    GemmPlan p;
    const int64_t per = grouped ? (g.total + g.groups - 1) / g.groups : g.total;
    const int64_t wide = n * (glu ? 2 : 1);
    const int64_t one_each = g.groups * ((wide + 127) / 128), room = (kRoundBlocks - one_each % kRoundBlocks) % kRoundBlocks;
    const bool some_longer = grouped && g.offset && !fp8 && per > 56 && g.total > 128 && room * 8 < one_each;
    auto tiles = [&](int t) { return worst_pieces(g, kTileRows[t], grouped) * ((wide + kTileColumns[t] - 1) / kTileColumns[t]); };
    p.tile = per > 128 && tiles(0) >= 200 ? 0 : some_longer ? 3 : grouped || per > 128 ? 1 : 2;
    p.splits = 1;
    p.ksplit = k;
    p.partial_bytes = 0;
    const int64_t t = tiles(p.tile);
    if (p.tile > 0) {
        const int bk = fp8 ? 128 : 64;
        const int64_t steps = (k + bk - 1) / bk;
        int64_t s = t > 0 ? kRoundBlocks / t : 1;
        if (s > steps / 4) s = steps / 4;
        if (s > 32) s = 32;
        if (s > 1) {
            const int64_t each = (steps + s - 1) / s;
            p.splits = (int)((steps + each - 1) / each);
            p.ksplit = each * bk;
            if (p.splits > 1) p.partial_bytes = (size_t)p.splits * g.total * ((n + 7) / 8 * 8 * (glu ? 2 : 1)) * 4;
        }
    }
    p.blocks = 2 * t * p.splits + 8;  // (FP8's 192 rows: at most 4/3 as many tiles)
    return p;
}

// Sums the pieces of a split reduction in order and applies the epilogue. A
// wave takes 256 columns of one row, 4 per lane: all its loads are independent
// and several are on their way at a time.
constexpr int kJoinRows = 4;

__device__ __forceinline__ float4_t join_pieces(const float* p, int64_t slice, int splits) {
    float4_t v = {0.f, 0.f, 0.f, 0.f};
    int s = 0;
    for (; s + 4 <= splits; s += 4) {
        float4_t x[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) x[u] = *reinterpret_cast<const float4_t*>(p + (s + u) * slice);
#pragma unroll
        for (int u = 0; u < 4; ++u) v += x[u];
    }
    for (; s < splits; ++s) v += *reinterpret_cast<const float4_t*>(p + s * slice);
    return v;
}

__global__ __launch_bounds__(256) void join_kernel(const GemmArgs a) {
    const Piece pc = find_piece<true>(a.g, kJoinRows, (int)blockIdx.x);
    if (pc.group < 0) return;
    const int r = threadIdx.x / kWave;
    const int64_t c = (int64_t)blockIdx.y * 256 + lane_id() * 4;
    if (c >= a.n || r >= pc.rows) return;
    const int have = (int)(a.n - c < 4 ? a.n - c : 4);
    const int64_t width = a.glu ? 2 * a.n : a.n;
    const int64_t np = (a.n + 7) / 8 * 8, pitch = a.glu ? 2 * np : np;  // a partial row, padded
    const int64_t slice = a.g.total * pitch, row = pc.row0 + r;
    const bool wide = (a.n & 3) == 0;
    float v[4], u[4] = {0.f, 0.f, 0.f, 0.f}, z[4];
    const float4_t sv = join_pieces(a.partial + row * pitch + c, slice, a.splits);
    float4_t su = {0.f, 0.f, 0.f, 0.f};
    if (a.glu) su = join_pieces(a.partial + row * pitch + np + c, slice, a.splits);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        v[q] = sv[q];
        u[q] = su[q];
    }
    if (a.bias) {
        const uint16_t* b = static_cast<const uint16_t*>(a.bias) + pc.group * width;
        load_run<4>(b + c, have, false, z);
#pragma unroll
        for (int q = 0; q < 4; ++q) v[q] += z[q];
        if (a.glu) {
            load_run<4>(b + a.n + c, have, false, z);
#pragma unroll
            for (int q = 0; q < 4; ++q) u[q] += z[q];
        }
    }
    if (a.preact) {
        store_run<4>(a.preact, row * width + c, v, have, false, wide);
        if (a.glu) store_run<4>(a.preact, row * width + a.n + c, u, have, false, wide);
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) v[q] = a.glu ? silu_f(v[q]) * u[q] : act_f(v[q], a.act);
    if (a.residual) {
        load_run<4>(static_cast<const uint16_t*>(a.residual) + row * a.n + c, have, wide, z);
#pragma unroll
        for (int q = 0; q < 4; ++q) v[q] += z[q];
    }
    store_run<4>(a.out, row * a.n + c, v, have, a.out_f32, wide);
}

hipError_t launch_join(const GemmArgs& a, bool grouped, hipStream_t stream) {
    const int64_t pieces = worst_pieces(a.g, kJoinRows, grouped);
    hipLaunchKernelGGL(join_kernel, dim3((unsigned)pieces, (unsigned)((a.n + 255) / 256)), dim3(256), 0, stream, a);
    return hipGetLastError();
}

hipError_t launch_forward_fp8(const GemmArgs& a, const GemmPlan& p, bool grouped, hipStream_t stream);

hipError_t launch_forward(const GemmArgs& in, const GemmPlan& p, bool fp8, bool grouped, hipStream_t stream) {
    GemmArgs a = in;
    a.splits = p.splits;
    a.ksplit = p.ksplit;
    hipError_t err;
    if (fp8)
        err = launch_forward_fp8(a, p, grouped, stream);
    else if (p.tile == 0)
        err = launch_gemm<256, 256, 2, 2, 0, 128, false, false, false>(a, grouped, stream);
    else if (p.tile == 1)
        err = launch_gemm<128, 128, 2, 2, 2, 128, false, false, false>(a, grouped, stream);
    else if (p.tile == 3)
        err = launch_gemm<192, 128, 2, 2, 2, 128, false, false, false>(a, grouped, stream);
    else
        err = launch_gemm<32, 128, 1, 4, 4, 128, false, false, false>(a, grouped, stream);
    if (err == hipSuccess && p.splits > 1) err = launch_join(a, grouped, stream);
    return err;
}

hipError_t preload_gemm() {
    hipFuncAttributes at;
    return hipFuncGetAttributes(&at, reinterpret_cast<const void*>(&join_kernel));
}

}  // namespace cgd
