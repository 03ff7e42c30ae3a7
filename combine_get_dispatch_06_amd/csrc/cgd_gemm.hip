// Forward products in bf16, the choice of tiles, and the kernel that joins a
// split reduction.
#include "cgd_gemm_launch.h"

namespace cgd {

// Tile by rows per group (grouped products see the average) and by how many
// tiles there are:
//   256 x 256 once it gives most CUs a tile; 128 x 128 below that; 64 and 32
//   rows where a group has fewer (what is read then is the weights, and a
//   taller tile would only multiply by zeros).
// A reduction is split where even so most CUs had no tile.
GemmPlan plan_forward(int64_t n, int glu, int64_t k, bool fp8, const Groups& g, bool grouped) {
    GemmPlan p;
    const int64_t per = grouped ? (g.total + g.groups - 1) / g.groups : g.total;
    const int64_t wide = n * (glu ? 2 : 1);
    auto tiles = [&](int bm, int bn) { return worst_pieces(g, bm, grouped) * ((wide + bn - 1) / bn); };
    if (per > 128 && tiles(256, 256) >= 200)
        p.tile = 0;
    else if (per > 64)
        p.tile = 1;
    else if (per > 32)
        p.tile = 2;
    else
        p.tile = 3;
    p.splits = 1;
    p.ksplit = k;
    p.partial_bytes = 0;
    p.blocks = tiles(256, 256);
    if (p.tile > 0) {
        const int bk = fp8 ? 128 : 64;
        const int64_t t = p.blocks = tiles(p.tile == 1 ? 128 : p.tile == 2 ? 64 : 32, 128);
        const int64_t steps = (k + bk - 1) / bk;
        int64_t s = t > 0 ? 512 / t : 1;
        if (s > steps / 4) s = steps / 4;
        if (s > 32) s = 32;
        if (s > 1) {
            const int64_t each = (steps + s - 1) / s;
            p.splits = (int)((steps + each - 1) / each);
            p.ksplit = each * bk;
            if (p.splits > 1) p.partial_bytes = (size_t)p.splits * g.total * wide * 4;
        }
    }
    p.blocks = p.blocks * p.splits + 8;
    return p;
}

// Sums the pieces of a split reduction in order and applies the epilogue. A
// block takes 8 rows of one group (dense: of the batch) and 256 columns.
constexpr int kJoinRows = 8;
__global__ __launch_bounds__(256) void join_kernel(const GemmArgs a) {
    const Piece pc = find_piece<true>(a.g, kJoinRows, (int)blockIdx.x);
    if (pc.group < 0) return;
    const int64_t c = (int64_t)blockIdx.y * 256 + threadIdx.x;
    if (c >= a.n) return;
    const int64_t wide = a.glu ? 2 * a.n : a.n;
    const int64_t slice = a.g.total * wide;
    const int rows = pc.rows < kJoinRows ? (int)pc.rows : kJoinRows;
    const uint16_t* b = static_cast<const uint16_t*>(a.bias);
    const float bias0 = b ? bf16_at(b + pc.group * wide + c) : 0.0f;
    const float bias1 = b && a.glu ? bf16_at(b + pc.group * wide + a.n + c) : 0.0f;
    for (int i = 0; i < rows; ++i) {
        const int64_t row = pc.row0 + i;
        const float* p = a.partial + row * wide + c;
        float v = 0.0f, u = 0.0f;
        for (int s = 0; s < a.splits; ++s) {
            v += p[s * slice];
            if (a.glu) u += p[s * slice + a.n];
        }
        v += bias0;
        u += bias1;
        if (a.preact) {
            uint16_t* z = static_cast<uint16_t*>(a.preact) + row * wide;
            z[c] = (uint16_t)pack_bf16x2(v, 0.0f);
            if (a.glu) z[a.n + c] = (uint16_t)pack_bf16x2(u, 0.0f);
        }
        v = a.glu ? silu_f(v) * u : act_f(v, a.act);
        if (a.residual) v += bf16_at(static_cast<const uint16_t*>(a.residual) + row * a.n + c);
        if (a.out_f32)
            static_cast<float*>(a.out)[row * a.n + c] = v;
        else
            static_cast<uint16_t*>(a.out)[row * a.n + c] = (uint16_t)pack_bf16x2(v, 0.0f);
    }
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
    else if (p.tile == 2)
        err = launch_gemm<64, 128, 1, 4, 3, 128, false, false, false>(a, grouped, stream);
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
