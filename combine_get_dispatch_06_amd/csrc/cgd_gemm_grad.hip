// Gradients of the products.
//   grad_x[m, i]    = sum_o d[m, o] * W[o, i]   (W read transposed)
//   grad_W[e][o, i] = sum over e's rows m of d[m, o] * x[m, i]   (both read transposed)
// A group without rows has zero gradients, which are written.
#include "cgd_gemm_launch.h"

namespace cgd {

// 256 x 256 tiles once they give most CUs one, smaller ones below that.
static int input_tile(const Groups& g, bool grouped, int64_t k) {
    const int64_t per = grouped ? (g.total + g.groups - 1) / g.groups : g.total;
    return per > 128 && worst_pieces(g, 256, grouped) * ((k + 255) / 256) >= 200 ? 0 : 1;
}
static int weight_tile(const Groups& g, int64_t width, int64_t k) {
    return (int64_t)g.groups * ((width + 255) / 256) * ((k + 255) / 256) >= 200 ? 0 : 1;
}

// A group's rows are split while there were fewer than 512 blocks, into pieces
// of at least 8 stages of 64 rows, and of a quarter as many stages as there are
// tiles: with many tiles the pieces' sums cost more than the idle CUs. Both
// gradients, without and with two pieces and more: 32768 x 256 x 7168 564 -> 462 us,
// 4000 x 512 x 1024 47 -> 31, 16384 x 2048 x 2048 282 -> 276, but 4096 x 2048 x 2048
// 88 -> 95 (left whole).
int weight_grad_splits(const Groups& g, int64_t width, int64_t k) {
    if (weight_tile(g, width, k) == 0) return 1;
    const int64_t tiles = (int64_t)g.groups * ((width + 127) / 128) * ((k + 127) / 128), stages = g.total / g.groups / 64;
    const int64_t least = tiles / 4 > 8 ? tiles / 4 : 8;
    int64_t s = 512 / tiles;
    if (s > stages / least) s = stages / least;
    return s < 1 ? 1 : s > 32 ? 32 : (int)s;
}

int64_t grad_blocks(const Groups& g, bool grouped, int64_t width, int64_t k) {
    const int ti = input_tile(g, grouped, k), tw = weight_tile(g, width, k);
    const int bm = ti == 0 ? 256 : 128, bn = bm, bw = tw == 0 ? 256 : 128;
    const int64_t bi = worst_pieces(g, bm, grouped) * ((k + bn - 1) / bn);
    const int64_t w = (int64_t)g.groups * weight_grad_splits(g, width, k) * ((width + bw - 1) / bw) * ((k + bw - 1) / bw);
    return (bi > w ? bi : w) + 8;
}

hipError_t launch_input_grad(const GemmArgs& a, bool grouped, hipStream_t stream) {
    if (input_tile(a.g, grouped, a.n) == 0) return launch_gemm<256, 256, 2, 2, 0, 128, false, true, false>(a, grouped, stream);
    return launch_gemm<128, 128, 2, 2, 5, 64, false, true, false>(a, grouped, stream);
}

hipError_t launch_weight_grad(const GemmArgs& a, hipStream_t stream) {
    if (weight_tile(a.g, a.m, a.n) == 0) return launch_gemm<256, 256, 2, 2, 0, 128, true, true, false>(a, true, stream);
    const hipError_t err = launch_gemm<128, 128, 2, 2, 5, 64, true, true, false>(a, true, stream);
    if (err != hipSuccess || a.splits == 1) return err;
    GemmArgs j = a;  // the gradient's rows as those of one dense product
    j.g = Groups{nullptr, nullptr, 0, a.g.groups * a.m, 1};
    return launch_join(j, false, stream);
}

hipError_t preload_gemm_grad() {
    hipFuncAttributes at;
    return hipFuncGetAttributes(&at, reinterpret_cast<const void*>(&gemm_kernel<128, 128, 2, 2, 5, 64, true, true, false>));
}

}  // namespace cgd
