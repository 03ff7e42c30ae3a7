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

int64_t grad_blocks(const Groups& g, bool grouped, int64_t width, int64_t k) {
    const int ti = input_tile(g, grouped, k), tw = weight_tile(g, width, k);
    const int bm = ti == 0 ? 256 : 128, bn = bm, bw = tw == 0 ? 256 : 128;
    const int64_t bi = worst_pieces(g, bm, grouped) * ((k + bn - 1) / bn);
    const int64_t w = (int64_t)g.groups * ((width + bw - 1) / bw) * ((k + bw - 1) / bw);
    return (bi > w ? bi : w) + 8;
}

hipError_t launch_input_grad(const GemmArgs& a, bool grouped, hipStream_t stream) {
    if (input_tile(a.g, grouped, a.n) == 0) return launch_gemm<256, 256, 2, 2, 0, 128, false, true, false>(a, grouped, stream);
    return launch_gemm<128, 128, 2, 2, 5, 64, false, true, false>(a, grouped, stream);
}

hipError_t launch_weight_grad(const GemmArgs& a, hipStream_t stream) {
    if (weight_tile(a.g, a.m, a.n) == 0) return launch_gemm<256, 256, 2, 2, 0, 128, true, true, false>(a, true, stream);
    return launch_gemm<128, 128, 2, 2, 5, 64, true, true, false>(a, true, stream);
}

hipError_t preload_gemm_grad() {
    hipFuncAttributes at;
    return hipFuncGetAttributes(&at, reinterpret_cast<const void*>(&gemm_kernel<128, 128, 2, 2, 5, 64, true, true, false>));
}

}  // namespace cgd
