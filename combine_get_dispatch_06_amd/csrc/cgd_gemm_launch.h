// Launches of the tiled products.
#pragma once

#include "cgd_gemm.h"

namespace cgd {

// Pieces of bm rows that the groups can have at most, whatever their sizes.
inline int64_t worst_pieces(const Groups& g, int bm, bool grouped) {
    if (!grouped) return (g.total + bm - 1) / bm;
    if (!g.offset) return (int64_t)g.groups * ((g.capacity + bm - 1) / bm);
    return g.total / bm + (g.groups < g.total ? g.groups : g.total);
}

template <int BM, int BN, int WM, int WN, int ST, int RB, bool QT, bool PT, bool FP8>
hipError_t launch_gemm(const GemmArgs& a, bool grouped, hipStream_t stream) {
    const int64_t half = a.glu ? BN / 2 : BN;
    const int64_t tn = (a.n + half - 1) / half;
    const int64_t tm = QT ? (int64_t)a.g.groups * ((a.m + BM - 1) / BM) : worst_pieces(a.g, BM, grouped);
    int64_t blocks = (tm * tn * a.splits + 7) / 8 * 8;  // 8 runs of tiles, one for each XCD
    // tiles with a CU to themselves: one block for each of the 256 CUs takes them in turn
    if ((ST == 0 || BM * BN > 192 * 128) && blocks > 256) blocks = 256;
    if (blocks == 0) return hipSuccess;
    hipLaunchKernelGGL((gemm_kernel<BM, BN, WM, WN, ST, RB, QT, PT, FP8>), dim3((unsigned)blocks), dim3(WM * WN * kWave), 0,
                       stream, a);
    return hipGetLastError();
}

}  // namespace cgd
