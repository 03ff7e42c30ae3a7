// Dropout from a counter-based generator; the mask is never stored.
//   out[i] = (u[i] >= limit ? x[i] * scale : 0) + residual[i]
// u: 16 bits for each element from Philox4x32-10 (J. Salmon, M. Moraes, R. Dror,
// D. Shaw, "Parallel random numbers: as easy as 1, 2, 3", 2011) under the key
// `seed`; elements 8 v to 8 v + 7 have the counter (v, offset), two to a word,
// the low half first. limit = round(p * 65536): 16 bits an element cost one
// generator call for one 16-byte vector, and scale = 65536 / (65536 - limit)
// belongs to the probability that is used, so the expectation is exact.
// A dropped element is 0 whatever it held, infinities and NaN included.
// The gradient is the same call on the gradient.
// Memory-bound: 4096 x 7168 with a residual 29 us (6.0 TB/s) with non-temporal loads, 33
// without; stores are ordinary ones (non-temporal 29, too): what comes next reads them.
// The generator's 20 wide multiplications a vector fit beside the loads (one vector
// a thread, or four: 1 us more).
#include "cgd_device.h"
#include "cgd_layer_launch.h"

namespace cgd {

namespace {

constexpr int kDropThreads = 256, kDropVectors = 2;  // vectors of a thread

__device__ __forceinline__ uint4 philox(uint64_t index, uint64_t offset, uint64_t seed) {
    uint32_t c0 = (uint32_t)index, c1 = (uint32_t)(index >> 32), c2 = (uint32_t)offset, c3 = (uint32_t)(offset >> 32);
    uint32_t k0 = (uint32_t)seed, k1 = (uint32_t)(seed >> 32);
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t p = (uint64_t)c0 * 0xD2511F53u, q = (uint64_t)c2 * 0xCD9E8D57u;
        c0 = (uint32_t)(q >> 32) ^ c1 ^ k0;
        c2 = (uint32_t)(p >> 32) ^ c3 ^ k1;
        c1 = (uint32_t)q;
        c3 = (uint32_t)p;
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return make_uint4(c0, c1, c2, c3);
}

// Two elements of a word.
__device__ __forceinline__ uint32_t drop2(uint32_t x, uint32_t u, uint32_t r, bool add, uint32_t limit, float scale) {
    float lo = (u & 0xFFFFu) >= limit ? bf16_lo(x) * scale : 0.0f;
    float hi = (u >> 16) >= limit ? bf16_hi(x) * scale : 0.0f;
    if (add) {
        lo += bf16_lo(r);
        hi += bf16_hi(r);
    }
    return pack_bf16x2(lo, hi);
}

// U vectors a thread; vector `first` + i of the tensor is vector i here.
// FAR: more than the Infinity Cache keeps, so the inputs are not worth a place there.
constexpr int64_t kFarBytes = int64_t(160) << 20;
template <int U, bool FAR>
__global__ __launch_bounds__(kDropThreads) void dropout_kernel(const DropoutArgs a, int64_t first) {
    uint64_t seed = a.seed, offset = a.offset;
    if (a.state) {
        seed += (uint64_t)a.state[0];
        offset += (uint64_t)a.state[1];
    }
    const int64_t whole = a.n / 8, vectors = (a.n + 7) / 8;
    const int64_t v0 = first + (int64_t)blockIdx.x * (kDropThreads * U) + threadIdx.x;
    uint4 x[U], r[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t v = v0 + u * kDropThreads;
        x[u] = r[u] = make_uint4(0, 0, 0, 0);
        if (v < whole) {
            const uint4* xv = reinterpret_cast<const uint4*>(a.x) + v;
            const uint4* rv = reinterpret_cast<const uint4*>(a.residual) + v;
            x[u] = FAR ? load_nt(xv) : *xv;
            if (a.residual) r[u] = FAR ? load_nt(rv) : *rv;
        }
    }
    const bool add = a.residual != nullptr;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t v = v0 + u * kDropThreads;
        if (v >= vectors) return;
        const uint4 z = philox((uint64_t)v, offset, seed);
        if (v < whole) {
            uint4 o;
            o.x = drop2(x[u].x, z.x, r[u].x, add, a.limit, a.scale);
            o.y = drop2(x[u].y, z.y, r[u].y, add, a.limit, a.scale);
            o.z = drop2(x[u].z, z.z, r[u].z, add, a.limit, a.scale);
            o.w = drop2(x[u].w, z.w, r[u].w, add, a.limit, a.scale);
            reinterpret_cast<uint4*>(a.out)[v] = o;
        } else {  // the last vector's part
            const uint32_t w[4] = {z.x, z.y, z.z, z.w};
            const int have = (int)(a.n - 8 * v);
#pragma unroll
            for (int i = 0; i < 7; ++i) {
                if (i >= have) break;
                const uint32_t one = a.x[8 * v + i], res = add ? a.residual[8 * v + i] : 0u;
                a.out[8 * v + i] = (uint16_t)drop2(one, w[i / 2] >> (16 * (i & 1)) & 0xFFFFu, res, add, a.limit, a.scale);
            }
        }
    }
}

}  // namespace

hipError_t launch_dropout(const DropoutArgs& a, hipStream_t stream) {
    constexpr int U = kDropVectors;
    if (a.n == 0) return hipSuccess;
    const int64_t vectors = (a.n + 7) / 8, most = kMaxWorkItems * U;
    for (int64_t v = 0; v < vectors; v += most) {
        const int64_t n = vectors - v < most ? vectors - v : most;
        const int64_t blocks = (n + kDropThreads * U - 1) / (kDropThreads * U);
        if (a.n * (a.residual ? 6 : 4) > kFarBytes)
            hipLaunchKernelGGL((dropout_kernel<U, true>), dim3((unsigned)blocks), dim3(kDropThreads), 0, stream, a, v);
        else
            hipLaunchKernelGGL((dropout_kernel<U, false>), dim3((unsigned)blocks), dim3(kDropThreads), 0, stream, a, v);
    }
    return hipGetLastError();
}

hipError_t preload_dropout() {
    hipFuncAttributes at;
    return hipFuncGetAttributes(&at, reinterpret_cast<const void*>(&dropout_kernel<kDropVectors, false>));
}

}  // namespace cgd
