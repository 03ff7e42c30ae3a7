// Low-rank adapters of many requests in one batch, and their gradients.
//   h[t] = a[j] x[t],  out[t] = residual[t] + scale[j] b[j] h[t],  j = index[t]
//   gh[t] = scale[j] b[j]^T grad[t],  grad_x[t] = a[j]^T gh[t]
//   grad_a[j] = sum over j's tokens of gh x^T,  grad_b[j] = sum of scale grad h^T
// Tokens are put in order of their adapter first (a stable order: sums do not
// depend on timing), those without one last; tiles of 16 tokens and up then
// have one adapter each, and rows are gathered through that order. The products
// are skinny, a rank is some 8 to 256: what bounds them is reading x and writing
// out once, so operands go from memory straight into the registers of the matrix
// instructions, 16 bytes a lane, without LDS in between, and the reduction over
// in_features is split until the CUs are busy.
// h and gh are fp32 sums; as operands of the second product they go in as two
// bf16 parts (v = hi + lo, off by 2^-16 of v at most), which costs matrix
// instructions that nothing waits for: results are rounded once.
#include "cgd_gemm_launch.h"
#include "cgd_layer_launch.h"

namespace cgd {

namespace {

typedef uint32_t uint4_t __attribute__((ext_vector_type(4)));

__device__ __forceinline__ bf16x8_t frag_at(const uint16_t* p) { return *reinterpret_cast<const bf16x8_t*>(p); }
__device__ __forceinline__ bf16x8_t no_frag() { return __builtin_bit_cast(bf16x8_t, uint4_t{0, 0, 0, 0}); }
__device__ __forceinline__ float4_t mul16(const bf16x8_t& rows, const bf16x8_t& columns, const float4_t& sum) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(rows, columns, sum, 0, 0, 0);
}

// v = hi + lo in bf16 pairs: of two values.
__device__ __forceinline__ void halves2(float a, float b, uint32_t* hi, uint32_t* lo) {
    const uint32_t h = pack_bf16x2(a, b);
    // what is infinite or NaN already has no second part
    const float da = fabsf(a) < __builtin_inff() ? a - bf16_lo(h) : 0.0f;
    const float db = fabsf(b) < __builtin_inff() ? b - bf16_hi(h) : 0.0f;
    *hi = h;
    *lo = pack_bf16x2(da, db);
}

// ---- order of the tokens ---------------------------------------------------

constexpr int kPlanThreads = 1024;
constexpr int kPlanWaves = kPlanThreads / kWave;

// Block g finds the tokens of adapter g (g = adapters: those without one): how
// many come before them, and in a second pass their places. No block waits for
// another. Each wave has a run of tokens, so the order within a group is the
// tokens' own.
__global__ __launch_bounds__(kPlanThreads) void adapter_plan_kernel(const int64_t* __restrict__ index, int tokens, int adapters,
                                                                    int32_t* __restrict__ offset, int32_t* __restrict__ order) {
    __shared__ int32_t less_of[kPlanWaves], same_of[kPlanWaves];
    const int mine = blockIdx.x, lane = lane_id(), wave = threadIdx.x / kWave;
    const int run = (tokens + kPlanThreads - 1) / kPlanThreads * kWave;
    const int t0 = wave * run, t1 = t0 + run < tokens ? t0 + run : tokens;
    auto group = [&](int t) {
        const int64_t j = index[t];
        return j >= 0 && j < adapters ? (int)j : adapters;
    };
    int less = 0, same = 0;
    for (int t = t0 + lane; t < t1; t += 4 * kWave) {
        int g[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) g[u] = t + u * kWave < t1 ? group(t + u * kWave) : INT32_MAX;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            less += g[u] < mine;
            same += g[u] == mine;
        }
    }
#pragma unroll
    for (int d = 32; d; d >>= 1) {
        less += __shfl_xor(less, d, kWave);
        same += __shfl_xor(same, d, kWave);
    }
    if (lane == 0) {
        less_of[wave] = less;
        same_of[wave] = same;
    }
    __syncthreads();
    int first = 0, at = 0;
    for (int w = 0; w < kPlanWaves; ++w) {
        first += less_of[w];
        at += w < wave ? same_of[w] : 0;
    }
    at += first;
    if (threadIdx.x == 0) {
        offset[mine] = first;
        if (mine == adapters) offset[mine + 1] = tokens;
    }
    if (same == 0) return;
    for (int t = t0; t < t1; t += kWave) {
        const bool hit = t + lane < t1 && group(t + lane) == mine;
        const uint64_t hits = ballot(hit);
        if (hit) order[at + __popcll(hits & lanemask_lt())] = t + lane;
        at += __popcll(hits);
    }
}

// ---- the first product: to the rank ------------------------------------------

struct ShrinkArgs {
    const uint16_t* x;       // [tokens, in]
    const uint16_t* w;       // [adapters, rank, in]
    const int32_t* offset;   // [adapters + 2]
    const int32_t* order;
    int64_t tokens, in, piece;  // piece: of `in` for one block, a multiple of 64
    int adapters, rank;
    float* partial;          // [pieces][token in order][rank]
};

// A block has 16 * MT tokens of one adapter and 16 * NT of the ranks over one
// piece of the reduction; its four waves take 64 of it in turn (128 bytes of a
// row at a time) and join their sums through LDS.
template <int MT, int NT>
__global__ __launch_bounds__(256) void adapter_shrink_kernel(const ShrinkArgs s) {
    constexpr int BM = 16 * MT, BN = 16 * NT, PITCH = BN + 4;
    __shared__ __attribute__((aligned(16))) float sums[4][BM][PITCH];
    const Groups groups{s.offset, nullptr, 0, s.tokens, s.adapters};
    const Piece pc = find_piece<true>(groups, BM, (int)blockIdx.x);
    if (pc.group < 0) return;
    const int lane = lane_id(), wave = threadIdx.x / kWave, m = lane & 15, g = lane >> 4;
    const int rows = pc.rows < BM ? (int)pc.rows : BM;
    const int rank0 = blockIdx.z * BN;
    const int64_t k0 = blockIdx.y * s.piece, k1 = k0 + s.piece < s.in ? k0 + s.piece : s.in;
    // rows past the tile's tokens, or past the rank, repeat the last: nothing of them is stored
    const uint16_t* xp[MT];
    const uint16_t* wp[NT];
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        const int r = i * 16 + m < rows ? i * 16 + m : rows - 1;
        xp[i] = s.x + s.order[pc.row0 + r] * s.in + g * 8;
    }
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        const int r = rank0 + j * 16 + m < s.rank ? rank0 + j * 16 + m : s.rank - 1;
        wp[j] = s.w + ((int64_t)pc.group * s.rank + r) * s.in + g * 8;
    }
    float4_t acc[MT][NT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j] = float4_t{0.f, 0.f, 0.f, 0.f};
    constexpr int U = MT * NT > 4 ? 2 : 4;  // units of 64 on their way at a time
    const int whole = (int)((k1 - k0) / 64), units = (int)((k1 - k0 + 63) / 64);
    int u = wave;
    for (; u + 4 * (U - 1) < whole; u += 4 * U) {
        bf16x8_t xf[U][2][MT], wf[U][2][NT];
#pragma unroll
        for (int v = 0; v < U; ++v)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int64_t k = k0 + (u + 4 * v) * 64 + h * 32;
#pragma unroll
                for (int i = 0; i < MT; ++i) xf[v][h][i] = frag_at(xp[i] + k);
#pragma unroll
                for (int j = 0; j < NT; ++j) wf[v][h][j] = frag_at(wp[j] + k);
            }
#pragma unroll
        for (int v = 0; v < U; ++v)
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                    for (int j = 0; j < NT; ++j) acc[i][j] = mul16(wf[v][h][j], xf[v][h][i], acc[i][j]);
    }
    for (; u < units; u += 4) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int64_t k = k0 + u * 64 + h * 32;
            const bool in = k + g * 8 < k1;
            bf16x8_t xf[MT], wf[NT];
#pragma unroll
            for (int i = 0; i < MT; ++i) xf[i] = in ? frag_at(xp[i] + k) : no_frag();
#pragma unroll
            for (int j = 0; j < NT; ++j) wf[j] = in ? frag_at(wp[j] + k) : no_frag();
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int j = 0; j < NT; ++j) acc[i][j] = mul16(wf[j], xf[i], acc[i][j]);
        }
    }
    // a lane has four consecutive ranks of one token
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) *reinterpret_cast<float4_t*>(&sums[wave][i * 16 + m][j * 16 + g * 4]) = acc[i][j];
    __syncthreads();
    float* out = s.partial + ((int64_t)blockIdx.y * s.tokens + pc.row0) * s.rank;
    for (int i = threadIdx.x; i < BM * NT * 4; i += 256) {
        const int r = i / (NT * 4), c = i % (NT * 4) * 4;
        if (r >= rows || rank0 + c >= s.rank) continue;
        float4_t v = *reinterpret_cast<const float4_t*>(&sums[0][r][c]);
#pragma unroll
        for (int w = 1; w < 4; ++w) v += *reinterpret_cast<const float4_t*>(&sums[w][r][c]);
        *reinterpret_cast<float4_t*>(out + (int64_t)r * s.rank + rank0 + c) = v;
    }
}

// ---- the second product: from the rank ----------------------------------------

struct ExpandArgs {
    const float* partial;    // [pieces][token in order][rank]
    int pieces;
    const uint16_t* w;       // [adapters, out, rank]
    const float* scale;      // [adapters] or null
    const int32_t* offset;
    const int32_t* order;
    int64_t tokens, width, chunk;  // chunk: of the out features for one block, a multiple of 256
    int adapters, rank;
    const uint16_t* residual;
    uint16_t* out;           // [tokens, width], or null
    float* hidden;           // joined sums [token][rank], or null
    float* scaled;           // joined sums times the scale [token in order][rank], or null
};

// A block has 16 * NT tokens of one adapter (or of none) and `chunk` out
// features. Its waves take 64 features at a time: the tile's rows are ordered
// so that a lane ends up with 16 consecutive features of a token, and the four
// lanes of a token with a whole 128-byte line.
template <int NT>
__global__ __launch_bounds__(256) void adapter_expand_kernel(const ExpandArgs e) {
    constexpr int BM = 16 * NT;
    extern __shared__ __attribute__((aligned(16))) uint16_t parts[];  // [hi, lo][token][pitch]
    const int pitch = e.rank + 8;
    const Groups groups{e.offset, nullptr, 0, e.tokens, e.adapters + 1};
    const Piece pc = find_piece<true>(groups, BM, (int)blockIdx.x);
    if (pc.group < 0) return;
    const int lane = lane_id(), wave = threadIdx.x / kWave, n = lane & 15, g = lane >> 4;
    const int rows = pc.rows < BM ? (int)pc.rows : BM;
    const bool none = pc.group == e.adapters;
    const float scale = none || !e.scale ? 1.0f : e.scale[pc.group];
    const int quads = e.rank / 4;
    for (int i = threadIdx.x; i < BM * quads; i += 256) {
        const int r = i / quads, c = (i - r * quads) * 4;
        float4_t v = {0.f, 0.f, 0.f, 0.f};
        if (r < rows && !none) v = join_pieces(e.partial + (pc.row0 + r) * e.rank + c, e.tokens * e.rank, e.pieces);
        if (r < rows && blockIdx.y == 0) {
            if (e.hidden) *reinterpret_cast<float4_t*>(e.hidden + (int64_t)e.order[pc.row0 + r] * e.rank + c) = v;
            if (e.scaled) *reinterpret_cast<float4_t*>(e.scaled + (pc.row0 + r) * e.rank + c) = v * scale;
        }
        v *= scale;
        uint2 hi, lo;
        halves2(v[0], v[1], &hi.x, &lo.x);
        halves2(v[2], v[3], &hi.y, &lo.y);
        *reinterpret_cast<uint2*>(parts + r * pitch + c) = hi;
        *reinterpret_cast<uint2*>(parts + (BM + r) * pitch + c) = lo;
    }
    if (!e.out) return;
    __syncthreads();
    int64_t token[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) token[t] = t * 16 + n < rows ? e.order[pc.row0 + t * 16 + n] : -1;
    const bool whole = e.width % 8 == 0, dual = e.rank % 32 == 0;
    const int eighths = e.rank / 8;  // 16-byte pieces of a row of w
    const int64_t end = (int64_t)(blockIdx.y + 1) * e.chunk < e.width ? (int64_t)(blockIdx.y + 1) * e.chunk : e.width;
    for (int64_t o0 = blockIdx.y * e.chunk + wave * 64; o0 < end; o0 += 256) {
        float4_t acc[4][NT];
#pragma unroll
        for (int p = 0; p < 4; ++p)
#pragma unroll
            for (int t = 0; t < NT; ++t) acc[p][t] = float4_t{0.f, 0.f, 0.f, 0.f};
        if (!none) {
            const uint16_t* wp[4];
#pragma unroll
            for (int p = 0; p < 4; ++p) {  // row n of tile p is feature (n / 4) * 16 + p * 4 + n % 4
                const int64_t o = o0 + (n >> 2) * 16 + p * 4 + (n & 3);
                wp[p] = e.w + ((int64_t)pc.group * e.width + (o < e.width ? o : e.width - 1)) * e.rank;
            }
            if (dual) {
                for (int k = 0; k < e.rank; k += 32) {
                    bf16x8_t wf[4];
#pragma unroll
                    for (int p = 0; p < 4; ++p) wf[p] = frag_at(wp[p] + k + g * 8);
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        const bf16x8_t hi = frag_at(parts + (t * 16 + n) * pitch + k + g * 8);
                        const bf16x8_t lo = frag_at(parts + (BM + t * 16 + n) * pitch + k + g * 8);
#pragma unroll
                        for (int p = 0; p < 4; ++p) acc[p][t] = mul16(wf[p], lo, mul16(wf[p], hi, acc[p][t]));
                    }
                }
            } else {  // the two parts one after the other along the reduction: a row of w twice
                for (int k = 0; k < 2 * eighths; k += 4) {
                    const int piece = k + g, part = piece >= eighths;
                    const int at = piece - part * eighths;
                    const bool in = piece < 2 * eighths;
                    bf16x8_t wf[4];
#pragma unroll
                    for (int p = 0; p < 4; ++p) wf[p] = in ? frag_at(wp[p] + at * 8) : no_frag();
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        const bf16x8_t h = in ? frag_at(parts + (part * BM + t * 16 + n) * pitch + at * 8) : no_frag();
#pragma unroll
                        for (int p = 0; p < 4; ++p) acc[p][t] = mul16(wf[p], h, acc[p][t]);
                    }
                }
            }
        }
        const int64_t o = o0 + g * 16;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            if (token[t] < 0 || o >= e.width) continue;
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const int have = (int)(e.width - o - q * 8 < 8 ? e.width - o - q * 8 : 8);
                if (have <= 0) continue;
                float v[8] = {acc[2 * q][t][0], acc[2 * q][t][1], acc[2 * q][t][2], acc[2 * q][t][3],
                              acc[2 * q + 1][t][0], acc[2 * q + 1][t][1], acc[2 * q + 1][t][2], acc[2 * q + 1][t][3]};
                const int64_t at = token[t] * e.width + o + q * 8;
                if (e.residual) {
                    float r[8];
                    load_run<8>(e.residual + at, have, whole, r);
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[i] += r[i];
                }
                store_run<8>(e.out, at, v, have, false, whole);
            }
        }
    }
}

// ---- the adapters' own gradients -----------------------------------------------

struct AdapterWeightArgs {
    const uint16_t* x;      // [tokens, in]
    const uint16_t* grad;   // [tokens, out]
    const float* scaled;    // gh [token in order][rank]
    const float* hidden;    // [token][rank]
    const float* scale;
    const int32_t* offset;
    const int32_t* order;
    int64_t in, out;
    int adapters, rank;
    int a_blocks;           // column blocks of grad_a; those of grad_b follow
    uint16_t* grad_a;
    uint16_t* grad_b;
};

// A block has 128 columns (of x for grad_a, of grad for grad_b) and 16 * RT
// ranks of one adapter; its NW waves take 32 of the adapter's tokens in turn and
// join their sums through LDS in a fixed order. The wide operand is needed with
// eight tokens of one column in a lane: a lane loads eight columns of eight
// tokens, 16 bytes each, and turns that square over in its own registers; the
// eight matrix tiles it makes have every eighth column each.
template <int RT, int NW>
__global__ __launch_bounds__(NW* kWave) void adapter_weight_kernel(const AdapterWeightArgs w) {
    extern __shared__ __attribute__((aligned(16))) float4_t joined[];  // [wave][RT * 8][lane]
    const int lane = lane_id(), wave = threadIdx.x / kWave, n = lane & 15, g = lane >> 4;
    const bool is_a = (int)blockIdx.x < w.a_blocks;
    const int64_t width = is_a ? w.in : w.out;
    const int64_t col = (int64_t)(is_a ? blockIdx.x : blockIdx.x - w.a_blocks) * 128 + n * 8;
    const uint16_t* wide = is_a ? w.x : w.grad;
    const float* thin = is_a ? w.scaled : w.hidden;
    const int j = blockIdx.y, rank0 = blockIdx.z * 16 * RT;
    const int begin = w.offset[j], end = w.offset[j + 1];
    const float scale = !is_a && w.scale ? w.scale[j] : 1.0f;
    float4_t acc[RT][8];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int c = 0; c < 8; ++c) acc[r][c] = float4_t{0.f, 0.f, 0.f, 0.f};
    for (int p0 = begin + wave * 32; p0 < end; p0 += NW * 32) {
        const int p = p0 + g * 8;
        uint4 row[8];
        int token[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) token[i] = p + i < end ? w.order[p + i] : -1;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            row[i] = token[i] >= 0 && col < width ? *reinterpret_cast<const uint4*>(wide + token[i] * width + col) : make_uint4(0, 0, 0, 0);
        bf16x8_t hi[RT], lo[RT];
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            const int k = rank0 + r * 16 + n;
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int64_t at = is_a ? p + i : token[i];
                v[i] = token[i] >= 0 && k < w.rank ? thin[at * w.rank + k] * scale : 0.0f;
            }
            uint32_t h[4], l[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) halves2(v[2 * i], v[2 * i + 1], &h[i], &l[i]);
            hi[r] = __builtin_bit_cast(bf16x8_t, uint4_t{h[0], h[1], h[2], h[3]});
            lo[r] = __builtin_bit_cast(bf16x8_t, uint4_t{l[0], l[1], l[2], l[3]});
        }
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            uint32_t q[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t a = reinterpret_cast<const uint32_t*>(&row[2 * i])[c / 2], b = reinterpret_cast<const uint32_t*>(&row[2 * i + 1])[c / 2];
                q[i] = c & 1 ? (a >> 16) | (b & 0xFFFF0000u) : (a & 0xFFFFu) | (b << 16);
            }
            const bf16x8_t f = __builtin_bit_cast(bf16x8_t, uint4_t{q[0], q[1], q[2], q[3]});
#pragma unroll
            for (int r = 0; r < RT; ++r) acc[r][c] = mul16(lo[r], f, mul16(hi[r], f, acc[r][c]));
        }
    }
    // the upper half of the waves that had tokens gives its sums to the lower, until one has them
    const int most = (end - begin + 31) / 32;
    for (int half = NW / 2; half; half /= 2) {
        if (half >= most) continue;
        __syncthreads();
        if (wave >= half && wave < 2 * half)
#pragma unroll
            for (int r = 0; r < RT; ++r)
#pragma unroll
                for (int c = 0; c < 8; ++c) joined[((wave - half) * RT * 8 + r * 8 + c) * kWave + lane] = acc[r][c];
        __syncthreads();
        if (wave < half)
#pragma unroll
            for (int r = 0; r < RT; ++r)
#pragma unroll
                for (int c = 0; c < 8; ++c) acc[r][c] += joined[(wave * RT * 8 + r * 8 + c) * kWave + lane];
    }
    if (wave || col >= width) return;
#pragma unroll
    for (int r = 0; r < RT; ++r) {
        const int k = rank0 + r * 16 + g * 4;
        if (k >= w.rank) continue;
        if (is_a) {  // [rank][in]: eight columns of four ranks
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float v[8] = {acc[r][0][i], acc[r][1][i], acc[r][2][i], acc[r][3][i], acc[r][4][i], acc[r][5][i], acc[r][6][i], acc[r][7][i]};
                store_run<8>(w.grad_a, ((int64_t)j * w.rank + k + i) * w.in + col, v, 8, false, true);
            }
        } else {  // [out][rank]: four ranks of eight columns
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                const float v[4] = {acc[r][c][0], acc[r][c][1], acc[r][c][2], acc[r][c][3]};
                store_run<4>(w.grad_b, ((int64_t)j * w.out + col + c) * w.rank + k, v, 4, false, true);
            }
        }
    }
}

// ---- transposes of the adapters: [rows][columns] -> [columns][rows] ---------------

// 64 x 64 at a time through LDS; rows and columns are multiples of 8. Blocks past
// a_blocks are b's.
__global__ __launch_bounds__(256) void adapter_turn_kernel(const uint16_t* a, const uint16_t* b, uint16_t* at, uint16_t* bt,
                                                           int64_t in, int64_t out, int rank, int a_blocks) {
    __shared__ uint16_t tile[64][66];
    const bool is_a = (int)blockIdx.x < a_blocks;
    const int64_t rows = is_a ? rank : out, columns = is_a ? in : rank;
    const int across = (int)((columns + 63) / 64);
    const int block = is_a ? blockIdx.x : blockIdx.x - a_blocks;
    const int64_t r0 = (int64_t)(block / across) * 64, c0 = (int64_t)(block % across) * 64;
    const uint16_t* from = (is_a ? a : b) + (int64_t)blockIdx.y * rows * columns;
    uint16_t* to = (is_a ? at : bt) + (int64_t)blockIdx.y * rows * columns;
    for (int i = threadIdx.x; i < 64 * 8; i += 256) {
        const int r = i / 8, c = i % 8 * 8;
        if (r0 + r >= rows || c0 + c >= columns) continue;
        const uint4 v = *reinterpret_cast<const uint4*>(from + (r0 + r) * columns + c0 + c);
        uint32_t* t = reinterpret_cast<uint32_t*>(&tile[r][c]);
        t[0] = v.x, t[1] = v.y, t[2] = v.z, t[3] = v.w;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 64 * 8; i += 256) {
        const int c = i / 8, r = i % 8 * 8;
        if (c0 + c >= columns || r0 + r >= rows) continue;
        uint32_t q[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) q[k] = tile[r + 2 * k][c] | (uint32_t)tile[r + 2 * k + 1][c] << 16;
        *reinterpret_cast<uint4*>(to + (c0 + c) * rows + r0 + r) = make_uint4(q[0], q[1], q[2], q[3]);
    }
}

// ---- host --------------------------------------------------------------------

size_t padded(size_t n) { return (n + 255) / 256 * 256; }

struct Room {  // places in the workspace
    size_t offset, order, partial, scaled, turned_a, turned_b, bytes;
};

int shrink_tiles(int64_t tokens) { return tokens >= 1024 ? 2 : 1; }
int64_t shrink_piece(int64_t tokens, int adapters, int rank, int64_t in) {
    const int bm = 16 * shrink_tiles(tokens);
    const int64_t tiles = (tokens + bm - 1) / bm * ((rank + 63) / 64);
    int64_t pieces = 512 / (tiles > 0 ? tiles : 1);
    if (pieces > in / 256) pieces = in / 256;
    if (pieces > 32) pieces = 32;
    if (pieces < 1) pieces = 1;
    return ((in + pieces - 1) / pieces + 63) / 64 * 64;
}
int64_t piece_count(int64_t tokens, int adapters, int rank, int64_t in) {
    const int64_t p = shrink_piece(tokens, adapters, rank, in);
    return (in + p - 1) / p;
}

Room room_for(int64_t tokens, int adapters, int rank, int64_t in, int64_t out, bool grad) {
    Room r;
    r.offset = 0;
    r.order = padded(((size_t)adapters + 2) * 4);
    r.partial = r.order + padded((size_t)tokens * 4);
    r.scaled = r.partial + padded((size_t)piece_count(tokens, adapters, rank, grad ? out : in) * tokens * rank * 4);
    r.turned_a = r.scaled + (grad ? padded((size_t)tokens * rank * 4) : 0);
    r.turned_b = r.turned_a + (grad ? padded((size_t)adapters * rank * in * 2) : 0);
    r.bytes = r.turned_b + (grad ? padded((size_t)adapters * rank * out * 2) : 0);
    return r;
}

hipError_t plan(const int64_t* index, int64_t tokens, int adapters, int32_t* offset, int32_t* order, hipStream_t stream) {
    hipLaunchKernelGGL(adapter_plan_kernel, dim3((unsigned)adapters + 1), dim3(kPlanThreads), 0, stream, index, (int)tokens,
                       adapters, offset, order);
    return hipGetLastError();
}

hipError_t shrink(const ShrinkArgs& s, hipStream_t stream) {
    const int mt = shrink_tiles(s.tokens), nt = s.rank <= 16 ? 1 : s.rank <= 32 ? 2 : 4;
    const Groups g{s.offset, nullptr, 0, s.tokens, s.adapters};
    const dim3 grid((unsigned)worst_pieces(g, 16 * mt, true), (unsigned)((s.in + s.piece - 1) / s.piece), (unsigned)((s.rank + 16 * nt - 1) / (16 * nt)));
#define CGD_SHRINK(M, N) hipLaunchKernelGGL((adapter_shrink_kernel<M, N>), grid, dim3(256), 0, stream, s)
    if (mt == 1 && nt == 1)
        CGD_SHRINK(1, 1);
    else if (mt == 1 && nt == 2)
        CGD_SHRINK(1, 2);
    else if (mt == 1)
        CGD_SHRINK(1, 4);
    else if (nt == 1)
        CGD_SHRINK(2, 1);
    else if (nt == 2)
        CGD_SHRINK(2, 2);
    else
        CGD_SHRINK(2, 4);
#undef CGD_SHRINK
    return hipGetLastError();
}

hipError_t expand(const ExpandArgs& in, hipStream_t stream) {
    ExpandArgs e = in;
    const int nt = e.tokens >= 2048 && e.rank <= 128 ? 4 : e.tokens >= 512 ? 2 : 1;  // (at most 64 KB of LDS)
    const Groups g{e.offset, nullptr, 0, e.tokens, e.adapters + 1};
    const int64_t tiles = worst_pieces(g, 16 * nt, true), steps = e.out ? (e.width + 255) / 256 : 1;
    int64_t chunks = (1024 + tiles - 1) / tiles;
    if (chunks > steps) chunks = steps;
    e.chunk = (steps + chunks - 1) / chunks * 256;
    const dim3 grid((unsigned)tiles, (unsigned)((steps * 256 + e.chunk - 1) / e.chunk));
    const size_t lds = (size_t)2 * 16 * nt * (e.rank + 8) * 2;
    if (nt == 4)
        hipLaunchKernelGGL(adapter_expand_kernel<4>, grid, dim3(256), lds, stream, e);
    else if (nt == 2)
        hipLaunchKernelGGL(adapter_expand_kernel<2>, grid, dim3(256), lds, stream, e);
    else
        hipLaunchKernelGGL(adapter_expand_kernel<1>, grid, dim3(256), lds, stream, e);
    return hipGetLastError();
}

}  // namespace

size_t adapter_workspace_bytes(int64_t tokens, int adapters, int rank, int64_t in, int64_t out) {
    return tokens ? room_for(tokens, adapters, rank, in, out, false).bytes : 0;
}
size_t adapter_grad_workspace_bytes(int64_t tokens, int adapters, int rank, int64_t in, int64_t out) {
    return room_for(tokens, adapters, rank, in, out, true).bytes;
}

hipError_t launch_adapters(const AdapterArgs& p, void* workspace, hipStream_t stream) {
    if (p.tokens == 0) return hipSuccess;
    char* ws = static_cast<char*>(workspace);
    const Room room = room_for(p.tokens, p.adapters, p.rank, p.in, p.out_features, false);
    int32_t* offset = reinterpret_cast<int32_t*>(ws + room.offset);
    int32_t* order = reinterpret_cast<int32_t*>(ws + room.order);
    float* partial = reinterpret_cast<float*>(ws + room.partial);
    hipError_t err = plan(p.index, p.tokens, p.adapters, offset, order, stream);
    if (err != hipSuccess) return err;
    const int64_t piece = shrink_piece(p.tokens, p.adapters, p.rank, p.in);
    err = shrink(ShrinkArgs{p.x, p.a, offset, order, p.tokens, p.in, piece, p.adapters, p.rank, partial}, stream);
    if (err != hipSuccess) return err;
    return expand(ExpandArgs{partial, (int)((p.in + piece - 1) / piece), p.b, p.scale, offset, order, p.tokens, p.out_features, 0,
                             p.adapters, p.rank, p.residual, p.out, p.hidden, nullptr},
                  stream);
}

hipError_t launch_adapters_grad(const AdapterGradArgs& p, void* workspace, hipStream_t stream) {
    char* ws = static_cast<char*>(workspace);
    const Room room = room_for(p.tokens, p.adapters, p.rank, p.in, p.out_features, true);
    int32_t* offset = reinterpret_cast<int32_t*>(ws + room.offset);
    int32_t* order = reinterpret_cast<int32_t*>(ws + room.order);
    float* partial = reinterpret_cast<float*>(ws + room.partial);
    float* scaled = reinterpret_cast<float*>(ws + room.scaled);
    uint16_t* at = reinterpret_cast<uint16_t*>(ws + room.turned_a);
    uint16_t* bt = reinterpret_cast<uint16_t*>(ws + room.turned_b);
    hipError_t err = plan(p.index, p.tokens, p.adapters, offset, order, stream);
    if (err != hipSuccess) return err;
    if (p.tokens && (p.grad_x || p.grad_a)) {
        const int64_t down = (p.rank + 63) / 64;
        const int64_t a_blocks = p.grad_x ? down * ((p.in + 63) / 64) : 0, b_blocks = down * ((p.out_features + 63) / 64);
        hipLaunchKernelGGL(adapter_turn_kernel, dim3((unsigned)(a_blocks + b_blocks), (unsigned)p.adapters), dim3(256), 0, stream,
                           p.a, p.b, at, bt, p.in, p.out_features, p.rank, (int)a_blocks);
        if ((err = hipGetLastError()) != hipSuccess) return err;
        const int64_t piece = shrink_piece(p.tokens, p.adapters, p.rank, p.out_features);
        err = shrink(ShrinkArgs{p.grad, bt, offset, order, p.tokens, p.out_features, piece, p.adapters, p.rank, partial}, stream);
        if (err != hipSuccess) return err;
        err = expand(ExpandArgs{partial, (int)((p.out_features + piece - 1) / piece), at, p.scale, offset, order, p.tokens, p.in, 0,
                                p.adapters, p.rank, nullptr, p.grad_x, nullptr, p.grad_a ? scaled : nullptr},
                     stream);
        if (err != hipSuccess) return err;
    }
    if (p.grad_a || p.grad_b) {
        AdapterWeightArgs w{p.x, p.grad, scaled, p.hidden, p.scale, offset, order, p.in, p.out_features, p.adapters, p.rank, 0, p.grad_a, p.grad_b};
        w.a_blocks = p.grad_a ? (int)((p.in + 127) / 128) : 0;
        const int blocks = w.a_blocks + (p.grad_b ? (int)((p.out_features + 127) / 128) : 0);
#define CGD_WEIGHTS(RT, NW)                                                                                                    \
    hipLaunchKernelGGL((adapter_weight_kernel<RT, NW>), dim3((unsigned)blocks, (unsigned)p.adapters, (unsigned)((p.rank + 16 * RT - 1) / (16 * RT))), \
                       dim3(NW* kWave), (size_t)NW / 2 * RT * 8 * kWave * 16, stream, w)
        if (p.rank <= 16)
            CGD_WEIGHTS(1, 8);
        else
            CGD_WEIGHTS(2, 8);
#undef CGD_WEIGHTS
        err = hipGetLastError();
    }
    return err;
}

hipError_t preload_adapters() {
    hipFuncAttributes at;
    return hipFuncGetAttributes(&at, reinterpret_cast<const void*>(&adapter_plan_kernel));
}

}  // namespace cgd
