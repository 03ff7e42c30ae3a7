// Low-rank adapters of many requests in one batch, and their gradients.
//   h[t] = a[j] x[t],  out[t] = residual[t] + scale[j] b[j] h[t],  j = index[t]
//   gh[t] = scale[j] b[j]^T grad[t],  grad_x[t] = a[j]^T gh[t]
//   grad_a[j] = sum over j's tokens of gh x^T,  grad_b[j] = sum of scale grad h^T
// Tokens are put in order of their adapter first (a stable order: sums do not
// depend on timing), those without one last; tiles of 16 or 32 tokens then have one
// adapter each, and rows are gathered through that order. The products are skinny, a
// rank is some 8 to 256: what bounds them is reading x and writing out once, so the
// reduction over in_features and the out features are split until the CUs are busy,
// and loads and stores take 128 bytes of a row at a time.
// 4093 tokens of 24 requests, rank 64, 7168 -> 4096 with a residual: order 5.9 us, first
// product 21 (59 MB of x: 2.8 TB/s), second 26 (67 MB of residual and out: 2.6 TB/s).
// Operands loaded the way the matrix instructions want them: 37 and 40; both products in
// one kernel like that: 73 and more. Tiles of one adapter on one XCD, so that its weights
// come into one L2: 1 us less for the first product, none for the second.
// h and gh are fp32 sums; as operands of the second product they go in as two
// bf16 parts (v = hi + lo, off by 2^-16 of v at most), which costs matrix
// instructions that nothing waits for: results are rounded once.
#include "cgd_gemm_launch.h"
#include "cgd_layer_launch.h"

namespace cgd {

namespace {

typedef uint32_t uint4_t __attribute__((ext_vector_type(4)));
typedef uint32_t uint2_t __attribute__((ext_vector_type(2)));

// LDS is written and read through one type.
__device__ __forceinline__ void put16(void* p, const uint4& v) { *static_cast<uint4_t*>(p) = uint4_t{v.x, v.y, v.z, v.w}; }
__device__ __forceinline__ bf16x8_t get16(const void* p) { return __builtin_bit_cast(bf16x8_t, *static_cast<const uint4_t*>(p)); }
__device__ __forceinline__ bf16x8_t no_frag() { return __builtin_bit_cast(bf16x8_t, uint4_t{0, 0, 0, 0}); }
__device__ __forceinline__ float4_t mul16(const bf16x8_t& rows, const bf16x8_t& columns, const float4_t& sum) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(rows, columns, sum, 0, 0, 0);
}

// v = hi + lo in bf16 pairs: of two values. Both parts have v's sign, and neither is 0 where
// v is not (below 2^-103 the second may be): hi is what lies next below |v| in bf16, also
// where v itself is a bf16 number, lo the rest, rounded (off by 2^-16 of v at most). So an
// infinite operand gives infinities of one sign and no NaN, by 0 times it or by adding
// two signs, and a value that would round to an infinity does not become one. Of an
// infinity hi is the largest bf16 number and lo the infinity; of 0 (of either sign) both are 0.
__device__ __forceinline__ void halves2(float a, float b, uint32_t* hi, uint32_t* lo) {
    a += 0.0f;  // -0 becomes 0
    b += 0.0f;
    const uint32_t ua = __builtin_elementwise_sub_sat(__float_as_uint(a), 1u), ub = __builtin_elementwise_sub_sat(__float_as_uint(b), 1u);
    *hi = __builtin_amdgcn_perm(ub, ua, 0x07060302u);  // the upper halves
    *lo = pack_bf16x2(a - __uint_as_float(ua & 0xFFFF0000u), b - __uint_as_float(ub & 0xFFFF0000u));
}

// ---- order of the tokens ---------------------------------------------------

// A tile: up to `tile` (16 or 32) tokens in order, all of one adapter (group
// `adapters`: of none; < 0: no tile). Group g's tiles begin at slot
// offset[g] / tile + g: as many slots lie between that and the next group's as its
// tiles need, or one more, which says so. So a group knows its slots without the
// others' counts. token: past the tile's rows the last of them again.
constexpr int kTallTile = 32;
struct Tile {
    int group, row0, rows, pad;
    int token[kTallTile];
};

constexpr int kPlanThreads = 1024;
constexpr int kPlanWaves = kPlanThreads / kWave;
constexpr int kPlanKept = 8;  // tokens of a lane whose groups stay in registers between the two passes

// Up to kLongPlan tokens: block g finds those of adapter g (g = adapters: of none): how
// many come before them, and in a second pass their places. No block waits for
// another. Each wave has a run of tokens, so the order within a group is the
// tokens' own.
__device__ __forceinline__ void plan_group(const int64_t* __restrict__ index, int tokens, int adapters, int mine,
                                           int32_t* __restrict__ offset, int32_t* __restrict__ order, Tile* __restrict__ tiles, int tile,
                                           int32_t* less_of, int32_t* same_of) {
    const int lane = lane_id(), wave = threadIdx.x / kWave;
    const int run = (tokens + kPlanThreads - 1) / kPlanThreads * kWave;
    const int t0 = wave * run, t1 = t0 + run < tokens ? t0 + run : tokens;
    auto group = [&](int t) {
        const int64_t j = index[t];
        return j >= 0 && j < adapters ? (int)j : adapters;
    };
    int less = 0, same = 0;  // of the wave's tokens
    auto count = [&](int g) {
        less += __popcll(ballot(g < mine));
        same += __popcll(ballot(g == mine));
    };
    int kept[kPlanKept];
#pragma unroll
    for (int u = 0; u < kPlanKept; ++u) kept[u] = t0 + u * kWave + lane < t1 ? group(t0 + u * kWave + lane) : INT32_MAX;
#pragma unroll
    for (int u = 0; u < kPlanKept; ++u) count(kept[u]);
    for (int t = t0 + kPlanKept * kWave; t < t1; t += 4 * kWave) {
        int g[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) g[u] = t + u * kWave + lane < t1 ? group(t + u * kWave + lane) : INT32_MAX;
#pragma unroll
        for (int u = 0; u < 4; ++u) count(g[u]);
    }
    if (lane == 0) {
        less_of[wave] = less;
        same_of[wave] = same;
    }
    __syncthreads();
    int first = 0, at = 0, all = 0;
    for (int w = 0; w < kPlanWaves; ++w) {
        first += less_of[w];
        all += same_of[w];
        at += w < wave ? same_of[w] : 0;
    }
    at += first;
    Tile* const slots = tiles + first / tile + mine;
    for (int i = threadIdx.x, n = (first + all) / tile + 1 - first / tile; i < n; i += kPlanThreads) {
        const int left = all - i * tile;
        slots[i].group = left > 0 ? mine : -1;
        slots[i].row0 = first + i * tile;
        slots[i].rows = left < tile ? left : tile;
    }
    if (threadIdx.x == 0) {
        offset[mine] = first;
        if (mine == adapters) offset[mine + 1] = tokens;
    }
    if (same == 0) return;
    auto place = [&](bool hit, int t) {
        const uint64_t hits = ballot(hit);
        if (hit) {
            const int to = at + __popcll(hits & lanemask_lt()), i = to - first;
            order[to] = t;
            slots[i / tile].token[i % tile] = t;
            if (to == first + all - 1)
                for (int k = i % tile + 1; k < tile; ++k) slots[i / tile].token[k] = t;
        }
        at += __popcll(hits);
    };
#pragma unroll
    for (int u = 0; u < kPlanKept; ++u) place(kept[u] == mine, t0 + u * kWave + lane);
    for (int t = t0 + kPlanKept * kWave; t < t1; t += kWave) place(t + lane < t1 && group(t + lane) == mine, t + lane);
}

__global__ __launch_bounds__(kPlanThreads) void adapter_plan_kernel(const int64_t* index, int tokens, int adapters, int32_t* offset,
                                                                    int32_t* order, Tile* tiles, int tile) {
    __shared__ int32_t less_of[kPlanWaves], same_of[kPlanWaves];
    plan_group(index, tokens, adapters, blockIdx.x, offset, order, tiles, tile, less_of, same_of);
}

// Many tokens go in chunks, a block each: the tokens of every group in a chunk are
// counted, the counts added up over the chunks, and every chunk places its own. The
// groups' blocks above all read all tokens: us with these and with chunks, 8192 tokens
// of 64 adapters 6.8 and 12, 16384 13 and 12, 65536 43 and 13; 2^18 of 512 194 and 22.
// Chunks of 1024 take 17, 16 and 23 for the last three.
constexpr int64_t kLongPlan = 16384;
constexpr int kChunkThreads = 256, kChunkKept = 2, kChunkWaves = kChunkThreads / kWave, kChunk = kChunkThreads * kChunkKept;
constexpr int kMostGroups = 513;  // the adapters', and that of none
struct ChunkArgs {
    const int64_t* index;
    int tokens, adapters, chunks, tile;
    int32_t* counts;  // [chunks + 1][groups]: of the chunk; then: of those before it, and (last) of all
    int32_t* offset;
    int32_t* order;
    Tile* tiles;
};

// A chunk's tokens: their groups, and how many of the same wave and group come before
// each. count: [wave][group] of the block, the waves' counts then.
struct ChunkTokens {
    int group[kChunkKept], rank[kChunkKept], t0;
    __device__ __forceinline__ ChunkTokens(const ChunkArgs& p, volatile int32_t (*count)[kMostGroups]) {
        const int wave = threadIdx.x / kWave;
        t0 = blockIdx.x * kChunk + wave * (kChunk / kChunkWaves) + lane_id();
#pragma unroll
        for (int u = 0; u < kChunkKept; ++u) {
            group[u] = 1023;  // no token
            if (t0 + u * kWave < p.tokens) {
                const int64_t j = p.index[t0 + u * kWave];
                group[u] = j >= 0 && j < p.adapters ? (int)j : p.adapters;
            }
        }
        for (int i = lane_id(); i <= p.adapters; i += kWave) count[wave][i] = 0;
#pragma unroll
        for (int u = 0; u < kChunkKept; ++u) {
            uint64_t same = ~uint64_t(0);  // the lanes of the same group, bit by bit of its number
#pragma unroll
            for (int b = 0; b < 10; ++b) {
                const bool set = group[u] >> b & 1;
                const uint64_t lanes = ballot(set);
                same &= set ? lanes : ~lanes;
            }
            const int before = __popcll(same & lanemask_lt());
            __builtin_amdgcn_wave_barrier();
            const int have = group[u] <= p.adapters ? count[wave][group[u]] : 0;
            rank[u] = have + before;
            __builtin_amdgcn_wave_barrier();
            if (before == 0 && group[u] <= p.adapters) count[wave][group[u]] = have + __popcll(same);
        }
        __syncthreads();
    }
};

__global__ __launch_bounds__(kChunkThreads) void adapter_count_kernel(const ChunkArgs p) {
    __shared__ int32_t count[kChunkWaves][kMostGroups];
    const ChunkTokens t(p, count);
    for (int i = threadIdx.x; i <= p.adapters; i += kChunkThreads) {
        int n = 0;
#pragma unroll
        for (int w = 0; w < kChunkWaves; ++w) n += count[w][i];
        p.counts[(int64_t)blockIdx.x * (p.adapters + 1) + i] = n;
    }
}

__device__ __forceinline__ int sum_up_to_lane(int v) {
#pragma unroll
    for (int d = 1; d < kWave; d *= 2) {
        const int other = __shfl_up(v, d, kWave);
        if (lane_id() >= d) v += other;
    }
    return v;
}

// A wave for each group.
__global__ __launch_bounds__(256) void adapter_sum_kernel(const ChunkArgs p) {
    const int groups = p.adapters + 1, i = blockIdx.x * 4 + threadIdx.x / kWave;
    if (i >= groups) return;
    int sum = 0;
    for (int c0 = lane_id(); c0 - lane_id() < p.chunks; c0 += 4 * kWave) {
        int v[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) v[u] = c0 + u * kWave < p.chunks ? p.counts[(int64_t)(c0 + u * kWave) * groups + i] : 0;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int to = sum_up_to_lane(v[u]);
            if (c0 + u * kWave < p.chunks) p.counts[(int64_t)(c0 + u * kWave) * groups + i] = sum + to - v[u];
            sum += __shfl(to, kWave - 1, kWave);
        }
    }
    if (lane_id() == 0) p.counts[(int64_t)p.chunks * groups + i] = sum;
}

__global__ __launch_bounds__(kChunkThreads) void adapter_place_kernel(const ChunkArgs p) {
    constexpr int OWN = (kMostGroups + kChunkThreads - 1) / kChunkThreads;  // groups of a thread
    __shared__ int32_t count[kChunkWaves][kMostGroups];
    __shared__ int32_t first[kMostGroups + 1], wave_sum[kChunkWaves];
    const ChunkTokens t(p, count);
    const int wave = threadIdx.x / kWave, groups = p.adapters + 1, tile = p.tile, i0 = threadIdx.x * OWN;
    int all[OWN], before[OWN], sum = 0;
#pragma unroll
    for (int k = 0; k < OWN; ++k) {
        all[k] = before[k] = 0;
        if (i0 + k < groups) {
            all[k] = p.counts[(int64_t)p.chunks * groups + i0 + k];
            before[k] = p.counts[(int64_t)blockIdx.x * groups + i0 + k];
        }
        sum += all[k];
    }
    const int to = sum_up_to_lane(sum);
    if (lane_id() == kWave - 1) wave_sum[wave] = to;
    __syncthreads();
    int start = to - sum;
    for (int w = 0; w < wave; ++w) start += wave_sum[w];
#pragma unroll
    for (int k = 0; k < OWN; ++k) {
        const int i = i0 + k;
        if (i >= groups) break;
        first[i] = start;
        int at = start + before[k];
#pragma unroll
        for (int w = 0; w < kChunkWaves; ++w) {
            const int n = count[w][i];
            count[w][i] = at;
            at += n;
        }
        if (blockIdx.x == 0) {
            p.offset[i] = start;
            for (int j = (all[k] + tile - 1) / tile, n = (start + all[k]) / tile + 1 - start / tile; j < n; ++j) p.tiles[start / tile + i + j].group = -1;
        }
        start += all[k];
        if (i == p.adapters) {
            first[groups] = start;
            if (blockIdx.x == 0) p.offset[groups] = start;
        }
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kChunkKept; ++u) {
        const int g = t.group[u], token = t.t0 + u * kWave;
        if (g > p.adapters) continue;
        const int at = count[wave][g] + t.rank[u], begin = first[g], end = first[g + 1], k = at - begin;
        Tile& slot = p.tiles[begin / tile + g + k / tile];
        p.order[at] = token;
        slot.token[k % tile] = token;
        if (k % tile == 0) {
            slot.group = g;
            slot.row0 = at;
            slot.rows = end - at < tile ? end - at : tile;
        }
        if (at == end - 1)
            for (int r = k % tile + 1; r < tile; ++r) slot.token[r] = token;
    }
}

// ---- the first product: to the rank ------------------------------------------

struct ShrinkArgs {
    const uint16_t* x;       // [tokens, in]
    const uint16_t* w;       // [adapters, rank, in]; TURNED: [adapters, in, rank]
    const int64_t* index;    // few tokens: the kernel makes the tiles itself
    Tile* tiles;             // one for each blockIdx.x
    int64_t tokens, in, piece;  // piece: of `in` for one block, a multiple of 64
    int adapters, rank;
    float* partial;          // [pieces][token in order][rank]
};

// At most kFewTokens tokens need no plan: a wave holds all their groups, and a ballot
// for 64 of them counts those before a group. Saves the plan's launch: 4 us, for 2 more
// of the first product with 128 tokens (and 5 with 512).
constexpr int kFewTokens = 256;
constexpr int kTile = 16;
struct FewTokens {
    static constexpr int CHUNKS = kFewTokens / kWave;
    int of[CHUNKS];
    int tokens;
    __device__ __forceinline__ FewTokens(const int64_t* index, int n, int adapters) : tokens(n) {
#pragma unroll
        for (int c = 0; c < CHUNKS; ++c) {
            of[c] = INT32_MAX;
            if (c * kWave + lane_id() < n) {
                const int64_t j = index[c * kWave + lane_id()];
                of[c] = j >= 0 && j < adapters ? (int)j : adapters;
            }
        }
    }
    __device__ __forceinline__ int before(int group) const {
        int n = 0;
#pragma unroll
        for (int c = 0; c < CHUNKS; ++c)
            if (c * kWave < tokens) n += __popcll(ballot(of[c] < group));
        return n;
    }
    // to[i] = the group's token number skip + i, for i < rows; -> the last of them, in its lane (-1 elsewhere)
    __device__ __forceinline__ int list(int group, int skip, int rows, int* to) const {
        int seen = -skip, last = -1;
#pragma unroll
        for (int c = 0; c < CHUNKS; ++c) {
            if (c * kWave >= tokens) break;
            const uint64_t hits = ballot(of[c] == group);
            const int at = seen + __popcll(hits & lanemask_lt());
            if (of[c] == group && at >= 0 && at < rows) {
                to[at] = c * kWave + lane_id();
                if (at == rows - 1) last = to[at];
            }
            seen += __popcll(hits);
        }
        return last;
    }
};

// Tile `want` of a few tokens, by the first wave of every block for itself: the groups'
// first slots ascend, so ten counts find the slot's group among 512.
__device__ __forceinline__ void plan_few(const int64_t* index, int tokens, int adapters, int want, Tile& p) {
    if (threadIdx.x < kWave) {
        const FewTokens t(index, tokens, adapters);
        int group = 0;  // the last one whose slots begin at `want` or before it
        for (int hi = adapters; group < hi;) {
            const int mid = (group + hi + 1) / 2;
            if (t.before(mid) / kTile + mid <= want)
                group = mid;
            else
                hi = mid - 1;
        }
        const int first = t.before(group), skip = (want - first / kTile - group) * kTile;
        const int left = t.before(group + 1) - first - skip, rows = left < kTile ? left : kTile;
        if (lane_id() == 0) {
            p.group = left > 0 ? group : -1;
            p.row0 = first + skip;
            p.rows = rows;
        }
        const int last = t.list(group, skip, rows, p.token);
        if (last >= 0)
            for (int k = rows; k < kTile; ++k) p.token[k] = last;
    }
    __syncthreads();
}

// Rows on their way from memory to the matrix instructions. These want 16 rows side
// by side in neighbouring lanes; loaded like that, every lane's 16 bytes are an
// access of their own (some 100 cycles for a wave's load, measured). So eight lanes
// load 128 bytes of one row, and the rows are turned over in LDS of the wave's own:
// 16-byte piece c of row r lies at c ^ (r % 8), which spreads the 16 rows that an
// operand takes, and the pieces of a row, over all banks.
constexpr int kRowBytes = 128;
__device__ __forceinline__ char* turn_place(char* room, int row, int piece) {
    return room + row * kRowBytes + (piece ^ (row & 7)) * 16;
}

// A block has a tile of up to 16 * MT tokens and 16 * NT of the ranks over one piece
// of the reduction; its four waves take 64 * U of it in turn, the next ones on their
// way while these are multiplied, and join their sums through LDS. TURNED: w's rows are
// those of the reduction, and the LDS transposing read makes the operand.
template <int MT, int NT, int U, bool FEW, bool TURNED>
__global__ __launch_bounds__(256, 3) void adapter_shrink_kernel(const ShrinkArgs s) {
    constexpr int BM = 16 * MT, BN = 16 * NT, PITCH = BN + 4, ROWS = BM + BN;
    constexpr int TURN = ROWS * kRowBytes * U, SUMS = 4 * BM * PITCH * 4;
    __shared__ __attribute__((aligned(16))) char room[4 * TURN > SUMS ? 4 * TURN : SUMS];
    __shared__ Tile few;
    const Tile* tile = &s.tiles[blockIdx.x];
    if constexpr (FEW) {
        plan_few(s.index, (int)s.tokens, s.adapters, blockIdx.x, few);
        if (blockIdx.y == 0 && blockIdx.z == 0 && threadIdx.x < sizeof(Tile) / 4)
            reinterpret_cast<int*>(&s.tiles[blockIdx.x])[threadIdx.x] = reinterpret_cast<const int*>(&few)[threadIdx.x];
        tile = &few;
    }
    const int lane = lane_id(), wave = threadIdx.x / kWave, n = lane & 15, g = lane >> 4;
    const int group = uniform(tile->group), row0 = uniform(tile->row0), rows = uniform(tile->rows);
    if (group < 0 || group == s.adapters) return;
    const int rank0 = blockIdx.z * BN;
    const int64_t k0 = blockIdx.y * s.piece, k1 = k0 + s.piece < s.in ? k0 + s.piece : s.in;
    // a load's eight rows: 8 q + lane / 8 of the tokens, then of the ranks (eight past
    // the rank: the first again; nothing of them is stored)
    const int r8 = lane >> 3, c8 = lane & 7;
    const uint16_t* xp[2 * MT];
#pragma unroll
    for (int q = 0; q < 2 * MT; ++q) xp[q] = s.x + tile->token[q * 8 + r8] * s.in + k0 + c8 * 8;
    constexpr int WP = 2 * NT, WR = kWave / WP;  // TURNED: 16-byte pieces of a row, rows of a load
    const int wr = lane / WP, wc = lane % WP;
    const uint16_t* const wp = TURNED ? s.w + ((int64_t)group * s.in + k0 + wr) * s.rank + rank0 + (rank0 + wc * 8 < s.rank ? wc * 8 : 0)
                                      : s.w + ((int64_t)group * s.rank + rank0 + r8) * s.in + k0 + c8 * 8;
    auto w_at = [&](int k, int q) {
        return reinterpret_cast<const uint4*>(TURNED ? wp + (int64_t)(k + q * WR) * s.rank : wp + (rank0 + q * 8 < s.rank ? q * 8 * s.in : 0) + k);
    };
    // 32 bytes of each of four rows at a time
    auto turned_place = [](int row, int piece) { return row * (BN * 2) + (piece ^ (NT == 4 ? (row & 3) << 1 : 0)) * 16; };
    char* const mine = room + wave * TURN;
    float4_t acc[MT][NT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j] = float4_t{0.f, 0.f, 0.f, 0.f};
    uint4 stage[U][2 * (MT + NT)];
    const int span = (int)(k1 - k0), whole = span / (64 * U);
    auto load = [&](int u) {
#pragma unroll
        for (int v = 0; v < U; ++v) {
            const int k = (u * U + v) * 64;
#pragma unroll
            for (int q = 0; q < 2 * MT; ++q) stage[v][q] = *reinterpret_cast<const uint4*>(xp[q] + k);
#pragma unroll
            for (int q = 0; q < 2 * NT; ++q)
                stage[v][2 * MT + q] = *w_at(k, q);
        }
    };
    auto turn = [&](int v, int q) {
        char* at = mine + v * ROWS * kRowBytes;
        if (TURNED && q >= 2 * MT)
            put16(at + BM * kRowBytes + turned_place((q - 2 * MT) * WR + wr, wc), stage[v][q]);
        else
            put16(turn_place(at, q * 8 + r8, c8), stage[v][q]);
    };
    auto multiply = [&](int v) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            bf16x8_t xf[MT], wf[NT];
#pragma unroll
            for (int i = 0; i < MT; ++i) xf[i] = get16(turn_place(mine + v * ROWS * kRowBytes, i * 16 + n, h * 4 + g));
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                char* at = mine + v * ROWS * kRowBytes;
                if constexpr (TURNED)
                    wf[j] = turned((const CGD_LDS(char)*)(at + BM * kRowBytes + turned_place(h * 32 + g * 8 + (n >> 2), j * 2 + (n >> 1 & 1)) + (n & 1) * 8),
                                   4 * BN * 2);
                else
                    wf[j] = get16(turn_place(at, BM + j * 16 + n, h * 4 + g));
            }
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int j = 0; j < NT; ++j) acc[i][j] = mul16(wf[j], xf[i], acc[i][j]);
        }
    };
    int u = wave;
    if (u < whole) load(u);
    for (; u < whole; u += 4) {
#pragma unroll
        for (int v = 0; v < U; ++v)
#pragma unroll
            for (int q = 0; q < 2 * (MT + NT); ++q) turn(v, q);
        __builtin_amdgcn_sched_barrier(0);
        if (u + 4 < whole) load(u + 4);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int v = 0; v < U; ++v) multiply(v);
        __builtin_amdgcn_sched_barrier(0);
    }
    if (u == whole) {  // what is left of the piece is one wave's, with zeros behind it
        for (int k = whole * U * 64; k < span; k += 64) {
            const bool in = k + c8 * 8 < span;
#pragma unroll
            for (int q = 0; q < 2 * MT; ++q) stage[0][q] = in ? *reinterpret_cast<const uint4*>(xp[q] + k) : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int q = 0; q < 2 * NT; ++q)
                stage[0][2 * MT + q] = (TURNED ? k + q * WR + wr < span : in) ? *w_at(k, q) : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int q = 0; q < 2 * (MT + NT); ++q) turn(0, q);
            __builtin_amdgcn_sched_barrier(0);
            multiply(0);
            __builtin_amdgcn_sched_barrier(0);
        }
    }
    __syncthreads();
    float(*sums)[BM][PITCH] = reinterpret_cast<float(*)[BM][PITCH]>(room);
    // a lane has four consecutive ranks of one token
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) *reinterpret_cast<float4_t*>(&sums[wave][i * 16 + n][j * 16 + g * 4]) = acc[i][j];
    __syncthreads();
    float* out = s.partial + ((int64_t)blockIdx.y * s.tokens + row0) * s.rank + rank0;
    for (int i = threadIdx.x; i < BM * NT * 4; i += 256) {
        const int r = i / (NT * 4), c = i % (NT * 4) * 4;
        if (r >= rows || rank0 + c >= s.rank) continue;
        float4_t v = *reinterpret_cast<const float4_t*>(&sums[0][r][c]);
#pragma unroll
        for (int w = 1; w < 4; ++w) v += *reinterpret_cast<const float4_t*>(&sums[w][r][c]);
        *reinterpret_cast<float4_t*>(out + (int64_t)r * s.rank + c) = v;
    }
}

// ---- the second product: from the rank ----------------------------------------

constexpr int kMostPieces = 16;  // of the first product's reduction

struct ExpandArgs {
    const float* partial;    // [pieces][token in order][rank]
    int pieces;
    const uint16_t* w;       // [adapters, width, rank]; TURNED: [adapters, rank, width]
    const float* scale;      // [adapters] or null
    const Tile* tiles;
    int64_t tokens, width, chunk;  // chunk: of the out features for one block, a multiple of 64 for each wave
    int adapters, rank;
    const uint16_t* residual;
    uint16_t* out;           // [tokens, width], or null
    float* hidden;           // joined sums [token][rank], or null
    float* scaled;           // joined sums times the scale [token in order][rank], or null
};

// A block has a tile of up to 16 * MT tokens and `chunk` out features. KS matrix
// instructions cover the rank, padded with zeros to 32 * KS, for each of the two
// parts of h; KS = 0: a rank of up to 16, whose parts lie side by side in one
// instruction. A wave takes F features at a time: their rows of b, which are one run
// of memory, come in whole and are turned over in the wave's own LDS, the next F on
// their way; so do the results, the other way round, so that neighbouring lanes
// write one token's features.
template <int MT, int KS, bool TURNED>
__global__ __launch_bounds__(256, KS <= 2 ? 2 : 1) void adapter_expand_kernel(const ExpandArgs e) {
    constexpr int BM = 16 * MT, RANK = KS ? 32 * KS : 16, PITCH = RANK + 8, KN = KS ? KS : 1;
    constexpr int F = KS > 4 ? 32 : 64, FT = F / 16, OUT = F + 4, LOADS = F * RANK / 512;  // (a load: 1 KB)
    constexpr int ROOM = F * RANK * 2, OUT_ROOM = BM * OUT * 4;
    static_assert(ROOM % 16 == 0 && OUT_ROOM % 16 == 0, "16-byte pieces");
    __shared__ __attribute__((aligned(16))) uint16_t parts[2][BM][PITCH];
    __shared__ __attribute__((aligned(16))) char room[4][ROOM > OUT_ROOM ? ROOM : OUT_ROOM];  // b's rows, then the results
    const Tile* tile = &e.tiles[blockIdx.x];
    const int lane = lane_id(), wave = threadIdx.x / kWave, n = lane & 15, g = lane >> 4;
    const int group = uniform(tile->group), row0 = uniform(tile->row0), rows = uniform(tile->rows);
    if (group < 0) return;
    const bool none = group == e.adapters, whole = e.width % 8 == 0;
    const int64_t end = (int64_t)(blockIdx.y + 1) * e.chunk < e.width ? (int64_t)(blockIdx.y + 1) * e.chunk : e.width;
    // w in LDS: rows of PR 16-byte pieces, RPL of them a load, the lane piece lp of row
    // lane / PR. A row is a feature's ranks (zeros past the rank; piece i of all lies at
    // i ^ (i / 8 ^ i / 64) % 8) or, TURNED, a rank's features, where the transposing read
    // takes 32 bytes of each of four rows at a time.
    constexpr int PR = TURNED ? F / 8 : RANK / 8, RPL = kWave / PR;
    const int lr = lane / PR, lp = lane % PR;
    const int64_t pitch = TURNED ? e.width : e.rank;
    const uint16_t* const wp = e.w + (int64_t)group * e.width * e.rank + lr * pitch + lp * 8;
    uint4 stage[LOADS];
    auto load = [&](int64_t o0) {
        const uint16_t* from = wp + (TURNED ? o0 : o0 * e.rank);
        const int64_t next = RPL * pitch;
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            const bool in = TURNED ? i * RPL + lr < e.rank && o0 + lp * 8 < e.width : lp * 8 < e.rank && o0 + i * RPL + lr < e.width;
            stage[i] = in ? *reinterpret_cast<const uint4*>(from + i * next) : make_uint4(0, 0, 0, 0);
        }
    };
    auto place = [](int i) {
        if constexpr (TURNED) {
            const int row = i / PR;
            return (i ^ ((row << 1 & 6) & (PR - 1))) * 16;
        }
        return (i ^ (((i >> 3) ^ (i >> 6)) & 7)) * 16;
    };
    // the results' lanes: 8 features of token 64 * 8 / F * q + lane / (F / 8)
    constexpr int LR = F / 8, TOKENS = kWave / LR, Q = BM / TOKENS;
    const int rt = lane / LR, ro = lane % LR * 8;
    int64_t at[Q];  // of the lane's features in out and residual, but for o0; < 0: no token
#pragma unroll
    for (int q = 0; q < Q; ++q) at[q] = q * TOKENS + rt < rows ? tile->token[q * TOKENS + rt] * e.width + ro : -1;
    uint4 residual[Q];
    auto load_residual = [&](int64_t o0) {
        if (!e.residual || !whole) return;
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            residual[q] = make_uint4(0, 0, 0, 0);
            if (at[q] >= 0 && o0 + ro < e.width) residual[q] = *reinterpret_cast<const uint4*>(e.residual + at[q] + o0);
        }
    };
    int64_t o0 = blockIdx.y * e.chunk + wave * F;
    const float scale = none || !e.scale ? 1.0f : e.scale[group];
    if (e.out && o0 < end) {
        if (!none) load(o0);
        load_residual(o0);
    }
    // the pieces' sums: all of a thread's values of several pieces on their way at a time
    constexpr int ITEMS = (BM * RANK + 1023) / 1024;
    float4_t sum[ITEMS];
    auto item_row = [&](int i) { return (int)(i * 256 + threadIdx.x) / (RANK / 4); };
    auto item_column = [&](int i) { return (int)(i * 256 + threadIdx.x) % (RANK / 4) * 4; };
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) sum[i] = float4_t{0.f, 0.f, 0.f, 0.f};
    if (!none) {
        const float* from[ITEMS];
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {  // (what lies past the tile or the rank reads what is there: its sums are not kept)
            const int r = item_row(i) < rows ? item_row(i) : rows - 1, c = item_column(i) < e.rank ? item_column(i) : 0;
            from[i] = e.partial + (int64_t)(row0 + r) * e.rank + c;
        }
        const int64_t next = e.tokens * e.rank;
        constexpr int AT_ONCE = ITEMS > 2 ? 2 : ITEMS > 1 ? 4 : kMostPieces;
        for (int p = 0; p < e.pieces; p += AT_ONCE) {
            float4_t v[AT_ONCE][ITEMS];
#pragma unroll
            for (int u = 0; u < AT_ONCE; ++u)
#pragma unroll
                for (int i = 0; i < ITEMS; ++i) v[u][i] = *reinterpret_cast<const float4_t*>(from[i] + (p + u < e.pieces ? p + u : 0) * next);
#pragma unroll
            for (int u = 0; u < AT_ONCE; ++u)
#pragma unroll
                for (int i = 0; i < ITEMS; ++i)
                    if (p + u < e.pieces) sum[i] += v[u][i];
        }
    }
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
        const int r = item_row(i), c = item_column(i);
        if (r >= BM) break;  // (a small tile of a small rank has fewer values than threads)
        const bool in = r < rows && c < e.rank;
        // (nothing times an infinite scale would be NaN in every feature)
        const float4_t v = in ? sum[i] : float4_t{0.f, 0.f, 0.f, 0.f}, k = in ? v * scale : v;
        if (in && blockIdx.y == 0) {
            if (e.hidden) *reinterpret_cast<float4_t*>(e.hidden + (int64_t)tile->token[r] * e.rank + c) = v;
            if (e.scaled) *reinterpret_cast<float4_t*>(e.scaled + (int64_t)(row0 + r) * e.rank + c) = k;
        }
        uint32_t h[2], l[2];
        halves2(k[0], k[1], &h[0], &l[0]);
        halves2(k[2], k[3], &h[1], &l[1]);
        *reinterpret_cast<uint2_t*>(&parts[0][r][c]) = uint2_t{h[0], h[1]};
        *reinterpret_cast<uint2_t*>(&parts[1][r][c]) = uint2_t{l[0], l[1]};
    }
    if (!e.out) return;
    sync_lds();
    char* const mine = room[wave];
    float(*const results)[OUT] = reinterpret_cast<float(*)[OUT]>(mine);
    for (; o0 < end; o0 += 4 * F) {
        float4_t acc[MT][FT];
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
            for (int p = 0; p < FT; ++p) acc[t][p] = float4_t{0.f, 0.f, 0.f, 0.f};
        if (!none) {
#pragma unroll
            for (int i = 0; i < LOADS; ++i) put16(mine + place(i * 64 + lane), stage[i]);
            __builtin_amdgcn_sched_barrier(0);
            if (o0 + 4 * F < end) load(o0 + 4 * F);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int k = 0; k < KN; ++k) {
                const int piece = KS ? k * 4 + g : g & 1;
                bf16x8_t wf[FT];
#pragma unroll
                for (int p = 0; p < FT; ++p) {
                    if constexpr (TURNED)
                        wf[p] = turned((const CGD_LDS(char)*)(mine + place((piece * 8 + (n >> 2)) * PR + p * 2 + (n >> 1 & 1)) + (n & 1) * 8), 4 * F * 2);
                    else
                        wf[p] = get16(mine + place((p * 16 + n) * PR + piece));
                }
#pragma unroll
                for (int t = 0; t < MT; ++t) {
                    if constexpr (KS > 0) {
                        const bf16x8_t hi = get16(&parts[0][t * 16 + n][k * 32 + g * 8]), lo = get16(&parts[1][t * 16 + n][k * 32 + g * 8]);
#pragma unroll
                        for (int p = 0; p < FT; ++p) acc[t][p] = mul16(wf[p], lo, mul16(wf[p], hi, acc[t][p]));
                    } else {
                        const bf16x8_t h = get16(&parts[g >> 1][t * 16 + n][(g & 1) * 8]);
#pragma unroll
                        for (int p = 0; p < FT; ++p) acc[t][p] = mul16(wf[p], h, acc[t][p]);
                    }
                }
            }
        }
        // a lane has four consecutive features of one token; b's rows are in registers by now
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
            for (int p = 0; p < FT; ++p) *reinterpret_cast<float4_t*>(&results[t * 16 + n][p * 16 + g * 4]) = acc[t][p];
        __builtin_amdgcn_wave_barrier();
        const int64_t o = o0 + ro;
        const int have = (int)(e.width - o < 8 ? e.width - o : 8);
        uint4 now[Q];
#pragma unroll
        for (int q = 0; q < Q; ++q) now[q] = residual[q];
        if (o0 + 4 * F < end) load_residual(o0 + 4 * F);
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            const float4_t lo = *reinterpret_cast<const float4_t*>(&results[q * TOKENS + rt][ro]);
            const float4_t hi = *reinterpret_cast<const float4_t*>(&results[q * TOKENS + rt][ro + 4]);
            if (at[q] < 0 || have <= 0) continue;
            float v[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
            if (whole) {
                if (e.residual) {
                    const uint32_t r[4] = {now[q].x, now[q].y, now[q].z, now[q].w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        v[2 * i] += bf16_lo(r[i]);
                        v[2 * i + 1] += bf16_hi(r[i]);
                    }
                }
                store_run<8>(e.out, at[q] + o0, v, 8, false, true);
            } else {
                if (e.residual) {
                    float r[8];
                    load_run<8>(e.residual + at[q] + o0, have, false, r);
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[i] += r[i];
                }
                store_run<8>(e.out, at[q] + o0, v, have, false, false);
            }
        }
        __builtin_amdgcn_wave_barrier();
    }
}

// ---- the adapters' own gradients -----------------------------------------------

struct AdapterWeightArgs {
    const uint16_t* x;      // [tokens, in]
    const uint16_t* grad;   // [tokens, out]
    const float* scaled;    // gh [token in order][rank]
    const float* hidden;    // [token][rank]
    const float* scale;
    const int64_t* index;   // few tokens: the kernel finds its own
    int tokens;
    const int32_t* offset;
    const int32_t* order;
    int64_t in, out;
    int adapters, rank;
    int a_blocks;           // column blocks of grad_a; those of grad_b follow
    uint16_t* grad_a;
    uint16_t* grad_b;
    int shares;             // of an adapter's tokens, a block each
    float* partial_a;       // several shares: their sums, [share] of grad_a's and of grad_b's elements
    float* partial_b;
};

// A block has 128 columns (of x for grad_a, of grad for grad_b) and 16 * RT
// ranks of one adapter; its NW waves take 32 of the adapter's tokens in turn and
// join their sums through LDS in a fixed order. The wide operand is needed with
// eight tokens of one column in a lane: a lane loads eight columns of eight
// tokens, 16 bytes each, and turns that square over in its own registers; the
// eight matrix tiles it makes have every eighth column each.
// 4095 tokens of 16 adapters, rank 16, 4096 -> 7168: 23 us for 94 MB (4.1 TB/s); grad_a
// alone takes 15, the chain of a block's waits (its adapter's offset, the order, rows,
// join). The next tokens on their way, at half as many waves: 23.6; grad_b's blocks in
// the first product's launch: 42 for both and grad_a, where they take 38 one by one.
template <int RT, int NW, bool FEW>
__global__ __launch_bounds__(NW* kWave) void adapter_weight_kernel(const AdapterWeightArgs w) {
    extern __shared__ __attribute__((aligned(16))) float4_t joined[];  // [wave][RT * 8][lane]
    __shared__ int own[FEW ? kFewTokens : 1], bounds[2];
    const int lane = lane_id(), wave = threadIdx.x / kWave, n = lane & 15, g = lane >> 4;
    const bool is_a = (int)blockIdx.x < w.a_blocks;
    const int64_t width = is_a ? w.in : w.out;
    const int64_t col = (int64_t)(is_a ? blockIdx.x : blockIdx.x - w.a_blocks) * 128 + n * 8;
    const uint16_t* wide = is_a ? w.x : w.grad;
    const float* thin = is_a ? w.scaled : w.hidden;
    const int j = blockIdx.y / w.shares, share = blockIdx.y - j * w.shares, rank0 = blockIdx.z * 16 * RT;
    if constexpr (FEW) {
        if (wave == 0) {
            const FewTokens t(w.index, w.tokens, w.adapters);
            const int first = t.before(j), n = t.before(j + 1) - first;
            t.list(j, 0, n, own);
            if (lane == 0) {
                bounds[0] = first;
                bounds[1] = first + n;
            }
        }
        __syncthreads();
    }
    int begin = FEW ? bounds[0] : w.offset[j], end = FEW ? bounds[1] : w.offset[j + 1];
    if (!FEW && w.shares > 1) {  // whole steps of the waves
        const int each = ((end - begin + w.shares - 1) / w.shares + NW * 32 - 1) / (NW * 32) * (NW * 32);
        begin = begin + share * each < end ? begin + share * each : end;
        end = begin + each < end ? begin + each : end;
    }
    const int* const order = FEW ? own : w.order + begin;  // of the adapter's tokens
    const float scale = !is_a && w.scale ? w.scale[j] : 1.0f;
    float4_t acc[RT][8];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int c = 0; c < 8; ++c) acc[r][c] = float4_t{0.f, 0.f, 0.f, 0.f};
    // 32 tokens on their way: past the last one it is loaded again, and nothing of it multiplied
    struct Step {
        uint4 row[8];
        float v[RT][8];
    };
    const uint16_t* const from = wide + (col < width ? col : 0);
    int rank_at[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r) rank_at[r] = rank0 + r * 16 + n < w.rank ? rank0 + r * 16 + n : w.rank - 1;
    auto load = [&](Step& s, int p0) {
        const int p = p0 + g * 8;
        int token[8];
        if (p0 + 32 <= end) {
            __builtin_memcpy(token, order + (p - begin), sizeof(token));
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) token[i] = order[(p + i < end ? p + i : end - 1) - begin];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) s.row[i] = *reinterpret_cast<const uint4*>(from + token[i] * width);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float* at = thin + (int64_t)(!is_a ? token[i] : p + i < end ? p + i : end - 1) * w.rank;
#pragma unroll
            for (int r = 0; r < RT; ++r) s.v[r][i] = at[rank_at[r]];
        }
    };
    auto multiply = [&](Step& s, int p0) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int r = 0; r < RT; ++r) s.v[r][i] *= scale;
        if (p0 + 32 > end)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (p0 + g * 8 + i >= end) {
                    s.row[i] = make_uint4(0, 0, 0, 0);
#pragma unroll
                    for (int r = 0; r < RT; ++r) s.v[r][i] = 0.0f;
                }
        bf16x8_t hi[RT], lo[RT];
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            uint32_t h[4], l[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) halves2(s.v[r][2 * i], s.v[r][2 * i + 1], &h[i], &l[i]);
            hi[r] = __builtin_bit_cast(bf16x8_t, uint4_t{h[0], h[1], h[2], h[3]});
            lo[r] = __builtin_bit_cast(bf16x8_t, uint4_t{l[0], l[1], l[2], l[3]});
        }
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            uint32_t q[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t lower = reinterpret_cast<const uint32_t*>(&s.row[2 * i])[c / 2], upper = reinterpret_cast<const uint32_t*>(&s.row[2 * i + 1])[c / 2];
                q[i] = c & 1 ? (lower >> 16) | (upper & 0xFFFF0000u) : (lower & 0xFFFFu) | (upper << 16);
            }
            const bf16x8_t f = __builtin_bit_cast(bf16x8_t, uint4_t{q[0], q[1], q[2], q[3]});
#pragma unroll
            for (int r = 0; r < RT; ++r) acc[r][c] = mul16(lo[r], f, mul16(hi[r], f, acc[r][c]));
        }
    };
    Step s;
    for (int p0 = begin + wave * 32; p0 < end; p0 += NW * 32) {
        load(s, p0);
        multiply(s, p0);
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
                const int64_t at = ((int64_t)j * w.rank + k + i) * w.in + col;
                if (!FEW && w.shares > 1)
                    store_run<8>(w.partial_a, share * (w.adapters * w.rank * w.in) + at, v, 8, true, true);
                else
                    store_run<8>(w.grad_a, at, v, 8, false, true);
            }
        } else {  // [out][rank]: four ranks of eight columns
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                const float v[4] = {acc[r][c][0], acc[r][c][1], acc[r][c][2], acc[r][c][3]};
                const int64_t at = ((int64_t)j * w.out + col + c) * w.rank + k;
                if (!FEW && w.shares > 1)
                    store_run<4>(w.partial_b, share * (w.adapters * w.rank * w.out) + at, v, 4, true, true);
                else
                    store_run<4>(w.grad_b, at, v, 4, false, true);
            }
        }
    }
}

// Adds the shares' sums, in order; four elements a thread, grad_a's and then grad_b's.
__global__ __launch_bounds__(256) void adapter_join_kernel(const AdapterWeightArgs w) {
    const int64_t na = w.grad_a ? w.adapters * w.rank * w.in / 4 : 0, nb = w.grad_b ? w.adapters * w.rank * w.out / 4 : 0;
    const int64_t v = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (v >= na + nb) return;
    const bool is_a = v < na;
    const int64_t i = is_a ? v : v - na, next = is_a ? na : nb;
    const float4_t* from = reinterpret_cast<const float4_t*>(is_a ? w.partial_a : w.partial_b) + i;
    float4_t sum = from[0];
    for (int s = 1; s < w.shares; s += 4) {
        float4_t part[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) part[u] = from[(s + u < w.shares ? s + u : 0) * next];
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (s + u < w.shares) sum += part[u];
    }
    reinterpret_cast<uint2*>(is_a ? w.grad_a : w.grad_b)[i] = make_uint2(pack_bf16x2(sum[0], sum[1]), pack_bf16x2(sum[2], sum[3]));
}

// ---- host --------------------------------------------------------------------

size_t padded(size_t n) { return (n + 255) / 256 * 256; }

struct Room {  // places in the workspace
    size_t offset, order, counts, tiles, partial, scaled, shares, bytes;
};

bool few(int64_t tokens) { return tokens <= kFewTokens; }
// Tiles of 32 tokens read an adapter's weights half as often, but there are half as many,
// and one of an adapter with few tokens is padded more. us with 16 and 32 rows, 4096 -> 4096
// with a residual unless said otherwise: 1024 tokens of 8 adapters, rank 16 18.4 and 18.6, rank
// 64 27.1 and 28.2, of 64 adapters, rank 16 19.4 and 22.6; 2048 of 8, rank 64 33.3 and 35.6; 4093
// of 8, rank 64, 7168 -> 4096 53.6 and 51.4, its gradient 93.5 and 87.6; 16384 of 16, rank 16 137 and 133.
int tile_tokens(int64_t tokens) { return tokens >= 1024 ? kTallTile : kTile; }
int64_t tile_slots(int64_t tokens, int adapters) { return tokens / tile_tokens(tokens) + adapters + 1; }

// Pieces of the reduction: until there are some two blocks for a CU, of at least
// 64 for each of a block's waves. us with half as many blocks, these, and twice as many: 2048
// tokens of 8 adapters, rank 64, 4096 -> 4096 33.8, 35.6, 37.9; 4093, rank 64, 7168 -> 4096 49.9, 51.4, 51.9;
// 4095 of 16, rank 16, 4096 -> 7168 45.0, 43.5, 44.0, its gradient 57.1, 54.5, 55.9; 8192 of 8, rank 64 79.1, 74.6, 76.9.
int64_t shrink_piece(int64_t tokens, int rank, int64_t in) {
    const int64_t tiles = (tokens + tile_tokens(tokens) - 1) / tile_tokens(tokens) * ((rank + 63) / 64);
    int64_t pieces = (rank > 32 ? 768 : 640) / (tiles > 0 ? tiles : 1);
    if (pieces > in / 256) pieces = in / 256;
    if (pieces > kMostPieces) pieces = kMostPieces;
    if (pieces < 1) pieces = 1;
    return ((in + pieces - 1) / pieces + 63) / 64 * 64;
}
int64_t piece_count(int64_t tokens, int rank, int64_t in) {
    const int64_t p = shrink_piece(tokens, rank, in);
    return (in + p - 1) / p;
}

int64_t chunk_count(int64_t tokens) { return (tokens + kChunk - 1) / kChunk; }

// Shares of an adapter's tokens in its gradients, each with blocks of its own and sums
// that another kernel adds: few adapters with many tokens would leave CUs idle. us of a
// whole gradient without and with shares, 4096 -> 4096: 65536 tokens of one adapter, rank
// 16 772 and 511, rank 64 955 and 773; 16384, rank 16 224 and 149. From a block for every
// second CU on they cost more than they give (16384 tokens of two, rank 64: 207 and 237),
// and below 1536 tokens of an adapter the launch does (1024 of one, rank 16: 25 and 26.5).
// The host does not know how the tokens are spread and takes it for even. Where all are one
// adapter's, that one's blocks have all the work: 16384 tokens, rank 16, of 8, 32 and 64
// adapters 227, 325 and 324 (spread evenly 147, 152 and 161), 4096 79, 79 and 80 (45, 47 and 52);
// rank 64, 16384 tokens of 32 387 (270).
int64_t weight_shares(int64_t tokens, int adapters, int rank, int64_t in, int64_t out) {
    const int64_t blocks = ((in + 127) / 128 + (out + 127) / 128) * adapters * ((rank + 31) / 32);
    if (blocks > 128 || tokens < int64_t(1536) * adapters) return 1;
    int64_t shares = 1024 / blocks;
    if (shares > tokens / (256 * adapters)) shares = tokens / (256 * adapters);
    return shares > 16 ? 16 : shares;
}

Room room_for(int64_t tokens, int adapters, int rank, int64_t in, int64_t out, bool grad) {
    Room r;
    r.offset = 0;
    r.order = padded(((size_t)adapters + 2) * 4);
    r.counts = r.order + padded((size_t)tokens * 4);
    r.tiles = r.counts + (tokens > kLongPlan ? padded((size_t)(chunk_count(tokens) + 1) * (adapters + 1) * 4) : 0);
    r.partial = r.tiles + padded((size_t)tile_slots(tokens, adapters) * sizeof(Tile));
    r.scaled = r.partial + padded((size_t)piece_count(tokens, rank, grad ? out : in) * tokens * rank * 4);
    r.shares = r.scaled + (grad ? padded((size_t)tokens * rank * 4) : 0);
    const int64_t shares = grad ? weight_shares(tokens, adapters, rank, in, out) : 1;
    r.bytes = r.shares + (shares > 1 ? padded((size_t)shares * adapters * rank * (in + out) * 4) : 0);
    return r;
}

hipError_t plan(const int64_t* index, int64_t tokens, int adapters, int32_t* offset, int32_t* order, int32_t* counts, Tile* tiles, hipStream_t stream) {
    if (tokens > kLongPlan) {
        const ChunkArgs p{index, (int)tokens, adapters, (int)chunk_count(tokens), tile_tokens(tokens), counts, offset, order, tiles};
        hipLaunchKernelGGL(adapter_count_kernel, dim3((unsigned)p.chunks), dim3(kChunkThreads), 0, stream, p);
        hipLaunchKernelGGL(adapter_sum_kernel, dim3((unsigned)(adapters + 4) / 4), dim3(256), 0, stream, p);
        hipLaunchKernelGGL(adapter_place_kernel, dim3((unsigned)p.chunks), dim3(kChunkThreads), 0, stream, p);
        return hipGetLastError();
    }
    hipLaunchKernelGGL(adapter_plan_kernel, dim3((unsigned)adapters + 1), dim3(kPlanThreads), 0, stream, index, (int)tokens, adapters, offset,
                       order, tiles, tile_tokens(tokens));
    return hipGetLastError();
}

// FEW: the kernel makes the tiles itself, and there is no plan.
template <int MT, bool FEW, bool TURNED>
void shrink_rank(const ShrinkArgs& s, hipStream_t stream) {
    const int nt = s.rank <= 16 ? 1 : s.rank <= 32 ? 2 : 4;
    const dim3 grid((unsigned)tile_slots(s.tokens, s.adapters), (unsigned)((s.in + s.piece - 1) / s.piece), (unsigned)((s.rank + 16 * nt - 1) / (16 * nt)));
#define CGD_SHRINK(N) hipLaunchKernelGGL((adapter_shrink_kernel<MT, N, (MT + N <= 3 ? 2 : 1), FEW, TURNED>), grid, dim3(256), 0, stream, s)
    if (nt == 1)
        CGD_SHRINK(1);
    else if (nt == 2)
        CGD_SHRINK(2);
    else
        CGD_SHRINK(4);
#undef CGD_SHRINK
}

template <int MT, bool TURNED>
void expand_rank(const ExpandArgs& e, const dim3& grid, hipStream_t stream) {
#define CGD_EXPAND(K) hipLaunchKernelGGL((adapter_expand_kernel<MT, K, TURNED>), grid, dim3(256), 0, stream, e)
    if (e.rank <= 16)
        CGD_EXPAND(0);
    else if (e.rank <= 32)
        CGD_EXPAND(1);
    else if (e.rank <= 64)
        CGD_EXPAND(2);
    else if (e.rank <= 128)
        CGD_EXPAND(4);
    else
        CGD_EXPAND(8);
#undef CGD_EXPAND
}

template <bool TURNED>
void expand(ExpandArgs e, hipStream_t stream) {
    const int tile = tile_tokens(e.tokens), step = e.rank <= 128 ? 256 : 128;  // features of a block's waves at a time
    const int64_t tiles = (e.tokens + tile - 1) / tile, steps = e.out ? (e.width + step - 1) / step : 1;
    // Every chunk's block joins the same pieces first, so more blocks are not always better. us with
    // half as many, these, and twice as many: 1024 tokens of 8 adapters, rank 64, 4096 -> 4096 27.5, 28.2,
    // 33.8; 2048 36.4, 35.6, 42.0; 4093, 7168 -> 4096 54.6, 51.4, 55.5; 4095 of 16, rank 16, 4096 -> 7168 44.1, 43.5,
    // 43.8; 8192 of 8, rank 64 72.4, 74.6, 66.6; 16384 of 16, rank 16 134, 133, 125.
    int64_t chunks = ((e.rank > 32 ? 384 : 640) + tiles - 1) / tiles;
    if (chunks > steps) chunks = steps;
    e.chunk = (steps + chunks - 1) / chunks * step;
    const dim3 grid((unsigned)tile_slots(e.tokens, e.adapters), (unsigned)((steps * step + e.chunk - 1) / e.chunk));
    if (tile == kTile)
        expand_rank<1, TURNED>(e, grid, stream);
    else
        expand_rank<2, TURNED>(e, grid, stream);
}

// The two products; the pieces of the first are set here. TURNED: backwards, where
// each weight is the other product's.
template <bool TURNED>
hipError_t products(ShrinkArgs s, ExpandArgs e, hipStream_t stream) {
    s.piece = shrink_piece(s.tokens, s.rank, s.in);
    e.pieces = (int)((s.in + s.piece - 1) / s.piece);
    if (few(s.tokens))
        shrink_rank<1, true, TURNED>(s, stream);
    else if (tile_tokens(s.tokens) == kTile)
        shrink_rank<1, false, TURNED>(s, stream);
    else
        shrink_rank<2, false, TURNED>(s, stream);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
    expand<TURNED>(e, stream);
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
    Tile* tiles = reinterpret_cast<Tile*>(ws + room.tiles);
    float* partial = reinterpret_cast<float*>(ws + room.partial);
    if (!few(p.tokens)) {
        const hipError_t err = plan(p.index, p.tokens, p.adapters, reinterpret_cast<int32_t*>(ws + room.offset),
                                    reinterpret_cast<int32_t*>(ws + room.order),
                                    reinterpret_cast<int32_t*>(ws + room.counts), tiles, stream);
        if (err != hipSuccess) return err;
    }
    return products<false>(ShrinkArgs{p.x, p.a, p.index, tiles, p.tokens, p.in, 0, p.adapters, p.rank, partial},
                           ExpandArgs{partial, 0, p.b, p.scale, tiles, p.tokens, p.out_features, 0, p.adapters, p.rank, p.residual, p.out,
                                      p.hidden, nullptr},
                           stream);
}

hipError_t launch_adapters_grad(const AdapterGradArgs& p, void* workspace, hipStream_t stream) {
    char* ws = static_cast<char*>(workspace);
    const Room room = room_for(p.tokens, p.adapters, p.rank, p.in, p.out_features, true);
    int32_t* offset = reinterpret_cast<int32_t*>(ws + room.offset);
    int32_t* order = reinterpret_cast<int32_t*>(ws + room.order);
    Tile* tiles = reinterpret_cast<Tile*>(ws + room.tiles);
    float* partial = reinterpret_cast<float*>(ws + room.partial);
    float* scaled = reinterpret_cast<float*>(ws + room.scaled);
    hipError_t err = hipSuccess;
    if (!few(p.tokens)) err = plan(p.index, p.tokens, p.adapters, offset, order, reinterpret_cast<int32_t*>(ws + room.counts), tiles, stream);
    if (err != hipSuccess) return err;
    if (p.tokens && (p.grad_x || p.grad_a)) {
        err = products<true>(ShrinkArgs{p.grad, p.b, p.index, tiles, p.tokens, p.out_features, 0, p.adapters, p.rank, partial},
                             ExpandArgs{partial, 0, p.a, p.scale, tiles, p.tokens, p.in, 0, p.adapters, p.rank, nullptr, p.grad_x, nullptr,
                                        p.grad_a ? scaled : nullptr},
                             stream);
        if (err != hipSuccess) return err;
    }
    if (p.grad_a || p.grad_b) {
        AdapterWeightArgs w{p.x, p.grad, scaled, p.hidden, p.scale, p.index, (int)p.tokens, offset, order, p.in, p.out_features, p.adapters, p.rank, 0, p.grad_a, p.grad_b, (int)weight_shares(p.tokens, p.adapters, p.rank, p.in, p.out_features), nullptr, nullptr};
        w.partial_a = reinterpret_cast<float*>(ws + room.shares);
        w.partial_b = w.partial_a + (int64_t)w.shares * p.adapters * p.rank * p.in;
        w.a_blocks = p.grad_a ? (int)((p.in + 127) / 128) : 0;
        const int blocks = w.a_blocks + (p.grad_b ? (int)((p.out_features + 127) / 128) : 0);
#define CGD_WEIGHTS(RT, NW, FEW)                                                                                                    \
    hipLaunchKernelGGL((adapter_weight_kernel<RT, NW, FEW>), dim3((unsigned)blocks, (unsigned)(p.adapters * w.shares), (unsigned)((p.rank + 16 * RT - 1) / (16 * RT))), \
                       dim3(NW* kWave), (size_t)NW / 2 * RT * 8 * kWave * 16, stream, w)
        // More waves where an adapter has many tokens. Rank 16, 4095 tokens, 4096 -> 7168, us with
        // 4, 8 and 16 waves: 16 adapters 26 29 32, four 27 25 24; rank 64 with 4 and 8: 16 adapters 45 64,
        // one 64 48. (Shares are of 4 waves each.)
        const bool many = p.tokens >= int64_t(768) * p.adapters && w.shares == 1;
        if (few(p.tokens) && p.rank <= 16)
            CGD_WEIGHTS(1, 4, true);
        else if (few(p.tokens))
            CGD_WEIGHTS(2, 4, true);
        else if (p.rank <= 16 && many)
            CGD_WEIGHTS(1, 16, false);
        else if (p.rank <= 16)
            CGD_WEIGHTS(1, 4, false);
        else if (many)
            CGD_WEIGHTS(2, 8, false);
        else
            CGD_WEIGHTS(2, 4, false);
#undef CGD_WEIGHTS
        if (w.shares > 1) {
            const int64_t vectors = (int64_t)p.adapters * p.rank * ((p.grad_a ? p.in : 0) + (p.grad_b ? p.out_features : 0)) / 4;
            hipLaunchKernelGGL(adapter_join_kernel, dim3((unsigned)((vectors + 255) / 256)), dim3(256), 0, stream, w);
        }
        err = hipGetLastError();
    }
    return err;
}

hipError_t preload_adapters() {
    hipFuncAttributes at;
    return hipFuncGetAttributes(&at, reinterpret_cast<const void*>(&adapter_plan_kernel));
}

}  // namespace cgd
