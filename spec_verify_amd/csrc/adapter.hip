// Low-rank adapters of many requests beside a shared projection (svq_adapter_add):
//
//   t[m]   = A_s x[m]                      s = rows[m], fp32
//   out[m] = bf16(base[m] + scale[s] * B_s t[m])
//
// and out[m] = base[m] where rows[m] names no adapter. Two launches:
//
// 1. down: t, split over K. A workgroup takes 16 rows, up to 64 ranks, one range
//    of K and one of the adapters that occur among its rows; its 8 waves take the
//    range's 128-element tiles round-robin (x and A are both K-major, so MFMA
//    operands are loaded straight from memory, 64 contiguous bytes a row per
//    instruction) and meet in LDS. Rows of other adapters in the tile ride along
//    and are not stored: an output element depends on its own row of x and on its
//    own adapter only, so one request's infinities or NaN never reach another.
// 2. up: a wave takes 64 columns of those 16 rows; B is the MFMA's A operand, so
//    a lane ends up with 16 consecutive columns of one row and reads base and
//    writes out in 16-byte pieces. The K ranges of t are summed in a fixed order.
//
// t stays fp32 up to the second product, whose bf16 operand is scale * t split in
// two (high and low halves, 16 significant bits): rounding it to one bf16 would put
// an error of the size of the output's own rounding on the sum. MFMA time is idle
// here: the bound is the bytes of A, B, base and out (or, for a few rows, latency).
#include <algorithm>

#include "svq_launch.h"

namespace svq {

namespace {

constexpr int kDownWaves = 8;
constexpr int kUpWaves = 4;

// The adapter of lane l's row (row l % 16 of the tile): -1 for none, -2 past the end.
__device__ __forceinline__ int tile_slot(const int32_t *rows, int64_t row0, int64_t M, int slots, int lane) {
    const int64_t m = row0 + (lane & 15);
    if (m >= M) return -2;
    const int s = rows[m];
    return (uint32_t)s < (uint32_t)slots ? s : -1;
}

// Lane of the first row with this lane's adapter (lanes 0..15; their rows).
__device__ __forceinline__ int tile_first(int slot, int lane) {
    int first = 15;
#pragma unroll
    for (int j = 14; j >= 0; --j)
        if (__builtin_amdgcn_readlane(slot, j) == slot) first = j;
    return min(first, lane & 15);
}

// The adapters of a tile as the lanes of their first rows; rows without one are a group
// of their own where `bare` asks for them.
__device__ __forceinline__ uint32_t tile_leaders(int slot, int first, int lane, bool bare) {
    return (uint32_t)__ballot(lane < 16 && first == lane && (slot >= 0 || (bare && slot == -1)));
}

// Those that fall to one of `ways` workgroups.
__device__ __forceinline__ uint32_t of_way(uint32_t leaders, int ways, int way) {
    uint32_t mine = 0;
    for (int ord = 0; leaders; leaders &= leaders - 1, ++ord)
        if (ord % ways == way) mine |= leaders & -leaders;
    return mine;
}

// RT rank tiles of 16 per workgroup. The K range is the fastest block index (their number
// is padded to a multiple of 8 where it is above 4): workgroups that read one range of A,
// for other rows, then run on one XCD and find it in its L2.
template <int RT>
__global__ __launch_bounds__(64 * kDownWaves) __attribute__((amdgpu_waves_per_eu(4))) void adapter_down_kernel(
    const uint16_t *__restrict__ x, const uint16_t *__restrict__ a, const int32_t *__restrict__ rows,
    float *__restrict__ part, int64_t M, int K, int R, int slots, int ways, int rank_chunks, int range_blocks, int T) {
    static_assert(RT <= kDownWaves, "one wave sums one rank tile");
    __shared__ f32x4 red[kDownWaves][RT][64];
    const int lane = threadIdx.x & 63, wave = wave_id();
    const int r = lane & 15, g = lane >> 4;
    int b = blockIdx.x;
    const int ks = b % range_blocks;
    b /= range_blocks;
    const int rc = b % rank_chunks;
    b /= rank_chunks;
    const int row_tiles = (int)((M + 15) >> 4);
    const int way = b / row_tiles;  // slowest: workgroups that find no adapter come last
    const int64_t row0 = (int64_t)(b % row_tiles) * 16;
    const int KT = K >> 7, kend = min(KT, (ks + 1) * T);
    if (ks * T >= KT) return;
    const int slot = tile_slot(rows, row0, M, slots, lane);
    uint32_t mine = of_way(tile_leaders(slot, tile_first(slot, lane), lane, false), ways, way);
    const int64_t xrow = min(row0 + r, M - 1);
    const uint16_t *xp = x + xrow * K + 8 * g;
    const int rank0 = rc * 16 * RT;

    for (; mine; mine &= mine - 1) {
        const int s = __builtin_amdgcn_readlane(slot, __builtin_ctz(mine));
        const uint16_t *ap[RT];
        bool in[RT];
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            const int rank = rank0 + 16 * i + r;
            in[i] = rank < R;  // ranks past R: no load, a zero operand
            ap[i] = a + ((int64_t)s * R + min(rank, R - 1)) * K + 8 * g;
        }
        f32x4 acc[RT];
#pragma unroll
        for (int i = 0; i < RT; ++i) acc[i] = f32x4{0.f, 0.f, 0.f, 0.f};
        for (int kt = ks * T + wave; kt < kend; kt += kDownWaves) {
            uint4 xv[4], av[RT][4];
#pragma unroll
            for (int j = 0; j < 4; ++j) xv[j] = *(const uint4 *)(xp + kt * 128 + 32 * j);
#pragma unroll
            for (int i = 0; i < RT; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    av[i][j] = in[i] ? *(const uint4 *)(ap[i] + kt * 128 + 32 * j) : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int i = 0; i < RT; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i] = mfma16x16x32(xv[j], av[i][j], acc[i]);
        }
#pragma unroll
        for (int i = 0; i < RT; ++i) red[wave][i][lane] = acc[i];
        __syncthreads();
        if (wave < RT) {
            f32x4 sum = red[0][wave][lane];
#pragma unroll
            for (int w = 1; w < kDownWaves; ++w) sum += red[w][wave][lane];
            const int rank = rank0 + 16 * wave + r;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int rs = __shfl(slot, 4 * g + i);
                if (rs == s && rank < R) part[((int64_t)ks * M + row0 + 4 * g + i) * R + rank] = sum[i];
            }
        }
        __syncthreads();
    }
}

// NS: 32-rank steps. A workgroup takes 256 columns of `tiles` consecutive row tiles. t of
// all of a tile's rows is put together once; then B of one adapter after the other is
// multiplied with it (the next one's loads are issued as soon as the registers are free)
// and each result row keeps its own adapter's product. B stays in registers from one tile
// to the next while the adapter is the same (a prompt's tiles). Column groups are the
// fastest block index, padded to a multiple of 8: the groups' parts of B stay in one
// XCD's L2 as A's ranges do.
template <int NS>
__global__ __launch_bounds__(64 * kUpWaves) void
adapter_up_kernel(const uint16_t *base, const float *__restrict__ part, const uint16_t *__restrict__ b,
                  const int32_t *__restrict__ rows, const float *__restrict__ scales, uint16_t *out, int64_t M, int N,
                  int R, int slots, int64_t ld_base, int64_t ld_out, int ways, int col_blocks, int tiles, int splits) {
    constexpr int kPitch = 32 * NS + 8;      // bf16 elements: rows 16 bytes apart in banks
    constexpr int kEach = 2 * NS;            // ranks of a thread where t is put together
    constexpr int kVec = kEach < 4 ? kEach : 4;
    constexpr int kAhead = NS == 1 ? 8 : (NS == 8 ? 2 : 4);  // K ranges of t in flight
    __shared__ __attribute__((aligned(16))) uint16_t thi[2][16][kPitch], tlo[2][16][kPitch];
    const int lane = threadIdx.x & 63, wave = wave_id();
    const int r = lane & 15, g = lane >> 4;
    int blk = blockIdx.x;
    const int cg = blk % col_blocks;
    blk /= col_blocks;
    const int row_tiles = (int)((M + 15) >> 4), tile_groups = (row_tiles + tiles - 1) / tiles;
    const int way = blk / tile_groups;       // slowest, as in the first launch
    const int tile0 = blk % tile_groups * tiles, tile1 = min(tile0 + tiles, row_tiles);
    if (cg * kUpWaves * 64 >= N) return;
    const int col0 = (cg * kUpWaves + wave) * 64;
    const int col = col0 + 16 * g;           // this lane's 16 output columns
    const int trow = threadIdx.x >> 4, rank0 = (threadIdx.x & 15) * kEach;  // and its row and ranks of t
    // MFMA row 4 g' + i of product q is column 16 g' + 4 q + i. Addresses are a scalar base
    // and a 32-bit offset.
    const int brow = 16 * (r >> 2) + (r & 3);
    const uint32_t b_off = (uint32_t)(brow * R + 8 * g) * 2, t_off = (uint32_t)(trow * R + rank0) * 4;
    uint4 bv[NS][4];
    int have = -1;                           // the adapter in bv
    auto load_b = [&](int s) {
        if (s == have) return;
        have = s;
        const char *p = (const char *)(b + ((int64_t)s * N + col0) * R);
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int st = 0; st < NS; ++st) {
                bv[st][q] = make_uint4(0, 0, 0, 0);
                if (col0 + brow + 4 * q < N && 32 * st + 8 * g < R)
                    bv[st][q] = *(const uint4 *)(p + (int64_t)8 * q * R + 64 * st + b_off);
            }
    };

    for (int tile = tile0, buf = 0; tile < tile1; ++tile, buf ^= 1) {
        const int64_t row0 = (int64_t)tile * 16, m = row0 + r;  // m: this lane's row
        const int slot = tile_slot(rows, row0, M, slots, lane);
        const int first = tile_first(slot, lane);
        const uint32_t leaders = tile_leaders(slot, first, lane, true);
        uint32_t mine = of_way(leaders, ways, way);
        if (!mine) continue;
        const int s0 = __builtin_amdgcn_readlane(slot, __builtin_ctz(mine));
        if (s0 >= 0) load_b(s0);
        // t of this thread's row and ranks, summed over the K ranges in order
        const int tslot = __shfl(slot, trow);
        float t[kEach];
#pragma unroll
        for (int i = 0; i < kEach; ++i) t[i] = 0.f;
        {
            const char *p = (const char *)(part + row0 * R);
            for (int k0 = 0; k0 < splits; k0 += kAhead) {
                float v[kAhead][kEach];
#pragma unroll
                for (int k = 0; k < kAhead; ++k) {
                    const char *pk = p + (int64_t)(k0 + k) * M * R * 4;
#pragma unroll
                    for (int i = 0; i < kEach; i += kVec) {
                        const bool in = tslot >= 0 && k0 + k < splits && rank0 + i < R;
                        if constexpr (kVec == 2) {
                            const float2 f = in ? *(const float2 *)(pk + t_off + 4 * i) : make_float2(0.f, 0.f);
                            v[k][i] = f.x, v[k][i + 1] = f.y;
                        } else {
                            const float4 f = in ? *(const float4 *)(pk + t_off + 4 * i) : make_float4(0.f, 0.f, 0.f, 0.f);
                            v[k][i] = f.x, v[k][i + 1] = f.y, v[k][i + 2] = f.z, v[k][i + 3] = f.w;
                        }
                    }
                }
#pragma unroll
                for (int k = 0; k < kAhead; ++k)
#pragma unroll
                    for (int i = 0; i < kEach; ++i) t[i] += v[k][i];
            }
        }
        const float scale = tslot >= 0 ? scales[tslot] : 0.f;
        const bool my_row = slot >= -1 && (mine >> first & 1) && col < N;
        uint4 y[2];
        if (my_row) {
#pragma unroll
            for (int h = 0; h < 2; ++h) y[h] = *(const uint4 *)(base + m * ld_base + col + 8 * h);
        }
        // scale * t, rounded in two halves
#pragma unroll
        for (int i = 0; i < kEach; i += 2) {
            uint32_t hi2 = 0, lo2 = 0;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float f = scale * t[i + e];
                const uint32_t hi = f32_to_bf16_rne(f);
                const uint32_t lo = (hi & 0x7F80u) == 0x7F80u ? 0 : f32_to_bf16_rne(f - bits_f32(hi << 16));
                hi2 |= hi << (16 * e);
                lo2 |= lo << (16 * e);
            }
            *(uint32_t *)&thi[buf][trow][rank0 + i] = hi2;
            *(uint32_t *)&tlo[buf][trow][rank0 + i] = lo2;
        }
        lds_barrier();  // one a tile: the next tile writes the other half
        while (mine) {
            const int s = __builtin_amdgcn_readlane(slot, __builtin_ctz(mine));
            mine &= mine - 1;
            if (s < 0) {  // rows without an adapter
                if (my_row && slot == s && (const uint16_t *)out != base) {
                    *(uint4 *)(out + m * ld_out + col) = y[0];
                    *(uint4 *)(out + m * ld_out + col + 8) = y[1];
                }
                continue;
            }
            load_b(s);  // (the first, and what follows rows without one: others are on their way)
            f32x4 acc[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) acc[q] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int st = 0; st < NS; ++st) {
                const uint4 hi = *(const uint4 *)&thi[buf][r][32 * st + 8 * g];
                const uint4 lo = *(const uint4 *)&tlo[buf][r][32 * st + 8 * g];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    acc[q] = mfma16x16x32(bv[st][q], hi, acc[q]);
                    acc[q] = mfma16x16x32(bv[st][q], lo, acc[q]);
                }
            }
            if (mine) {
                const int next = __builtin_amdgcn_readlane(slot, __builtin_ctz(mine));
                if (next >= 0) load_b(next);
            }
            if (my_row && slot == s) {
                uint32_t o[8];
#pragma unroll
                for (int w = 0; w < 8; ++w) {
                    const uint32_t v = (&y[w >> 2].x)[w & 3];
                    const float lo = bits_f32(v << 16) + acc[w >> 1][2 * (w & 1)];
                    const float hi = bits_f32(v & 0xFFFF0000u) + acc[w >> 1][2 * (w & 1) + 1];
                    o[w] = (uint32_t)f32_to_bf16_rne(lo) | ((uint32_t)f32_to_bf16_rne(hi) << 16);
                }
                *(uint4 *)(out + m * ld_out + col) = make_uint4(o[0], o[1], o[2], o[3]);
                *(uint4 *)(out + m * ld_out + col + 8) = make_uint4(o[4], o[5], o[6], o[7]);
            }
        }
    }
}

}  // namespace

AdapterPlan plan_adapter(int64_t M, int64_t N, int64_t K, int64_t R, int64_t slots) {
    AdapterPlan p{};
    p.row_tiles = (M + 15) / 16;
    const int64_t distinct = std::min<int64_t>(std::min<int64_t>(M, 16), slots);  // adapters in a tile, at most
    p.rank_tiles = R <= 16 ? 1 : (R <= 32 ? 2 : 4);
    p.rank_chunks = (int)((R + 16 * p.rank_tiles - 1) / (16 * p.rank_tiles));
    // K ranges: one 128-element tile a wave while that fills the chip, longer ones for
    // many rows; a power of two, or a multiple of 8 blocks
    const int64_t KT = K / 128, groups = p.row_tiles * p.rank_chunks;
    int64_t blocks = std::max<int64_t>(1, std::min<int64_t>((KT + kDownWaves - 1) / kDownWaves, 512 / groups));
    if (groups < 64 && blocks > 4) blocks = (blocks + 7) / 8 * 8;
    p.tiles_per_split = (int)((KT + blocks - 1) / blocks);
    if (groups >= 64) {  // (a range of many rows' x is not shared: whole rounds of the waves)
        p.tiles_per_split = (p.tiles_per_split + kDownWaves - 1) / kDownWaves * kDownWaves;
        blocks = (KT + p.tiles_per_split - 1) / p.tiles_per_split;
    }
    p.splits = (int)((KT + p.tiles_per_split - 1) / p.tiles_per_split);
    p.range_blocks = (int)blocks;
    // adapters of one tile side by side while tiles alone do not fill the chip
    p.down_ways = (int)std::max<int64_t>(1, std::min<int64_t>(distinct, 1024 / (groups * blocks)));
    p.col_blocks = (int)((N + 64 * kUpWaves - 1) / (64 * kUpWaves));
    if (p.col_blocks > 4) p.col_blocks = (p.col_blocks + 7) / 8 * 8;
    // rows without an adapter are a group of their own
    p.up_tiles = (int)std::max<int64_t>(1, std::min<int64_t>(8, p.row_tiles * p.col_blocks / 1024));
    const int64_t up_groups = (p.row_tiles + p.up_tiles - 1) / p.up_tiles * p.col_blocks;
    p.up_ways = (int)std::max<int64_t>(1, std::min<int64_t>(std::min<int64_t>(distinct + 1, 16), 2560 / up_groups));
    p.workspace_bytes = kCounterBytes + (size_t)p.splits * M * R * 4;
    return p;
}

hipError_t launch_adapter_add(const AdapterPlan &p, const void *base, int64_t ld_base, const void *x, const void *a,
                              const void *b, const int32_t *rows, const float *scales, void *out, int64_t ld_out,
                              int64_t M, int64_t N, int64_t K, int R, int slots, void *workspace,
                              hipStream_t stream) {
    float *part = (float *)ws_partials(workspace);
    const dim3 down((uint32_t)(p.row_tiles * p.down_ways * p.rank_chunks * p.range_blocks));
#define SVQ_DOWN(RT)                                                                                                 \
    hipLaunchKernelGGL((adapter_down_kernel<RT>), down, dim3(64 * kDownWaves), 0, stream, (const uint16_t *)x,       \
                       (const uint16_t *)a, rows, part, M, (int)K, R, slots, p.down_ways, p.rank_chunks,             \
                       p.range_blocks, p.tiles_per_split)
    if (p.rank_tiles == 1) SVQ_DOWN(1);
    else if (p.rank_tiles == 2) SVQ_DOWN(2);
    else SVQ_DOWN(4);
#undef SVQ_DOWN
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const dim3 up((uint32_t)((p.row_tiles + p.up_tiles - 1) / p.up_tiles * p.up_ways * p.col_blocks));
#define SVQ_UP(NS)                                                                                                  \
    hipLaunchKernelGGL((adapter_up_kernel<NS>), up, dim3(64 * kUpWaves), 0, stream, (const uint16_t *)base, part,   \
                       (const uint16_t *)b, rows, scales, (uint16_t *)out, M, (int)N, R, slots, ld_base, ld_out,    \
                       p.up_ways, p.col_blocks, p.up_tiles, p.splits)
    if (R <= 32) SVQ_UP(1);
    else if (R <= 64) SVQ_UP(2);
    else if (R <= 128) SVQ_UP(4);
    else SVQ_UP(8);
#undef SVQ_UP
    return hipGetLastError();
}

}  // namespace svq
