// Low-rank adapters of many requests beside a shared projection (svq_adapter_add):
//
//   t[m]   = A_s x[m]                      s = rows[m], fp32
//   out[m] = bf16(base[m] + scale[s] * B_s t[m])
//
// and out[m] = base[m] where rows[m] names no adapter.
//
// Rows are worked on in items: up to 16 rows of one adapter, out of 256 consecutive rows
// wherever they stand among them. An adapter that several requests share is then read
// once per 16 of their rows. Two launches (or one, where little is to be read):
//
// 1. down: t, split over K. A workgroup finds its item (each row's rank among the rows of
//    its adapter, by ballots on the bits of the index; one writes the item down for the
//    second launch), and takes up to 64 ranks and one range of K; its 8 waves take the range's 128-element tiles round-robin (x and A are both
//    K-major, so MFMA operands are loaded straight from memory, 64 contiguous bytes a
//    row per instruction) and meet in LDS.
// 2. up: a wave takes 64 columns of an item's rows; B is the MFMA's A operand, so a lane
//    ends up with 16 consecutive columns of one row and reads base and writes out in
//    16-byte pieces. The K ranges of t are summed in a fixed order.
//
// An output element depends on its own row of x and on its own adapter only, so one
// request's infinities or NaN never reach another.
//
// Measured (us on the GPU, all launches; bytes of x, A, B, base and out once):
//   M = 1, K = N = 5120, R = 16: 8.0 (latency: each launch waits for memory twice)
//   M = 37, K = 640, N = 1040, R = 24, 5 adapters: 5.5 (one launch)
//   M = 128, K = 5120, N = 17408, R = 32, 32 adapters: 17.1 (52 MB: 3.1 TB/s)
//   M = 128, K = 17408, N = 5120, R = 64, 6 adapters: 19.1 (25 MB: 1.3 TB/s)
//   M = 2001, K = 5120, N = 6144, R = 16, 3 adapters: 26.0 (70 MB: 2.7 TB/s)
//
// t stays fp32 in the second product too: its bf16 operand is scale * t cut into three parts
// of 8 significant bits, which together are all 24. (Two parts rounded to nearest keep 16:
// where base and the product cancel (K = 5120, R = 16), the rms error then is 2.07e-3 of the
// result instead of 1.48e-3, and a value past the largest bf16 becomes an infinity.) MFMA time is
// idle here, so the third part costs 1.5% at most: the bound is the bytes of A, B, base and out
// (or, for a few rows, latency).
#include <algorithm>

#include "svq_requests.h"

namespace svq {

namespace {

constexpr int kDownWaves = 8;
constexpr int kUpWaves = 4;

constexpr int kBlockRows = 256;  // rows among which items are formed
constexpr int kParts = kBlockRows / 64;

// The items of a block of rows, in the order of their first rows. A lane keeps rows lane,
// 64 + lane, ...: the adapter (`slots` for none) and the rank among the block's rows of
// that adapter; 16 consecutive ranks are an item.
struct Items {
    int slot[kParts], rank[kParts];
    uint64_t lead[kParts];  // rows whose rank is a multiple of 16
    int parts;

    __device__ __forceinline__ void find(const int32_t *rows, int64_t row0, int64_t M, int slots, int lane) {
        const int n = (int)min(M - row0, (int64_t)kBlockRows);
        parts = (n + 63) >> 6;
        uint64_t in[kParts], same[kParts][kParts];
#pragma unroll
        for (int j = 0; j < kParts; ++j) {
            slot[j] = slots;
            const int i = 64 * j + lane;
            if (i < n) slot[j] = rows[row0 + i];
        }
#pragma unroll
        for (int j = 0; j < kParts; ++j) {
            lead[j] = 0;
            if (j >= parts) break;
            if ((uint32_t)slot[j] >= (uint32_t)slots) slot[j] = slots;
            in[j] = __ballot(64 * j + lane < n);
            if (64 * j + lane >= n) slot[j] = -1;
#pragma unroll
            for (int i = 0; i <= j; ++i) same[i][j] = in[i];
        }
        for (int b = 0; slots >> b; ++b) {
            uint64_t set[kParts];
#pragma unroll
            for (int j = 0; j < kParts; ++j) {
                if (j >= parts) break;
                set[j] = __ballot(slot[j] >> b & 1);
                const uint64_t other = (slot[j] >> b & 1) ? 0 : ~0ull;
#pragma unroll
                for (int i = 0; i <= j; ++i) same[i][j] &= set[i] ^ other;
            }
        }
#pragma unroll
        for (int j = 0; j < kParts; ++j) {
            if (j >= parts) break;
            int k = mbcnt(same[j][j]);
#pragma unroll
            for (int i = 0; i < j; ++i) k += __popcll(same[i][j]);
            rank[j] = k;
            lead[j] = __ballot(slot[j] >= 0 && k % 16 == 0);
        }
    }

    static __device__ __forceinline__ int mbcnt(uint64_t mask) {  // set bits below this lane
        return (int)__builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0));
    }

    // Item p: its adapter (`slots` for rows without one), or -1 if there are fewer; ids[0..15],
    // which hold -1, become its rows within the block.
    __device__ __forceinline__ int get(int p, int lane, int *ids) const {
        int s = -1, q = 0, before = 0;
#pragma unroll
        for (int j = 0; j < kParts; ++j) {
            if (j >= parts) break;
            const uint64_t hit = __ballot((lead[j] >> lane & 1) && before + mbcnt(lead[j]) == p);
            if (hit) {
                const int l = __builtin_ctzll(hit);
                s = __builtin_amdgcn_readlane(slot[j], l);
                q = __builtin_amdgcn_readlane(rank[j], l) >> 4;
            }
            before += __popcll(lead[j]);
        }
        if (s < 0) return s;
#pragma unroll
        for (int j = 0; j < kParts; ++j) {
            if (j >= parts) break;
            if (slot[j] == s && rank[j] >> 4 == q) ids[rank[j] & 15] = 64 * j + lane;
        }
        return s;
    }
};

// An fp32 value as the exact sum of three bf16 patterns, each cut off the rest (below 2^-110
// what falls under the smallest bf16 is lost). Infinities and NaN are the first part.
struct Parts {
    uint32_t part[3];
    __device__ __forceinline__ explicit Parts(float f) {
        const uint32_t u = f32_bits(f);
        if ((u & 0x7F800000u) == 0x7F800000u) {
            part[0] = u >> 16 | ((u & 0x7FFFFFu) ? 0x40u : 0);
            part[1] = part[2] = 0;
        } else {
            const float r = f - bits_f32(u & 0xFFFF0000u);
            const uint32_t v = f32_bits(r);
            part[0] = u >> 16;
            part[1] = v >> 16;
            part[2] = f32_bits(r - bits_f32(v & 0xFFFF0000u)) >> 16;
        }
    }
};

// An item as the second launch reads it.
struct Item {
    int slot;     // `slots`: rows without an adapter; -1: no item
    int row0;     // the block of rows
    int pad[14];
    int row[16];  // within the block; -1 past the last
};

// RT rank tiles of 16 per workgroup. The K range is the fastest block index (their number
// is padded to a multiple of 8 where it is above 4): workgroups that read one range of A,
// for other rows, then run on one XCD and find it in its L2. The item is the slowest one:
// workgroups that find none left come last (as the first ones they held up the others:
// 10.4 us instead of 6.7 at M = 128, R = 32). Of those 6.7 us 1.9 go to the rows' indexes
// and the item, 2 to the loads and 1 to the sum over waves.
template <int RT>
__global__ __launch_bounds__(64 * kDownWaves) __attribute__((amdgpu_waves_per_eu(4))) void adapter_down_kernel(
    const uint16_t *__restrict__ x, const uint16_t *__restrict__ a, const int32_t *__restrict__ rows,
    Item *__restrict__ table, float *__restrict__ part, int64_t M, int K, int R, int slots, int rank_chunks,
    int range_blocks, int T) {
    static_assert(RT <= kDownWaves, "one wave sums one rank tile");
    __shared__ f32x4 red[kDownWaves][RT][64];
    __shared__ __attribute__((aligned(16))) int ids[16], item_slot;
    const int lane = threadIdx.x & 63, wave = wave_id();
    const int r = lane & 15, g = lane >> 4;
    int b = blockIdx.x;
    const int ks = b % range_blocks;
    b /= range_blocks;
    const int rc = b % rank_chunks;
    b /= rank_chunks;
    const int blocks = (int)((M + kBlockRows - 1) / kBlockRows);
    const int64_t row0 = (int64_t)(b % blocks) * kBlockRows;
    const int item = b;  // of all blocks of rows
    const int KT = K >> 7, kend = min(KT, (ks + 1) * T);
    if (ks * T >= KT) return;
    if (wave == 0) {
        Items items;
        items.find(rows, row0, M, slots, lane);
        if (lane < 16) ids[lane] = -1;
        __builtin_amdgcn_wave_barrier();  // a wave's LDS accesses are done in order
        const int found = items.get(b / blocks, lane, ids);
        if (lane == 0) item_slot = found;
    }
    __syncthreads();
    const int s = __builtin_amdgcn_readfirstlane(item_slot);
    if (ks == 0 && rc == 0 && wave == 1 && lane < 16) {
        table[item].row[lane] = ids[lane];
        if (lane == 0) {
            table[item].slot = s;
            table[item].row0 = (int)row0;
        }
    }
    if (s < 0 || s == slots) return;
    const int64_t xrow = row0 + max(ids[r], ids[0]);  // past the last: the first again
    const uint16_t *xp = x + xrow * K + 8 * g;
    const int rank0 = rc * 16 * RT;
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
            const int id = ids[4 * g + i];
            if (id >= 0 && rank < R) part[((int64_t)ks * M + row0 + id) * R + rank] = sum[i];
        }
    }
}

// NS: 32-rank steps. A workgroup takes 256 columns of an item. Column groups are the
// fastest block index, padded to a multiple of 8: the groups' parts of B stay in one XCD's
// L2 as A's ranges do. One item a workgroup: in a loop over several, with B kept while
// the adapter stays, the registers go from 46 to 113 (rank 32) and half of the waves that
// hide the loads are gone (M = 128, R = 32: 20 us instead of 10.5, 4.0 TB/s).
template <int NS>
__global__ __launch_bounds__(64 * kUpWaves) void adapter_up_kernel(
    const uint16_t *base, const float *__restrict__ part, const uint16_t *__restrict__ b,
    const Item *__restrict__ table, const float *__restrict__ scales, uint16_t *out, int64_t M, int N, int R,
    int slots, int64_t ld_base, int64_t ld_out, int col_blocks, int splits) {
    constexpr int kPitch = 32 * NS + 8;      // bf16 elements: rows 16 bytes apart in banks
    constexpr int kEach = 2 * NS;            // ranks of a thread where t is put together
    constexpr int kVec = kEach < 4 ? kEach : 4;
    constexpr int kAhead = NS <= 2 ? 8 : (NS == 4 ? 4 : 2);  // K ranges of t in flight
    __shared__ __attribute__((aligned(16))) uint16_t ts[3][16][kPitch];  // scale * t in three parts
    const int lane = threadIdx.x & 63, wave = wave_id();
    const int r = lane & 15, g = lane >> 4;
    const int cg = blockIdx.x % col_blocks;
    const Item &item = table[blockIdx.x / col_blocks];
    if (cg * kUpWaves * 64 >= N) return;
    const int s = item.slot;
    if (s < 0) return;
    const int col0 = (cg * kUpWaves + wave) * 64;
    const int col = col0 + 16 * g;           // this lane's 16 output columns
    const int trow = threadIdx.x >> 4, rank0 = (threadIdx.x & 15) * kEach;  // and its row and ranks of t
    // MFMA row 4 g' + i of product q is column 16 g' + 4 q + i. Addresses are a scalar base
    // and a 32-bit offset.
    const int brow = 16 * (r >> 2) + (r & 3);
    const uint32_t b_off = (uint32_t)(brow * R + 8 * g) * 2;
    const int64_t row0 = item.row0;
    const int id = item.row[r], tid = item.row[trow];
    const int64_t m = row0 + id;             // this lane's row
    const bool mine = id >= 0 && col < N;
    uint4 y[2];
    if (s == slots) {  // rows without an adapter
        if (mine && (const uint16_t *)out != base) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
                *(uint4 *)(out + m * ld_out + col + 8 * h) = *(const uint4 *)(base + m * ld_base + col + 8 * h);
        }
        return;
    }
    // t of this thread's row and ranks, summed over the K ranges in order. Loads complete in
    // order: those of B and base, which take longer, are issued behind the last ranges'.
    float t[kEach], v[kAhead][kEach];
    const char *tp = (const char *)(part + row0 * R);
    const uint32_t t_off = (uint32_t)(tid * R + rank0) * 4;
    auto ranges = [&](int k0) {
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const char *pk = tp + (int64_t)(k0 + k) * M * R * 4;
#pragma unroll
            for (int i = 0; i < kEach; i += kVec) {
                const bool in = tid >= 0 && k0 + k < splits && rank0 + i < R;
                if constexpr (kVec == 2) {
                    const float2 f = in ? *(const float2 *)(pk + t_off + 4 * i) : make_float2(0.f, 0.f);
                    v[k][i] = f.x, v[k][i + 1] = f.y;
                } else {
                    const float4 f = in ? *(const float4 *)(pk + t_off + 4 * i) : make_float4(0.f, 0.f, 0.f, 0.f);
                    v[k][i] = f.x, v[k][i + 1] = f.y, v[k][i + 2] = f.z, v[k][i + 3] = f.w;
                }
            }
        }
    };
    auto add = [&] {
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
#pragma unroll
            for (int i = 0; i < kEach; ++i) t[i] += v[k][i];
    };
#pragma unroll
    for (int i = 0; i < kEach; ++i) t[i] = 0.f;
    int k0 = 0;
    for (; k0 + kAhead < splits; k0 += kAhead) {
        ranges(k0);
        add();
    }
    ranges(k0);
    uint4 bv[NS][4];
    const char *bp = (const char *)(b + ((int64_t)s * N + col0) * R);
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int st = 0; st < NS; ++st) {
            bv[st][q] = make_uint4(0, 0, 0, 0);
            if (col0 + brow + 4 * q < N && 32 * st + 8 * g < R)
                bv[st][q] = *(const uint4 *)(bp + (int64_t)8 * q * R + 64 * st + b_off);
        }
    if (mine) {
#pragma unroll
        for (int h = 0; h < 2; ++h) y[h] = *(const uint4 *)(base + m * ld_base + col + 8 * h);
    }
    add();
    const float scale = scales[s];
#pragma unroll
    for (int i = 0; i < kEach; i += 2) {
        const Parts even(scale * t[i]), odd(scale * t[i + 1]);
#pragma unroll
        for (int h = 0; h < 3; ++h) *(uint32_t *)&ts[h][trow][rank0 + i] = even.part[h] | odd.part[h] << 16;
    }
    lds_barrier();
    f32x4 acc[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) acc[q] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int st = 0; st < NS; ++st)
#pragma unroll
        for (int h = 0; h < 3; ++h) {
            const uint4 tv = *(const uint4 *)&ts[h][r][32 * st + 8 * g];
#pragma unroll
            for (int q = 0; q < 4; ++q) acc[q] = mfma16x16x32(bv[st][q], tv, acc[q]);
        }
    if (mine) {
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

// Both products in one launch, for a short K and few items: a workgroup takes 512 columns
// of an item and computes the item's whole t itself. That reads A once per workgroup, and a
// compute unit gets about 30 GB/s of it (5 us for 160 KB); against that stands a launch with its
// waits for memory (M = 37, K = 640, N = 1040, R = 24: 5.5 us instead of 8.0). RT rank tiles.
constexpr int kOneWaves = 16;
constexpr int kOneColumns = 32 * kOneWaves;
template <int RT>
__global__ __launch_bounds__(64 * kOneWaves) __attribute__((amdgpu_waves_per_eu(4))) void adapter_one_kernel(
    const uint16_t *base, const uint16_t *__restrict__ x, const uint16_t *__restrict__ a,
    const uint16_t *__restrict__ b, const int32_t *__restrict__ rows, const float *__restrict__ scales, uint16_t *out,
    int64_t M, int N, int K, int R, int slots, int64_t ld_base, int64_t ld_out, int col_blocks) {
    constexpr int NS = (RT + 1) / 2;     // 32-rank steps
    constexpr int kPitch = 32 * NS + 8;
    constexpr int kAhead = RT == 1 ? 2 : 1;  // K tiles in flight
    static_assert(256 * RT <= 64 * kOneWaves, "one thread sums one element of t");
    __shared__ float red[kOneWaves][RT * 256];
    __shared__ __attribute__((aligned(16))) uint16_t ts[3][16][kPitch];  // scale * t in three parts
    __shared__ __attribute__((aligned(16))) int ids[16], item_slot;
    const int lane = threadIdx.x & 63, wave = wave_id();
    const int r = lane & 15, g = lane >> 4;
    const int cb = blockIdx.x % col_blocks, item = blockIdx.x / col_blocks;
    const int blocks = (int)((M + kBlockRows - 1) / kBlockRows);
    const int64_t row0 = (int64_t)(item % blocks) * kBlockRows;
    if (wave == 0) {
        Items items;
        items.find(rows, row0, M, slots, lane);
        if (lane < 16) ids[lane] = -1;
        __builtin_amdgcn_wave_barrier();  // a wave's LDS accesses are done in order
        const int found = items.get(item / blocks, lane, ids);
        if (lane == 0) item_slot = found;
    }
    __syncthreads();
    const int s = __builtin_amdgcn_readfirstlane(item_slot);
    if (s < 0) return;
    // MFMA row 4 g' + i of product q is column 8 g' + 4 q + i: a lane ends up with 8
    // consecutive columns of one row
    const int col0 = (cb * kOneWaves + wave) * 32;
    const int col = col0 + 8 * g, id = ids[r];
    const int64_t m = row0 + id;
    const bool mine = id >= 0 && col < N;
    uint4 y = make_uint4(0, 0, 0, 0);
    if (mine) y = *(const uint4 *)(base + m * ld_base + col);
    if (s == slots) {  // rows without an adapter
        if (mine && (const uint16_t *)out != base) *(uint4 *)(out + m * ld_out + col) = y;
        return;
    }
    uint4 bv[NS][2];
    const int brow = col0 + 8 * (r >> 2) + (r & 3);
#pragma unroll
    for (int q = 0; q < 2; ++q)
#pragma unroll
        for (int st = 0; st < NS; ++st) {
            bv[st][q] = make_uint4(0, 0, 0, 0);
            if (brow + 4 * q < N && 32 * st + 8 * g < R)
                bv[st][q] = *(const uint4 *)(b + ((int64_t)s * N + brow + 4 * q) * R + 32 * st + 8 * g);
        }
    const float scale = scales[s];
    const uint16_t *xp = x + (row0 + max(id, ids[0])) * K + 8 * g;  // past the last: the first again
    const uint16_t *ap[RT];
    bool in[RT];
#pragma unroll
    for (int i = 0; i < RT; ++i) {
        in[i] = 16 * i + r < R;  // ranks past R: no load, a zero operand
        ap[i] = a + ((int64_t)s * R + min(16 * i + r, R - 1)) * K + 8 * g;
    }
    f32x4 acc[RT];
#pragma unroll
    for (int i = 0; i < RT; ++i) acc[i] = f32x4{0.f, 0.f, 0.f, 0.f};
    const int KT = K >> 7;
    for (int k0 = wave; k0 < KT; k0 += kAhead * kOneWaves) {
        uint4 xv[kAhead][4], av[kAhead][RT][4];
#pragma unroll
        for (int h = 0; h < kAhead; ++h) {
            const int kt = k0 + h * kOneWaves;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                xv[h][j] = kt < KT ? *(const uint4 *)(xp + kt * 128 + 32 * j) : make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int i = 0; i < RT; ++i)
                    av[h][i][j] = kt < KT && in[i] ? *(const uint4 *)(ap[i] + kt * 128 + 32 * j) : make_uint4(0, 0, 0, 0);
            }
        }
#pragma unroll
        for (int h = 0; h < kAhead; ++h)
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int i = 0; i < RT; ++i) acc[i] = mfma16x16x32(xv[h][j], av[h][i][j], acc[i]);
    }
#pragma unroll
    for (int i = 0; i < RT; ++i) *(f32x4 *)&red[wave][256 * i + 4 * lane] = acc[i];
    __syncthreads();
    const int at = threadIdx.x;
    if (at < 256 * RT) {  // element i of lane l of tile j: row 4 (l / 16) + i, rank 16 j + l % 16
        float t = red[0][at];
#pragma unroll
        for (int w = 1; w < kOneWaves; ++w) t += red[w][at];
        const int row = 4 * (at >> 6 & 3) + (at & 3), rank = 16 * (at >> 8) + (at >> 2 & 15);
        // Ranks past R are zero whatever their sum of zero products: it is NaN where x holds
        // an infinity.
        const Parts v(rank < R ? scale * t : 0.f);
#pragma unroll
        for (int h = 0; h < 3; ++h) ts[h][row][rank] = (uint16_t)v.part[h];
    } else if (RT == 1 && at < 512) {  // of a step of 32 ranks, those past the tile
#pragma unroll
        for (int h = 0; h < 3; ++h) ts[h][at >> 4 & 15][16 + (at & 15)] = 0;
    }
    __syncthreads();
    f32x4 o[2];
    o[0] = o[1] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int st = 0; st < NS; ++st)
#pragma unroll
        for (int h = 0; h < 3; ++h) {
            const uint4 tv = *(const uint4 *)&ts[h][r][32 * st + 8 * g];
#pragma unroll
            for (int q = 0; q < 2; ++q) o[q] = mfma16x16x32(bv[st][q], tv, o[q]);
        }
    if (mine) {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t v = (&y.x)[j];
            w[j] = (uint32_t)f32_to_bf16_rne(bits_f32(v << 16) + o[j >> 1][2 * (j & 1)]) |
                   (uint32_t)f32_to_bf16_rne(bits_f32(v & 0xFFFF0000u) + o[j >> 1][2 * (j & 1) + 1]) << 16;
        }
        *(uint4 *)(out + m * ld_out + col) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

}  // namespace

AdapterPlan plan_adapter(int64_t M, int64_t N, int64_t K, int64_t R, int64_t slots) {
    AdapterPlan p{};
    p.row_blocks = (M + kBlockRows - 1) / kBlockRows;
    const int64_t n = std::min<int64_t>(M, kBlockRows);
    // items of a block, at most: a part item for each adapter and for rows without one
    p.items = (int)std::min<int64_t>(n, n / 16 + std::min<int64_t>(n, slots + 1));
    p.rank_tiles = R <= 16 ? 1 : (R <= 32 ? 2 : 4);
    p.rank_chunks = (int)((R + 16 * p.rank_tiles - 1) / (16 * p.rank_tiles));
    // K ranges: one 128-element tile a wave while that fills the chip, longer ones for
    // many rows
    const int64_t KT = K / 128, groups = (M + 15) / 16 * p.rank_chunks;
    int64_t blocks = std::max<int64_t>(1, std::min<int64_t>((KT + kDownWaves - 1) / kDownWaves, 1024 / groups));
    if (groups < 64 && blocks > 4) blocks = (blocks + 7) / 8 * 8;
    p.tiles_per_split = (int)((KT + blocks - 1) / blocks);
    if (groups >= 64) {  // (a range of many rows' x is not shared: whole rounds of the waves)
        p.tiles_per_split = (p.tiles_per_split + kDownWaves - 1) / kDownWaves * kDownWaves;
        blocks = (KT + p.tiles_per_split - 1) / p.tiles_per_split;
    }
    p.splits = (int)((KT + p.tiles_per_split - 1) / p.tiles_per_split);
    p.range_blocks = (int)blocks;
    p.col_blocks = (int)((N + 64 * kUpWaves - 1) / (64 * kUpWaves));
    if (p.col_blocks > 4) p.col_blocks = (p.col_blocks + 7) / 8 * 8;
    // One launch: while A's part is 80 KB at most (N = 2560, one row, us: R = 16, K = 2560 6.6, two
    // launches 8.1; K = 5120, N = 5120 9.4 and 8.0; R = 32, K = 1280 6.6 and 8.5, K = 2560 8.9 and
    // 8.9) and the chip holds the workgroups at once (R = 16, K = 640, N = 5120: 16 adapters 5.2
    // and 8.1, 32 adapters, which are 320 workgroups, 9.6 and 8.8).
    p.one_launch = R <= 32 && 16 * p.rank_tiles * K <= 40960 &&
                   p.row_blocks * p.items * ((N + kOneColumns - 1) / kOneColumns) <= 256;
    p.workspace_bytes = kCounterBytes + (size_t)p.row_blocks * p.items * sizeof(Item) + (size_t)p.splits * M * R * 4;
    return p;
}

namespace {

// Both launches for blocks of rows that they take: the two are in stream order, so every
// stretch of rows may use the same workspace.
hipError_t launch_two(const AdapterPlan &p, const void *base, int64_t ld_base, const void *x, const void *a,
                      const void *b, const int32_t *rows, const float *scales, void *out, int64_t ld_out, int64_t M,
                      int64_t N, int64_t K, int R, int slots, void *workspace, hipStream_t stream) {
    const int64_t row_blocks = (M + kBlockRows - 1) / kBlockRows;
    Item *table = (Item *)ws_partials(workspace);
    float *part = (float *)(table + row_blocks * p.items);
    const dim3 down((uint32_t)(row_blocks * p.items * p.rank_chunks * p.range_blocks));
#define SVQ_DOWN(RT)                                                                                                 \
    hipLaunchKernelGGL((adapter_down_kernel<RT>), down, dim3(64 * kDownWaves), 0, stream, (const uint16_t *)x,       \
                       (const uint16_t *)a, rows, table, part, M, (int)K, R, slots, p.rank_chunks, p.range_blocks,   \
                       p.tiles_per_split)
    if (p.rank_tiles == 1) SVQ_DOWN(1);
    else if (p.rank_tiles == 2) SVQ_DOWN(2);
    else SVQ_DOWN(4);
#undef SVQ_DOWN
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const dim3 up((uint32_t)(row_blocks * p.items * p.col_blocks));
#define SVQ_UP(NS)                                                                                                  \
    hipLaunchKernelGGL((adapter_up_kernel<NS>), up, dim3(64 * kUpWaves), 0, stream, (const uint16_t *)base, part,   \
                       (const uint16_t *)b, table, scales, (uint16_t *)out, M, (int)N, R, slots, ld_base, ld_out,    \
                       p.col_blocks, p.splits)
    if (R <= 32) SVQ_UP(1);
    else if (R <= 64) SVQ_UP(2);
    else if (R <= 128) SVQ_UP(4);
    else SVQ_UP(8);
#undef SVQ_UP
    return hipGetLastError();
}

}  // namespace

hipError_t launch_adapter_add(const AdapterPlan &p, const void *base, int64_t ld_base, const void *x, const void *a,
                              const void *b, const int32_t *rows, const float *scales, void *out, int64_t ld_out,
                              int64_t M, int64_t N, int64_t K, int R, int slots, void *workspace,
                              hipStream_t stream) {
    if (p.one_launch) {
        const int cols = (int)((N + kOneColumns - 1) / kOneColumns);
        const dim3 grid((uint32_t)(p.row_blocks * p.items * cols));
#define SVQ_ONE(RT)                                                                                                  \
    hipLaunchKernelGGL((adapter_one_kernel<RT>), grid, dim3(64 * kOneWaves), 0, stream, (const uint16_t *)base,      \
                       (const uint16_t *)x, (const uint16_t *)a, (const uint16_t *)b, rows, scales, (uint16_t *)out, \
                       M, (int)N, (int)K, R, slots, ld_base, ld_out, cols)
        if (R <= 16) SVQ_ONE(1);
        else SVQ_ONE(2);
#undef SVQ_ONE
        return hipGetLastError();
    }
    // a launch has fewer than 2^32 threads: the first is kept to half of that, and the second is
    // never as large (M N < 2^30)
    const int64_t most = std::max<int64_t>(1, (int64_t(1) << 31) / (64 * kDownWaves) /
                                                  ((int64_t)p.items * p.rank_chunks * p.range_blocks)) * kBlockRows;
    for (int64_t m = 0; m < M; m += most) {
        const hipError_t e = launch_two(p, (const uint16_t *)base + m * ld_base, ld_base, (const uint16_t *)x + m * K, a, b,
                                        rows + m, scales, (uint16_t *)out + m * ld_out, ld_out, std::min(M - m, most), N,
                                        K, R, slots, workspace, stream);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace svq
