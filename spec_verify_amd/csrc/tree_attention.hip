// Attention of the rows of a verify chunk to a paged cache and to their own paths in the
// tree of drafts (svq_tree_attention):
//
//   out[m][h] = sum_j w_j v_j / sum_j w_j,   w_j = exp(scale * q[m][h] . k_j)
//
// over the tokens j that the row sees. One pass over the tokens: scores of a tile of 64,
// the running maximum and sum of the weights, the weighted sum of values rescaled when the
// maximum moves.
//
// The H / KVH heads of a group read the same keys, so a sequence's rows are (node, head of
// the group) pairs, in blocks of 16 to 128. With tokens as the matrix instructions' rows
// and the block's rows as their columns (scores = K Q^T, sums = V^T W^T), a lane holds
// scores of one row only, its weights are already the second product's operand, and the
// row's maximum scales its own accumulators: nothing moves between lanes but the maximum.
//
// The tokens that a sequence's rows may see are numbered without gaps: first ones (sinks),
// the window's, and then (bf16 cache; after an 8-bit cache in tiles of their own) the
// chunk's rows. A tile in which some row does not see some token gets a 64-bit mask a row.
//
// Work is shared by steps (one tile of tokens for one block of rows), not by sequences:
// every workgroup finds its equal part of all steps from the lengths, so sequences of very
// different lengths keep the chip equally busy. A block of rows that ends up in several
// workgroups is joined by a second launch from its parts' maxima, sums and fp32 values.
#include <algorithm>

#include "svq_tree.h"

namespace svq {

namespace {

constexpr int kTile = 64;          // tokens in a tile
constexpr int kStaged = 1024;      // parents kept in LDS; of wider trees the rest is read where it lies

typedef short s16x4 __attribute__((ext_vector_type(4)));

struct Side {
    const char *cache;            // keys or values of the cache
    int64_t page, token, head;    // its strides in bytes
    const float *scale;
    const uint16_t *rows;         // of the chunk
    int64_t ld;
};

struct Params {
    const uint16_t *q;
    int64_t ld_q;
    Side k, v;
    const int32_t *table, *lengths, *starts, *parents;
    int64_t ld_table;
    uint32_t pages, page_size, page_magic, page_shift;
    int cache_tokens;             // most of a sequence: max_pages * page_size
    float scale;                  // log2(e) times the caller's: weights are powers of two
    int window, sinks;            // window <= 0: none
    uint16_t *out;
    int64_t ld_out;
    int M, S, heads, group;       // KV heads, query heads of each
    int grid;
    int4 *joins;                  // [grid]: sequence, head, block of rows, parts that follow the first
    float *parts;                 // [grid][2] blocks of sums, then of (maximum, sum)
    float2 *stats;
};

// floor(n / page_size) for n < 2^31
__device__ __forceinline__ uint32_t page_of(const Params &p, uint32_t n) {
    return p.page_size == 1 ? n : __umulhi(n, p.page_magic) >> p.page_shift;
}

// A sequence's rows and the numbering of the tokens that they may see.
struct Sequence {
    int s, first, n;   // its rows
    int len;           // cached tokens
    int sinks, from;   // tokens 0 .. sinks - 1 of the cache come first, then those from `from` on
    int cached;        // how many that are
    int cache_tiles;   // E4M3: tiles of cached tokens; the chunk's follow in tiles of their own
    int tiles;
    int blocks;

    template <bool E4M3>
    __device__ __forceinline__ void load(const Params &p, int seq, int block_rows) {
        s = seq;
        first = min(max(p.starts[s], 0), p.M);
        n = max(min(p.starts[s + 1], p.M) - first, 0);
        len = min(max(p.lengths[s], 0), p.cache_tokens);
        sinks = 0;
        from = 0;
        if (p.window > 0) {
            sinks = min(max(p.sinks, 0), len);
            // the first row, at position len, sees the window's oldest token
            from = max((int)max((int64_t)len - p.window + 1, (int64_t)0), sinks);
            if (from > len) from = len;
        }
        cached = sinks + len - from;
        cache_tiles = (int)(((int64_t)cached + kTile - 1) / kTile);
        tiles = E4M3 ? cache_tiles + (int)(((int64_t)n + kTile - 1) / kTile)
                     : (int)(((int64_t)cached + n + kTile - 1) / kTile);
        blocks = (int)(((int64_t)n * p.group + block_rows - 1) / block_rows);
    }
    __device__ __forceinline__ int64_t steps(const Params &p) const { return (int64_t)p.heads * blocks * tiles; }
};

// Chunks of 16 bytes of a tile's row change places by the row's number, so that the 16
// rows that a read takes at one column lie in different banks, and so do the 8 rows of
// half a transposed read (which takes pairs of chunks).
template <int D>
__device__ __forceinline__ int swizzle(int row) {
    if constexpr (D == 64) return ((row >> 1) & 3) << 1 | ((row >> 3) & 1);
    else return (row & 7) << 1 | ((row >> 3) & 1);
}

__device__ __forceinline__ f32x4 mfma16x16x16(s16x4 a, s16x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x16bf16_1k(a, b, c, 0, 0, 0);
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    const f32x2 v = {a, b};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
}

// The largest over the four 16-lane rows of a wave, for each lane of a row.
__device__ __forceinline__ float rows4_max(float v) {
    auto a = __builtin_amdgcn_permlane16_swap(f32_bits(v), f32_bits(v), false, false);
    v = fmaxf(bits_f32(a[0]), bits_f32(a[1]));
    auto b = __builtin_amdgcn_permlane32_swap(f32_bits(v), f32_bits(v), false, false);
    return fmaxf(bits_f32(b[0]), bits_f32(b[1]));
}

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// exp2(m - top) for a maximum m <= top; no weight has been seen below -inf
__device__ __forceinline__ float decay(float m, float top) { return exp2_fast(m - (top == -INFINITY ? 0.f : top)); }

// D elements a head; RT 16-row tiles a wave, WR waves over rows, WK waves over tokens.
template <int D, bool E4M3, int RT, int WR, int WK>
struct Shape {
    static constexpr int kWaves = WR * WK, kThreads = 64 * kWaves;
    static constexpr int kRows = 16 * RT * WR;
    static constexpr int kBlocks = kTile / 16 / WK;   // 16-token blocks of a tile that a wave takes
    static constexpr int kRowBytes = D * 2;
    static constexpr int kTileBytes = kTile * kRowBytes;
    static constexpr int kLds = 2 * kTileBytes + kRows * 8 + kStaged * 4 + 256;
};

template <int D, bool E4M3, int RT, int WR, int WK>
__global__ __launch_bounds__((64 * WR * WK), 1) void attend_kernel(const Params p) {
    using Z = Shape<D, E4M3, RT, WR, WK>;
    constexpr int NB = Z::kBlocks, C = D / 32, DT = D / 16;
    __shared__ __attribute__((aligned(256))) char lds[Z::kLds];
    char *const lds_k = lds, *const lds_v = lds + Z::kTileBytes;
    uint64_t *const masks = (uint64_t *)(lds + 2 * Z::kTileBytes);
    int *const staged = (int *)(masks + Z::kRows);
    int64_t *const scratch = (int64_t *)(staged + kStaged);

    const int lane = threadIdx.x & 63, wave = wave_id(), tid = threadIdx.x;
    const int wr = wave / WK, wk = wave % WK;
    const int col = lane & 15, quad = lane >> 4;

    // ---- this workgroup's steps, of all sequences' in order ----
    const int w = xcd_contiguous(blockIdx.x, p.grid);
    Sequence sq;
    int64_t total, mine, seq_at;  // all steps, those before this thread's sequences, those before sq
    {
        const int per = (p.S + Z::kThreads - 1) / Z::kThreads;
        const int s0 = min(tid * per, p.S), s1 = min(s0 + per, p.S);
        int64_t sum = 0;
        for (int s = s0; s < s1; ++s) {
            sq.load<E4M3>(p, s, Z::kRows);
            sum += sq.steps(p);
        }
        int64_t run = sum;
        for (int d = 1; d < 64; d <<= 1) {
            const int64_t up = __shfl_up(run, d);
            if (lane >= d) run += up;
        }
        if (lane == 63) scratch[wave] = run;
        __syncthreads();
        mine = run - sum;
        total = 0;
        for (int i = 0; i < Z::kWaves; ++i) {
            if (i < wave) mine += scratch[i];
            total += scratch[i];
        }
        __syncthreads();
        const int parts = (int)min((int64_t)p.grid, total);
        if (w >= parts) {
            if (tid == 0) p.joins[w] = make_int4(0, 0, 0, 0);
            return;
        }
        const int64_t x0 = total * w / parts;
        if (mine <= x0 && x0 < mine + sum) {
            int64_t at = mine;
            int s = s0;
            for (;; ++s) {
                sq.load<E4M3>(p, s, Z::kRows);
                const int64_t st = sq.steps(p);
                if (x0 < at + st) break;
                at += st;
            }
            scratch[0] = s;
            scratch[1] = at;
        }
        __syncthreads();
        sq.load<E4M3>(p, (int)scratch[0], Z::kRows);
        seq_at = scratch[1];
    }
    const int parts = (int)min((int64_t)p.grid, total);
    const int64_t end = total * (w + 1) / parts;
    int64_t x = total * w / parts;
    int4 join = make_int4(0, 0, 0, 0);

    while (x < end) {
        while (x >= seq_at + sq.steps(p)) {
            seq_at += sq.steps(p);
            sq.load<E4M3>(p, sq.s + 1, Z::kRows);
        }
        const int64_t unit = (x - seq_at) / sq.tiles;
        const int t0 = (int)(x - seq_at - unit * sq.tiles);
        const int t1 = (int)min((int64_t)sq.tiles, t0 + (end - x));
        const int h = (int)(unit / sq.blocks), block = (int)(unit % sq.blocks);
        const int rows = sq.n * p.group;  // (host: M * H < 2^31)
        const int row0 = block * Z::kRows;

        // ---- q, and each lane's rows ----
        uint4 qf[RT][C];
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
            const int r = row0 + (wr * RT + rt) * 16 + col;
            const int node = r / p.group, head = h * p.group + r % p.group;
            const uint4 *src = (const uint4 *)(p.q + (int64_t)(sq.first + node) * p.ld_q + (int64_t)head * D) + quad;
#pragma unroll
            for (int c = 0; c < C; ++c) qf[rt][c] = r < rows ? src[4 * c] : make_uint4(0, 0, 0, 0);
        }
        float ks = p.scale, vs = 1.f;
        if (E4M3) {
            if (p.k.scale) ks *= p.k.scale[h];
            if (p.v.scale) vs = p.v.scale[h];
        }
        const int32_t *parents = p.parents ? p.parents + sq.first : nullptr;
        __syncthreads();  // the last unit's reads of LDS are done
        if (parents)
            for (int i = tid; i < min(sq.n, kStaged); i += Z::kThreads) staged[i] = parents[i];
        auto parent_of = [&](int i) {
            const int up = i < kStaged ? staged[i] : parents[i];
            return up >= 0 && up < i ? up : -1;
        };

        f32x4 acc[RT][DT];
        float top[RT], sum[RT];
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
            top[rt] = -INFINITY;
            sum[rt] = 0.f;
#pragma unroll
            for (int dt = 0; dt < DT; ++dt) acc[rt][dt] = f32x4{0.f, 0.f, 0.f, 0.f};
        }

        for (int t = t0; t < t1; ++t) {
            const bool own = E4M3 && t >= sq.cache_tiles;  // a tile of the chunk's rows alone
            if (E4M3 && t == sq.cache_tiles)
                // what stands so far is in units of the cache's scale
#pragma unroll
                for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                    for (int dt = 0; dt < DT; ++dt) acc[rt][dt] *= vs;

            // ---- where the tile's tokens lie: lane i finds token i ----
            const int base = own ? sq.cached + (t - sq.cache_tiles) * kTile : t * kTile;
            const int limit = own ? sq.cached + sq.n : E4M3 ? sq.cached : sq.cached + sq.n;
            const char *ka = nullptr, *va = nullptr;
            {
                const int64_t u = (int64_t)base + lane;
                if (u < limit) {
                    if (u < sq.cached) {
                        const int pos = u < sq.sinks ? (int)u : (int)u - sq.sinks + sq.from;
                        const uint32_t at = page_of(p, pos);
                        const uint32_t page = (uint32_t)p.table[(int64_t)sq.s * p.ld_table + at];
                        const int in = pos - (int)(at * p.page_size);
                        if (page < p.pages) {
                            ka = p.k.cache + page * p.k.page + in * p.k.token + h * p.k.head;
                            va = p.v.cache + page * p.v.page + in * p.v.token + h * p.v.head;
                        }
                    } else {
                        const int64_t m = sq.first + (u - sq.cached);
                        ka = (const char *)(p.k.rows + m * p.k.ld + (int64_t)h * D);
                        va = (const char *)(p.v.rows + m * p.v.ld + (int64_t)h * D);
                    }
                }
            }
            const uint64_t there = __ballot(ka != nullptr);
            // tiles that every row sees whole need no mask
            bool masked = ~there != 0 || base + kTile > sq.cached;
            if (p.window > 0 && (int64_t)base < (int64_t)sq.sinks + sq.n - 1 && base + kTile > sq.sinks) masked = true;

            // ---- the tile into LDS ----
            __syncthreads();
            auto fill = [&](const char *addr, char *to) {
                constexpr int kChunks = Z::kRowBytes / 16;             // 16-byte chunks of a row in LDS
                constexpr int kRowsAtOnce = 64 / kChunks > 0 ? 64 / kChunks : 1;
                constexpr int kSteps = kTile / kRowsAtOnce / Z::kWaves;
#pragma unroll
                for (int i = 0; i < kSteps; ++i) {
                    const int row = (wave * kSteps + i) * kRowsAtOnce + lane / kChunks;
                    const int chunk = (lane % kChunks) ^ swizzle<D>(row);
                    const uint64_t a = (uint64_t)__shfl((long long)(uint64_t)addr, row);
                    uint4 v = make_uint4(0, 0, 0, 0);
                    if (a) {
                        if (E4M3 && !own) {
                            const uint2 c = *(const uint2 *)(a + chunk * 8);
                            v = make_uint4(e4m3_pair_scaled<false>(c.x, 1.f), e4m3_pair_scaled<true>(c.x, 1.f),
                                           e4m3_pair_scaled<false>(c.y, 1.f), e4m3_pair_scaled<true>(c.y, 1.f));
                        } else {
                            v = *(const uint4 *)(a + chunk * 16);
                        }
                    }
                    *(uint4 *)(to + row * Z::kRowBytes + (lane % kChunks) * 16) = v;
                }
            };
            fill(ka, lds_k);
            fill(va, lds_v);
            if (masked) {
                for (int i = tid; i < Z::kRows; i += Z::kThreads) {
                    const int r = row0 + i, node = r / p.group;
                    uint64_t bits = 0;
                    if (r < rows) {
                        auto below = [](int64_t n) { return n <= 0 ? 0 : n >= 64 ? ~0ull : (1ull << n) - 1; };
                        // positions of the row, and the distance a path's token may have
                        int depth = node;
                        if (parents && p.window > 0) {
                            depth = 0;
                            for (int i = parent_of(node); i >= 0; i = parent_of(i)) ++depth;
                        }
                        const int64_t at = (int64_t)sq.len + depth;
                        bits = below((int64_t)sq.cached - base);
                        if (p.window > 0) {
                            const int64_t old = sq.sinks + max(at - p.window + 1 - sq.from, (int64_t)0);
                            bits &= ~below(old - base) | below((int64_t)sq.sinks - base);
                        }
                        const int far = p.window > 0 ? p.window : INT32_MAX;
                        const int64_t sunk = p.window > 0 ? (int64_t)p.sinks - sq.len : 0;  // depths below are sinks
                        const int64_t off = (int64_t)sq.cached - base;  // bit of the sequence's first row
                        if (!parents) {
                            // nodes 0 .. node, those nearer than `far` or of depths that are sinks
                            const uint64_t line = below(off + node + 1) & ~below(off);
                            bits |= line & (~below(off + (int64_t)node - far + 1) | below(off + sunk));
                        } else {
                            int d = 0;
                            for (int i = node; i >= 0 && off + i >= 0; i = parent_of(i), ++d)
                                if (off + i < 64 && (d < far || depth - d < sunk)) bits |= 1ull << (off + i);
                        }
                        bits &= there;
                    }
                    masks[i] = bits;
                }
            }
            __syncthreads();

            // ---- scores of this wave's blocks of tokens ----
            f32x4 sc[RT][NB];
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                const int row = (wk * NB + b) * 16 + col;
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) sc[rt][b] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    const uint4 kf = *(const uint4 *)(lds_k + row * Z::kRowBytes + (((4 * c + quad) ^ swizzle<D>(row)) * 16));
#pragma unroll
                    for (int rt = 0; rt < RT; ++rt) sc[rt][b] = mfma16x16x32(kf, qf[rt][c], sc[rt][b]);
                }
            }
            // ---- weights ----
            const float to2 = own ? p.scale : ks;
            uint2 wt[RT][NB];  // bf16 weights of tokens 4 quad .. 4 quad + 3 of each block
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
                uint64_t bits = ~0ull;
                if (masked) bits = masks[(wr * RT + rt) * 16 + col] >> (wk * NB * 16 + 4 * quad);
                float high = top[rt];
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float s = sc[rt][b][i] * to2;
                        if (masked && !(bits >> (16 * b + i) & 1)) s = -INFINITY;
                        sc[rt][b][i] = s;
                        high = fmaxf(high, s);
                    }
                high = rows4_max(high);
                const float safe = high == -INFINITY ? 0.f : high;
                const float down = exp2_fast(top[rt] - safe);
                top[rt] = high;
                float add = 0.f;
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    float e[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) add += e[i] = exp2_fast(sc[rt][b][i] - safe);
                    wt[rt][b] = make_uint2(pack_bf16(e[0], e[1]), pack_bf16(e[2], e[3]));
                }
                sum[rt] = sum[rt] * down + add;
#pragma unroll
                for (int dt = 0; dt < DT; ++dt) acc[rt][dt] *= down;
            }
            // ---- weighted values ----
            auto value = [&](int b, int dt) {
                const int row = (wk * NB + b) * 16 + 4 * quad + (col >> 2);
                const int chunk = (2 * dt + ((col >> 1) & 1)) ^ swizzle<D>(row);
                return __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                    (__attribute__((address_space(3))) s16x4 *)(lds_v + row * Z::kRowBytes + chunk * 16 + (col & 1) * 8));
            };
            bool rough = false;  // a value that some row does not see is infinite or NaN
            if (masked) {
                bool bad = false;
                for (int i = tid; i < Z::kTileBytes / 16; i += Z::kThreads) {
                    const uint4 v = ((const uint4 *)lds_v)[i];
                    for (uint32_t x : {v.x, v.y, v.z, v.w})
                        bad |= (x & 0x7F80u) == 0x7F80u || (x & 0x7F800000u) == 0x7F800000u;
                }
                rough = __syncthreads_or(bad);
            }
            auto finite = [](s16x4 v) {
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = (v[i] & 0x7F80) == 0x7F80 ? (short)0 : v[i];
                return v;
            };
            auto add_values = [&](auto take) {
                if constexpr (NB == 1) {
#pragma unroll
                    for (int dt = 0; dt < DT; ++dt) {
                        const s16x4 a = take(value(0, dt));
#pragma unroll
                        for (int rt = 0; rt < RT; ++rt)
                            acc[rt][dt] = mfma16x16x16(a, __builtin_bit_cast(s16x4, wt[rt][0]), acc[rt][dt]);
                    }
                } else {
#pragma unroll
                    for (int b = 0; b < NB; b += 2)
#pragma unroll
                        for (int dt = 0; dt < DT; ++dt) {
                            const uint2 a = __builtin_bit_cast(uint2, take(value(b, dt)));
                            const uint2 c = __builtin_bit_cast(uint2, take(value(b + 1, dt)));
#pragma unroll
                            for (int rt = 0; rt < RT; ++rt)
                                acc[rt][dt] = mfma16x16x32(make_uint4(a.x, a.y, c.x, c.y),
                                                           make_uint4(wt[rt][b].x, wt[rt][b].y, wt[rt][b + 1].x,
                                                                      wt[rt][b + 1].y),
                                                           acc[rt][dt]);
                        }
                }
            };
            if (!rough) {
                add_values([](s16x4 v) { return v; });
            } else {
                // finite values as ever (0 * infinity would reach the rows that do not see it); of the
                // others, how many of each kind every row sees
                add_values(finite);
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int dt = 0; dt < DT; ++dt) {
                        const s16x4 v = value(b, dt);
                        s16x4 up, down, none;
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            up[i] = v[i] == (short)0x7F80 ? (short)0x3F80 : (short)0;
                            down[i] = v[i] == (short)0xFF80 ? (short)0x3F80 : (short)0;
                            none[i] = (v[i] & 0x7FFF) > 0x7F80 ? (short)0x3F80 : (short)0;
                        }
#pragma unroll
                        for (int rt = 0; rt < RT; ++rt) {
                            const uint64_t bits = masks[(wr * RT + rt) * 16 + col] >> ((wk * NB + b) * 16 + 4 * quad);
                            s16x4 seen;
#pragma unroll
                            for (int i = 0; i < 4; ++i) seen[i] = bits >> i & 1 ? (short)0x3F80 : (short)0;
                            const f32x4 zero{0.f, 0.f, 0.f, 0.f};
                            const f32x4 nu = mfma16x16x16(up, seen, zero), nd = mfma16x16x16(down, seen, zero),
                                        nn = mfma16x16x16(none, seen, zero);
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                if (nu[i] > 0.f) acc[rt][dt][i] += INFINITY;
                                if (nd[i] > 0.f) acc[rt][dt][i] -= INFINITY;
                                if (nn[i] > 0.f) acc[rt][dt][i] = NAN;
                            }
                        }
                    }
            }
        }
        if (E4M3 && t1 <= sq.cache_tiles)
#pragma unroll
            for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                for (int dt = 0; dt < DT; ++dt) acc[rt][dt] *= vs;

        // ---- the sums of the four 16-lane rows, then of the waves over tokens ----
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) sum[rt] = rows4_sum(sum[rt]);
#pragma unroll
        for (int half = WK / 2; half >= 1; half /= 2) {
            __syncthreads();
            float *const at = (float *)lds;
            float2 *const st = (float2 *)masks;  // [waves over rows][half][16 RT], in place of masks and parents
            static_assert(WK / 2 * Z::kRows * 4 * D <= 2 * Z::kTileBytes, "parts fit the tiles");
            static_assert(WK / 2 <= 2, "statistics fit the masks and the parents");
            if (wk >= half && wk < 2 * half) {
                const int slot = wr * half + wk - half;
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) {
                    if (quad == 0) st[(slot * RT + rt) * 16 + col] = make_float2(top[rt], sum[rt]);
#pragma unroll
                    for (int dt = 0; dt < DT; ++dt) ((f32x4 *)at)[((slot * RT + rt) * DT + dt) * 64 + lane] = acc[rt][dt];
                }
            }
            __syncthreads();
            if (wk < half) {
                const int slot = wr * half + wk;
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) {
                    const float2 o = st[(slot * RT + rt) * 16 + col];
                    const float high = fmaxf(top[rt], o.x);
                    const float a = decay(top[rt], high), b = decay(o.x, high);
                    top[rt] = high;
                    sum[rt] = sum[rt] * a + o.y * b;
#pragma unroll
                    for (int dt = 0; dt < DT; ++dt)
                        acc[rt][dt] = acc[rt][dt] * a + ((f32x4 *)at)[((slot * RT + rt) * DT + dt) * 64 + lane] * b;
                }
            }
        }

        // ---- out, or a part of it ----
        const bool whole = t0 == 0 && t1 == sq.tiles;
        if (wk == 0) {
            const int64_t slot = 2 * (int64_t)w + (t0 == 0);
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
                const int i = (wr * RT + rt) * 16 + col, r = row0 + i;
                if (r >= rows) continue;
                if (whole) {
                    const int node = r / p.group, head = h * p.group + r % p.group;
                    uint16_t *o = p.out + (int64_t)(sq.first + node) * p.ld_out + (int64_t)head * D + 4 * quad;
                    const float inv = sum[rt] == 0.f ? 0.f : 1.f / sum[rt];
#pragma unroll
                    for (int dt = 0; dt < DT; ++dt) {
                        const f32x4 a = acc[rt][dt] * inv;
                        *(uint2 *)(o + 16 * dt) = make_uint2(pack_bf16(a[0], a[1]), pack_bf16(a[2], a[3]));
                    }
                } else {
                    float *o = p.parts + (slot * Z::kRows + i) * D + 4 * quad;
#pragma unroll
                    for (int dt = 0; dt < DT; ++dt) *(f32x4 *)(o + 16 * dt) = acc[rt][dt];
                    if (quad == 0) p.stats[slot * Z::kRows + i] = make_float2(top[rt], sum[rt]);
                }
            }
        }
        if (t0 == 0 && t1 < sq.tiles) {
            // the parts that follow: one a workgroup, up to the one with this unit's last step
            const int64_t last = x + sq.tiles - 1;
            const int64_t to = ((last + 1) * parts - 1) / total;
            join = make_int4(sq.s, h, block, (int)(to - w));
        }
        x += t1 - t0;
    }
    if (tid == 0) p.joins[w] = join;
}

// Joins a block of rows whose first part is workgroup x's: one row of it a workgroup.
template <int D>
__global__ __launch_bounds__(256) void join_kernel(const Params p, int block_rows) {
    const int w = blockIdx.x;
    const int4 j = p.joins[w];
    if (j.w == 0) return;
    const int lane = threadIdx.x & 63, wave = wave_id();
    const int first = min(max(p.starts[j.x], 0), p.M);
    const int n = max(min(p.starts[j.x + 1], p.M) - first, 0);
    const int i = blockIdx.y, r = j.z * block_rows + i;
    if (r >= n * p.group) return;
    __shared__ float2 stat[4];
    __shared__ float vals[4][D];
    constexpr int E = D / 64;
    // wave v takes parts v, v + 4, ...
    float top = -INFINITY, sum = 0.f, acc[E];
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
    auto slot = [&](int part) { return part == 0 ? 2 * (int64_t)w + 1 : 2 * ((int64_t)w + part); };
    for (int part = wave; part <= j.w; part += 4) {
        const int64_t at = slot(part) * block_rows + i;
        const float2 st = p.stats[at];
        const float high = fmaxf(top, st.x), a = decay(top, high), b = decay(st.x, high);
        top = high;
        sum = sum * a + st.y * b;
        const float *src = p.parts + at * D + lane * E;
        for (int e = 0; e < E; ++e) acc[e] = acc[e] * a + src[e] * b;
    }
    if (lane == 0) stat[wave] = make_float2(top, sum);
    for (int e = 0; e < E; ++e) vals[wave][lane * E + e] = acc[e];
    __syncthreads();
    if (wave) return;
    float high = -INFINITY, all = 0.f, o[E];
    for (int v = 0; v < 4; ++v) high = fmaxf(high, stat[v].x);
    for (int e = 0; e < E; ++e) o[e] = 0.f;
    for (int v = 0; v < 4; ++v) {
        const float b = decay(stat[v].x, high);
        all += stat[v].y * b;
        for (int e = 0; e < E; ++e) o[e] += vals[v][lane * E + e] * b;
    }
    const float inv = all == 0.f ? 0.f : 1.f / all;
    uint16_t *to = p.out + (int64_t)(first + r / p.group) * p.ld_out + (int64_t)(j.y * p.group + r % p.group) * D;
    for (int e = 0; e < E; ++e) to[lane * E + e] = f32_to_bf16_rne(o[e] * inv);
}

}  // namespace

AttendPlan plan_tree_attention(int64_t M, int64_t S, int64_t H, int64_t KVH, int64_t D, int num_cus) {
    AttendPlan p{};
    const int64_t rows = (M * (H / KVH) + S - 1) / S;  // of a sequence, on average
    p.block_rows = rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 64 ? 64 : 128;
    p.grid = num_cus;
    const size_t slots = 2 * (size_t)p.grid * p.block_rows;
    p.workspace_bytes = kCounterBytes + (((size_t)p.grid * 16 + 255) & ~(size_t)255) + slots * (D * 4 + 8);
    return p;
}

namespace {

template <int D, bool E4M3, int RT, int WR, int WK>
hipError_t launch_shape(const Params &p, hipStream_t stream) {
    using Z = Shape<D, E4M3, RT, WR, WK>;
    auto kernel = attend_kernel<D, E4M3, RT, WR, WK>;
    hipLaunchKernelGGL(kernel, dim3(p.grid), dim3(Z::kThreads), 0, stream, p);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(join_kernel<D>, dim3(p.grid, Z::kRows), dim3(256), 0, stream, p, Z::kRows);
    return hipGetLastError();
}

template <int D, bool E4M3>
hipError_t launch_rows(const Params &p, int block_rows, hipStream_t stream) {
    switch (block_rows) {
    case 16: return launch_shape<D, E4M3, 1, 1, 4>(p, stream);
    case 32: return launch_shape<D, E4M3, 2, 1, 4>(p, stream);
    case 64: return launch_shape<D, E4M3, 2, 2, 2>(p, stream);
    default: return launch_shape<D, E4M3, 2, 4, 1>(p, stream);
    }
}

template <int D>
hipError_t launch_type(const Params &p, int block_rows, bool e4m3, hipStream_t stream) {
    return e4m3 ? launch_rows<D, true>(p, block_rows, stream) : launch_rows<D, false>(p, block_rows, stream);
}

}  // namespace

hipError_t launch_tree_attention(const AttendPlan &plan, const void *q, int64_t ld_q, const void *k, int64_t ld_k,
                                 const void *v, int64_t ld_v, const svq_kv_cache &c, const int32_t *starts,
                                 const int32_t *parents, float scale, int window, int sinks, void *out, int64_t ld_out,
                                 int64_t M, int64_t S, int H, int KVH, int D, void *workspace, hipStream_t stream) {
    Params p{};
    const bool e4m3 = c.type == SVQ_CACHE_E4M3;
    const int64_t size = e4m3 ? 1 : 2;
    p.q = (const uint16_t *)q;
    p.ld_q = ld_q;
    p.k = Side{(const char *)c.k, c.k_strides[0] * size, c.k_strides[1] * size, c.k_strides[2] * size, c.k_scale,
               (const uint16_t *)k, ld_k};
    p.v = Side{(const char *)c.v, c.v_strides[0] * size, c.v_strides[1] * size, c.v_strides[2] * size, c.v_scale,
               (const uint16_t *)v, ld_v};
    p.table = c.page_table;
    p.ld_table = c.ld_table;
    p.lengths = c.lengths;
    p.starts = starts;
    p.parents = parents;
    p.pages = (uint32_t)c.pages;
    p.page_size = (uint32_t)c.page_size;
    // n / d = n * ceil(2^(31 + L) / d) >> (31 + L) for every n < 2^31, with 2^(L-1) < d <= 2^L
    int L = 0;
    while ((int64_t(1) << L) < c.page_size) ++L;
    if (L) {
        p.page_magic = (uint32_t)(((uint64_t(1) << (31 + L)) + c.page_size - 1) / c.page_size);
        p.page_shift = (uint32_t)(L - 1);
    }
    p.cache_tokens = (int)((int64_t)c.max_pages * c.page_size);
    p.scale = scale * 1.44269504088896340736f;
    p.window = window;
    p.sinks = sinks;
    p.out = (uint16_t *)out;
    p.ld_out = ld_out;
    p.M = (int)M;
    p.S = (int)S;
    p.heads = KVH;
    p.group = H / KVH;
    p.grid = plan.grid;
    p.joins = (int4 *)ws_partials(workspace);
    p.parts = (float *)((char *)p.joins + (((size_t)plan.grid * 16 + 255) & ~(size_t)255));
    p.stats = (float2 *)(p.parts + 2 * (size_t)plan.grid * plan.block_rows * D);
    switch (D) {
    case 64: return launch_type<64>(p, plan.block_rows, e4m3, stream);
    case 128: return launch_type<128>(p, plan.block_rows, e4m3, stream);
    default: return launch_type<256>(p, plan.block_rows, e4m3, stream);
    }
}

}  // namespace svq
