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
//
// Measured (24 query heads on 4 key heads, D = 256; both launches, replayed at clocks that 0.3 s of the same
// have settled: the first launches after a pause are slower, those of 32 x 64 rows by up to a fifth):
//   1 row over 1500 tokens                       15.4 us  latency: 11.7 (lengths 0.8, shares 0.5, q 1,
//                                                         first tiles 2.4, steps and sums) and the join 4
//   5 rows over 65000                            63.8 us  the cache at 4.2 TB/s
//   32 x 4 rows over 8192, 8-bit cache          137 us    the cache at 4.0 TB/s; decoding to bf16 and the
//                                                         products' issue stand beside the loads
//   32 x 64 rows over 4096                      367 us    561 TFLOP/s. No unit is full: matrix 27% of
//                                                         their cycles, LDS 35%, vector 38%; without its
//                                                         loads 391 of then 399 us, without its products 329
//   16 x 24 rows, window 2000, D = 128, 20 heads 42 us    31 in 8 steps a workgroup between prologue and
//                                                         parts, 10 of join
#include <algorithm>
#include <cfloat>
#include <type_traits>

#include "svq_dma.h"
#include "svq_pack.h"
#include "svq_tree.h"
#include "svq_tree_sight.h"

namespace svq {

namespace {

constexpr int kStaged = 256;       // of wider ones, parents kept in LDS; the rest is read where it lies
constexpr int kEntries = 1024;     // page table entries kept in LDS
// How far (in powers of two) scores may pass the reference of the weights before it moves: weights
// up to 2^8 cost fp32 sums nothing, and sums and columns are then rescaled in few steps only.
constexpr float kSlack = 8.f;

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef int i32x2 __attribute__((ext_vector_type(2)));

// floor(n / d) for n < 2^31: n * ceil(2^(31 + L) / d) >> (31 + L) with 2^(L-1) < d <= 2^L
struct Divide {
    uint32_t magic, shift;  // shift: L - 1; d = 1 has neither

    static Divide by(uint32_t d) {
        int L = 0;
        while ((uint64_t(1) << L) < d) ++L;
        return L ? Divide{(uint32_t)(((uint64_t(1) << (31 + L)) + d - 1) / d), (uint32_t)L - 1} : Divide{0, 0};
    }
    __device__ __forceinline__ int operator()(int n) const {
        return magic ? (int)(__umulhi((uint32_t)n, magic) >> shift) : n;
    }
};

struct Side {
    const char *cache;            // keys or values of the cache
    uint32_t page, token;         // its strides in bytes
    int64_t head;
    const float *scale;
    const uint16_t *rows;         // of the chunk
    uint32_t ld;                  // in bytes
};

// A block of rows that its workgroup began and others go on with.
struct Join {
    int first, rows, head, row0;  // of the sequence: first row, number of (row, head) pairs; KV head; the block's first pair
    int more;                     // parts that follow, one a team; 0: none
};

struct Params {
    const uint16_t *q;
    int64_t ld_q;
    Side k, v;
    const int32_t *table, *lengths, *starts, *parents;
    int64_t ld_table;
    uint32_t pages, page_size;
    Divide by_page, by_group;
    int cache_tokens;             // most of a sequence: max_pages * page_size
    float scale;                  // log2(e) times the caller's: weights are powers of two
    int window, sinks;            // window <= 0: none
    uint16_t *out;
    int64_t ld_out;
    int M, S, heads, group;       // KV heads, query heads of each
    int teams, members;
    struct Join *joins;           // [team][member]
    float *parts;                 // [grid][2] blocks of sums, then of (maximum, sum)
    float2 *stats;
};

// A sequence's rows and the numbering of the tokens that they may see.
struct Sequence : Numbering {
    int first, n;      // its rows
    int cache_tiles;   // E4M3: tiles of cached tokens; the chunk's follow in tiles of their own
    int tiles;
    int blocks, runs;  // blocks of rows; times that a team takes as many as it has members

    __device__ __forceinline__ void read(const Params &p, int s) {
        first = min(max(p.starts[s], 0), p.M);
        n = max(min(p.starts[s + 1], p.M) - first, 0);
        len = min(max(p.lengths[s], 0), p.cache_tokens);
    }
    template <bool E4M3, int ROWS>
    __device__ __forceinline__ void count(const Params &p) {
        Numbering::count(p.window, p.sinks);
        cache_tiles = (cached + kTile - 1) / kTile;
        tiles = E4M3 ? cache_tiles + (n + kTile - 1) / kTile : (cached + n + kTile - 1) / kTile;
        blocks = (n * p.group + ROWS - 1) / ROWS;
        runs = ((uint32_t)blocks + p.members - 1) / p.members;
    }
    __device__ __forceinline__ int steps(const Params &p) const { return p.heads * runs * tiles; }
};

// In LDS the 16-byte chunks of a tile's row stand at other places, by the row's number, so
// that what is read at once lies in different banks: the 16 rows of a score's operand at one
// column; of a transposed read of bf16, 8 rows and two neighbouring chunks; of codes, one
// chunk of rows 0 .. 7 and 16 .. 23. The row's lowest bits are in the address already where a
// row is shorter than the 16 chunks that the banks hold.
template <int CHUNKS, bool CODES>
__device__ __forceinline__ int swizzle(int row) {
    if constexpr (!CODES && CHUNKS >= 16) return (row & 7) << 1 | ((row >> 3) & 1);
    else if constexpr (!CODES) return ((row >> 1) & 3) << 1 | ((row >> 3) & 1);
    else if constexpr (CHUNKS >= 16) return (row & 7) | ((row >> 3 ^ row >> 4) & 1) << 3;
    else if constexpr (CHUNKS == 8) return ((row >> 1) & 3) | ((row >> 3 ^ row >> 4) & 1) << 2;
    else return ((row >> 2) & 1) | ((row >> 3 ^ row >> 4) & 1) << 1;
}

// What absent tokens are loaded from.
__device__ __attribute__((aligned(16))) const uint4 kZeros[32] = {};

// 16 bytes a lane from memory into LDS, lane i's at lds + 16 i. (Not counted by the compiler,
// which would wait for all loads in flight before each read of LDS: the waits are explicit.
// Reads of other places may pass it; barriers, which are volatile too, may not.)
__device__ __forceinline__ void load_to_lds(uint64_t from, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" : : "v"(from), "s"(lds) : "m0");
}

// Eight E4M3 codes as bf16 (exact).
__device__ __forceinline__ uint4 decode8(uint32_t a, uint32_t b) {
    return make_uint4(e4m3_pair_scaled<false>(a, 1.f), e4m3_pair_scaled<true>(a, 1.f), e4m3_pair_scaled<false>(b, 1.f),
                      e4m3_pair_scaled<true>(b, 1.f));
}

// The largest over the four 16-lane rows of a wave, for each lane of a row.
__device__ __forceinline__ float rows4_max(float v) {
    auto a = __builtin_amdgcn_permlane16_swap(f32_bits(v), f32_bits(v), false, false);
    v = fmaxf(bits_f32(a[0]), bits_f32(a[1]));
    auto b = __builtin_amdgcn_permlane32_swap(f32_bits(v), f32_bits(v), false, false);
    return fmaxf(bits_f32(b[0]), bits_f32(b[1]));
}

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// exp2(m - top) for a reference m <= top; no weight has been seen below -inf
__device__ __forceinline__ float decay(float m, float top) { return exp2_fast(m - (top == -INFINITY ? 0.f : top)); }

// A value that all lanes hold, in a scalar register.
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// The same value, computed from again where it is used: what is made of lane numbers would
// otherwise be kept across the loop over tiles, in memory where registers are short, and
// reading it back there would wait for all tiles in flight.
__device__ __forceinline__ int fresh(int v) {
    asm volatile("" : "+v"(v));
    return v;
}

// The kernel's arguments, read from memory again where this is called: kept in scalar
// registers throughout, they would push others (and those vector registers) out.
__device__ __forceinline__ const Params &arguments() {
    auto a = (const __attribute__((address_space(4))) Params *)__builtin_amdgcn_kernarg_segment_ptr();
    asm volatile("" : "+s"(a));
    return *(const Params *)a;
}

// Sums of the lanes up to each.
template <int CTRL, int ROWS>
__device__ __forceinline__ int add_dpp(int v) {
    return v + __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xF, false);
}
__device__ __forceinline__ int wave_scan(int v) {
    v = add_dpp<0x111, 0xF>(v);  // row_shr 1, 2, 4, 8
    v = add_dpp<0x112, 0xF>(v);
    v = add_dpp<0x114, 0xF>(v);
    v = add_dpp<0x118, 0xF>(v);
    v = add_dpp<0x142, 0xA>(v);  // lane 15 of the row before, to rows 1 and 3
    return add_dpp<0x143, 0xC>(v);  // lane 31 to rows 2 and 3
}

// The steps are shared as `q` for every team and one more for the first `r`.
struct Shares {
    uint32_t q, r;
    __device__ __forceinline__ int begin(int team) const { return (int)(q * team + min((uint32_t)team, r)); }
    __device__ __forceinline__ int team_of(uint32_t step) const {
        const uint32_t head = (q + 1) * r;
        return (int)(step < head ? step / (q + 1) : r + (step - head) / q);
    }
};

// Waits until at most PER * n loads are in flight, n <= MOST.
template <int PER, int MOST>
__device__ __forceinline__ void wait_parts(int n) {
    if constexpr (MOST == 0) wait_vmcnt<0>();
    else if (n >= MOST) wait_vmcnt<PER * MOST>();
    else wait_parts<PER, MOST - 1>(n);
}

// D elements a head; WR groups of waves over rows, RT 16-row tiles each; WK waves a group,
// which share a tile's tokens for the scores, and the columns for the sums: each key and each
// value is read from LDS once a group, and a wave's sums stay in D / 16 / WK * RT quads of
// registers. (32 x 64 rows at D = 256, then 399 us: 8 groups of one wave 401 to 408, 4 waves of
// 512 registers 456, half of the waves half a step behind the others 399 for 392 without; 32 rows
// as one group of two tiles, 4 waves, 165 us for 148 with 8-bit codes.)
template <int D, bool E4M3, int RT, int WR, int WK>
struct Shape {
    static constexpr int kWaves = WR * WK, kThreads = 64 * kWaves;
    static constexpr int kRows = 16 * RT * WR;
    static constexpr int kBlocks = kTile / 16 / WK;           // 16-token blocks of a tile that a wave weighs
    static constexpr int kPart = kTile * D * (E4M3 ? 1 : 2);  // bytes of a tile's keys, or values
    // Places for keys, and for values: a tile is worked on while the next is on its way (four
    // places of parts under 32 KiB: 151 us for 147 with 8-bit codes, 44.8 for 43.2 at D = 128)
    static constexpr int kSlots = 2;
    static constexpr int kArea = 2 * kSlots * kPart;
    // groups of operands read from LDS before their use: as registers allow
    static constexpr int kAhead = D * RT >= 512 ? 3 : 4;
    static constexpr int kOdd = 2 * kRows * D / 8;            // two bits each: infinities and NaN that rows see
    static constexpr int kWeights = kRows * kTile * 2;
    static constexpr int kRefs = kRows * WK * 4;
    static constexpr int kLds = kArea + kWeights + kRefs + kRows * 8 + kStaged * 4 + kEntries * 4 + kSlots * 16 + 256 + kOdd;
    static_assert(kLds <= 160 * 1024, "a compute unit's LDS");
};

template <int D, bool E4M3, int RT, int WR, int WK>
__global__ __launch_bounds__((64 * WR * WK), 1) void attend_kernel(const Params) {
    const Params &p = arguments();
    using Z = Shape<D, E4M3, RT, WR, WK>;
    constexpr int NB = Z::kBlocks, C = D / 32, MINE = D / 16 / WK, SLOTS = Z::kSlots, kAhead = Z::kAhead;
    // keys of SLOTS tiles, values of as many; or one tile of bf16 beside an 8-bit cache
    __shared__ __attribute__((aligned(256))) char lds[Z::kLds];
    uint2 *const weights = (uint2 *)(lds + Z::kArea);                  // [row tile][block][lane]
    float *const refs = (float *)(lds + Z::kArea + Z::kWeights);       // [wave of a group][row]
    uint64_t *const masks = (uint64_t *)(lds + Z::kArea + Z::kWeights + Z::kRefs);
    int *const staged = (int *)(masks + Z::kRows);
    int *const entries = staged + kStaged;
    uint64_t *const seen = (uint64_t *)(entries + kEntries);  // of the tiles in LDS, which tokens are there
    int *const scratch = (int *)(seen + 2 * SLOTS);
    uint32_t *const odd = (uint32_t *)(scratch + 64);  // [infinity, -infinity (NaN: both)][row][D / 32]
    const uint32_t area = lds_addr(lds);

    const int lane = threadIdx.x & 63, wave = wave_id(), tid = threadIdx.x;
    const int wr = wave / WK, wk = wave % WK;
    const int col = lane & 15, quad = lane >> 4;

    // ---- this team's steps, of all sequences' in order ----
    const int w = xcd_contiguous(blockIdx.x, p.teams * p.members);
    const int team = (uint32_t)w / p.members, member = w - team * p.members;
    Sequence sq;
    Shares shares;
    int seq, seq_at, used;  // the sequence of the first step, the steps before it; teams with any
    {
        const int per = (p.S + Z::kThreads - 1) / Z::kThreads;
        const int s0 = min(tid * per, p.S), s1 = min(s0 + per, p.S);
        Sequence each;
        int sum = 0;
        bool bad = false;
        for (int s = s0; s < s1; ++s) {
            each.read(p, s);
            each.count<E4M3, Z::kRows>(p);
            sum += each.steps(p);
            bad |= p.starts[s + 1] < p.starts[s];
        }
        const int run = wave_scan(sum);
        if (lane == 63) scratch[wave] = run;
        // (sequences that share rows may have more steps than the host has counted: none is taken)
        bad = __syncthreads_or(bad);
        int before = run - sum, total = 0;
#pragma unroll
        for (int i = 0; i < Z::kWaves; ++i) {
            if (i < wave) before += scratch[i];
            total += scratch[i];
        }
        total = bad ? 0 : uniform(total);
        used = min(p.teams, total);
        if (team >= used) {
            if (tid == 0) p.joins[w].more = 0;
            return;
        }
        shares.q = (uint32_t)total / used;
        shares.r = total - shares.q * used;
        const int x0 = shares.begin(team);
        if (before <= x0 && x0 < before + sum) {
            int s = s0;
            while (per > 1) {
                each.read(p, s);
                each.count<E4M3, Z::kRows>(p);
                const int st = each.steps(p);
                if (x0 < before + st) break;
                before += st;
                ++s;
            }
            scratch[16] = s;
            scratch[17] = before;
            scratch[18] = each.first;
            scratch[19] = each.n;
            scratch[20] = each.len;
        }
        __syncthreads();
        seq = uniform(scratch[16]);
        seq_at = uniform(scratch[17]);
        sq.first = uniform(scratch[18]);
        sq.n = uniform(scratch[19]);
        sq.len = uniform(scratch[20]);
        sq.count<E4M3, Z::kRows>(p);
    }
    const int end = shares.begin(team + 1);
    int x = shares.begin(team);
    Join join = {};

    while (x < end) {
        const Params &p = arguments();
        while (x >= seq_at + sq.steps(p)) {
            seq_at += sq.steps(p);
            sq.read(p, ++seq);
            sq.count<E4M3, Z::kRows>(p);
        }
        const int unit = (uint32_t)(x - seq_at) / (uint32_t)sq.tiles;
        const int t0 = x - seq_at - unit * sq.tiles, t1 = min(sq.tiles, t0 + end - x);
        const int h = (uint32_t)unit / (uint32_t)sq.runs, block = (unit - h * sq.runs) * p.members + member;
        x += t1 - t0;
        if (block >= sq.blocks) continue;
        const int rows = sq.n * p.group;  // (host: M * H < 2^31)
        const int row0 = block * Z::kRows;
        auto node_of = [&](const Params &p, int r) { return p.by_group(r); };
        auto head_of = [&](const Params &p, int r, int node) { return h * p.group + r - node * p.group; };

        // ---- q; the parents; the pages of the first tiles ----
        uint4 qf[RT][C];
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
            const int r = row0 + (wr * RT + rt) * 16 + col, node = node_of(p, r);
            // elements that a lane's keys hold: 8 of every 32, or 16 codes of every 64
            const uint4 *src = (const uint4 *)(p.q + (int64_t)(sq.first + node) * p.ld_q + (int64_t)head_of(p, r, node) * D);
#pragma unroll
            for (int c = 0; c < C; ++c)
                qf[rt][c] = r < rows ? src[E4M3 ? 8 * (c / 2) + 2 * quad + c % 2 : 4 * c + quad] : make_uint4(0, 0, 0, 0);
        }
        float own = p.scale, ks, vs = 1.f;
        if (!(own > 0.f)) {
            // a scale that is not positive goes into q, as -1 or 0: the largest score is then the largest
            // product's (and 0 times an infinity is NaN)
            const float by = own < 0.f ? -1.f : own == 0.f ? 0.f : 1.f;
            auto scaled = [&](uint32_t x) { return pack_bf16(bits_f32(x << 16) * by, bits_f32(x & 0xFFFF0000u) * by); };
#pragma unroll
            for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                for (int c = 0; c < C; ++c)
                    qf[rt][c] = make_uint4(scaled(qf[rt][c].x), scaled(qf[rt][c].y), scaled(qf[rt][c].z), scaled(qf[rt][c].w));
            own = own < 0.f ? -own : own == 0.f ? 1.f : own;
        }
        ks = own;
        if (E4M3) {
            if (p.k.scale) {
                // (a product that fp32 does not hold is not 0: what is masked, -inf, would be NaN)
                ks *= p.k.scale[h];
                ks = ks < FLT_MIN ? FLT_MIN : ks;
            }
            if (p.v.scale) vs = p.v.scale[h];
        }
        const int cut = E4M3 ? min(t1, sq.cache_tiles) : t1;  // tiles past it hold the chunk's rows alone
        const int32_t *const parents = p.parents ? p.parents + sq.first : nullptr;
        // pages in use, counted without a gap between the first tokens' and the window's
        const int sink_pages = sq.sinks > 0 ? p.by_page(sq.sinks - 1) + 1 : 0;
        const int page_gap = p.by_page(sq.from) - sink_pages;
        const Divide by_page = p.by_page;
        auto page_number = [&](int u, int page) { return u < sq.sinks ? page : page - page_gap; };
        int entry0 = 0, entry1 = 0;  // those whose table entries LDS holds
        bool all_entries = false;    // LDS holds those of all tiles that follow
        auto look_up = [&](int base) {
            if (all_entries || base >= sq.cached) return;
            const int last = min(base + kTile, sq.cached) - 1;
            if (page_number(last, by_page(sq.position(last))) < entry1) return;
            __syncthreads();
            const Params &p = arguments();
            const int32_t *table = p.table + (int64_t)seq * p.ld_table;
            const int most = min(cut * kTile, sq.cached) - 1;
            entry0 = page_number(base, p.by_page(sq.position(base)));
            entry1 = page_number(most, p.by_page(sq.position(most))) + 1;
            all_entries = entry1 <= entry0 + kEntries;
            entry1 = min(entry1, entry0 + kEntries);
            for (int i = fresh(tid); i < entry1 - entry0; i += Z::kThreads) {
                const int c = entry0 + i;
                entries[i] = table[c < sink_pages ? c : c + page_gap];
            }
            __syncthreads();
        };
        __syncthreads();  // the last unit's reads of LDS are done
        uint64_t *const lines = (uint64_t *)staged;  // of each node, itself and its ancestors
        if (parents && (p.window > 0 || t1 * kTile > sq.cached)) {
            if (sq.n > kNodes) {
                for (int i = tid; i < min(sq.n, kStaged); i += Z::kThreads) staged[i] = parents[i];
            } else if (wave == 0) {
                // twice as far up in every round
                int up = lane < sq.n ? parents[lane] : -1;
                if (up >= lane) up = -1;
                uint64_t line = 1ull << lane;
                for (int far = 1; far < sq.n; far *= 2) {
                    const int from = up < 0 ? lane : up;
                    const uint64_t more = __shfl((unsigned long long)line, from);
                    const int next = __shfl(up, from);
                    if (up >= 0) line |= more;
                    up = up < 0 ? -1 : next;
                }
                lines[lane] = line;
            }
        }
        auto parent_of = [&](int i) {
            const int up = i < kStaged ? staged[i] : parents[i];
            return up >= 0 && up < i ? up : -1;
        };

        // Weights are 2^(score - reference), and a row's reference the same for all of its group's
        // waves: the smallest whole number not below a score that has passed the one before by
        // kSlack (2^kSlack is nothing to fp32 sums; what is whole rescales bf16 weights exactly).
        f32x4 acc[RT][MINE];        // columns 16 MINE wk and on
        float top[RT], sum[RT];     // reference; sum of this wave's weights
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
            top[rt] = -INFINITY;
            sum[rt] = 0.f;
#pragma unroll
            for (int d = 0; d < MINE; ++d) acc[rt][d] = f32x4{0.f, 0.f, 0.f, 0.f};
        }

        // Where the tokens of a tile lie: lane i finds token base + i; kZeros for none. Returns
        // the bits of those that are there.
        uint64_t ka = 0, va = 0;
        const uint64_t k_cache = (uint64_t)(p.k.cache + h * p.k.head), v_cache = (uint64_t)(p.v.cache + h * p.v.head);
        // (of the chunk's rows as if they began at token 0)
        auto rows_from = [&](const Side &x) {
            return (uint64_t)(x.rows + (int64_t)h * D) + ((int64_t)sq.first - sq.cached) * (int64_t)x.ld;
        };
        const uint64_t k_rows = rows_from(p.k), v_rows = rows_from(p.v);
        const uint32_t pages = p.pages, page_size = p.page_size, k_page = p.k.page, k_token = p.k.token, v_page = p.v.page,
                       v_token = p.v.token;
        auto locate = [&](int base, int limit) {
            const int u = base + fresh(lane), last = min(limit, sq.cached);
            const int uc = min(u, max(last, 1) - 1);  // (a tile of the chunk's rows alone reads any entry)
            const int pos = sq.position(uc), page = by_page(pos);
            const uint32_t entry = (uint32_t)entries[base < last ? page_number(uc, page) - entry0 : 0];
            const uint32_t in = (uint32_t)pos - page * page_size;
            bool there = u < last && entry < pages;
            ka = there ? k_cache + (uint64_t)entry * k_page + (uint64_t)in * k_token : (uint64_t)kZeros;
            va = there ? v_cache + (uint64_t)entry * v_page + (uint64_t)in * v_token : (uint64_t)kZeros;
            if (base + kTile > last && last < limit) {
                const Params &p = arguments();
                const bool row = u >= last && u < limit;
                ka = row ? k_rows + (uint64_t)(uint32_t)u * p.k.ld : ka;
                va = row ? v_rows + (uint64_t)(uint32_t)u * p.v.ld : va;
                there |= row;
            }
            return __ballot(there);
        };
        // A tile's rows of BYTES bytes into LDS, in pieces of 1 KiB that the waves share: this
        // wave's i-th. (Its rows are the first piece's with other bits, and the swizzle is linear.)
        auto place = [&](auto row_bytes) {
            constexpr int BYTES = decltype(row_bytes)::value, CHUNKS = BYTES / 16, kPieces = kTile * BYTES / 1024;
            const int row = wave * (kPieces > Z::kWaves ? kPieces / Z::kWaves : 1) * (64 / CHUNKS) + lane / CHUNKS;
            return make_int2(row * 4, (lane % CHUNKS ^ swizzle<CHUNKS, BYTES == D>(row)) * 16);
        };
        auto fill_piece = [&](auto row_bytes, int2 at, uint64_t from, uint32_t to, int i) {
            constexpr int BYTES = decltype(row_bytes)::value, CHUNKS = BYTES / 16, kPieces = kTile * BYTES / 1024;
            constexpr int kMine = kPieces > Z::kWaves ? kPieces / Z::kWaves : 1;
            if (kPieces < Z::kWaves && wave >= kPieces) return;
            const int row = at.x + i * (64 / CHUNKS) * 4, chunk = at.y ^ swizzle<CHUNKS, BYTES == D>(i * (64 / CHUNKS)) * 16;
            const uint32_t lo = (uint32_t)__builtin_amdgcn_ds_bpermute(row, (int)from);
            const uint32_t hi = (uint32_t)__builtin_amdgcn_ds_bpermute(row, (int)(from >> 32));
            load_to_lds(((uint64_t)hi << 32 | lo) + chunk, to + (wave * kMine + i) * 1024);
        };
        auto fill = [&](auto row_bytes, int2 at, uint64_t from, uint32_t to) {
            constexpr int kPieces = kTile * decltype(row_bytes)::value / 1024;
#pragma unroll
            for (int i = 0; i < (kPieces > Z::kWaves ? kPieces / Z::kWaves : 1); ++i) fill_piece(row_bytes, at, from, to, i);
        };
        constexpr int kMine = Z::kPart / 1024 > Z::kWaves ? Z::kPart / 1024 / Z::kWaves : 1;  // pieces a wave loads at once
        constexpr std::integral_constant<int, D * (E4M3 ? 1 : 2)> cache_row{};
        constexpr std::integral_constant<int, 2 * D> bf16_row{};
        const int2 cache_place = place(cache_row);

        const int edge = sq.edge(p.window, sq.n);  // (tiles that every row sees whole need no mask)
        auto make_masks = [&](int base, uint64_t there) {
            const Params &p = arguments();
            for (int i = fresh(tid); i < Z::kRows; i += Z::kThreads) {
                const int r = row0 + i, node = node_of(p, r);
                uint64_t bits = 0;
                if (r < rows)
                    bits = there & (!parents         ? sq.chain(p.window, p.sinks, base, node)
                                    : sq.n <= kNodes ? sq.path(p.window, p.sinks, base, lines[node])
                                                     : sq.walk(p.window, p.sinks, base, node, parent_of));
                masks[i] = bits;
            }
        };

        f32x4 sc[RT][NB];
        uint2 wt[RT][kTile / 16];  // bf16 weights of tokens 4 quad .. 4 quad + 3 of each block
        float mine[RT];            // the reference of its own
        // scores of this wave's blocks of tokens, from keys in LDS
        auto scores = [&](auto codes, uint32_t keys, auto between) {
            constexpr bool CODES = decltype(codes)::value;
            constexpr int BYTES = CODES ? D : 2 * D, CHUNKS = BYTES / 16;
            // chunk c of a row is at c ^ swizzle: the lane's own bits are in the address from the
            // start, those of an operand are changed or added to it
            constexpr bool WIDE = CODES || E4M3;  // a lane's two operands are neighbours
            const int l = fresh(lane), col = l & 15, quad = l >> 4;
            const int row = wk * NB * 16 + col;
            const lds_u8 *const from = lds_opaque(keys + row * BYTES + ((WIDE && !CODES ? 2 * quad : quad) ^ swizzle<CHUNKS, CODES>(row)) * 16);
            auto chunk_at = [&](int b, int chunk) {
                constexpr int kMixed = CHUNKS < 16 ? CHUNKS - 1 : 15;
                return lds_ld16((const lds_u8 *)((uint32_t)(uintptr_t)from ^ (chunk & kMixed) * 16) +
                                (chunk & ~kMixed) * 16 + b * 16 * BYTES);
            };
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) sc[rt][b] = f32x4{0.f, 0.f, 0.f, 0.f};
            // groups of one operand (of codes two), the blocks in turn, read kAhead groups before
            // their use
            constexpr int PER = CODES ? 2 : 1, GROUPS = NB * C / PER;
            auto read = [&](int g) {
                const int b = g % NB, c = g / NB * PER;
                // (codes: the next block's swizzle differs in its highest bit)
                if constexpr (CODES) return chunk_at(b, 2 * c ^ (b % 2 ? (CHUNKS < 16 ? CHUNKS / 2 : 8) : 0));
                else return chunk_at(b, WIDE ? 4 * (c & ~1) + c % 2 : 4 * c);
            };
            uint4 raw[kAhead + 1];
#pragma unroll
            for (int g = 0; g < kAhead && g < GROUPS; ++g) raw[g] = read(g);
#pragma unroll
            for (int g = 0; g < GROUPS; ++g) {
                if (g + kAhead < GROUPS) raw[(g + kAhead) % (kAhead + 1)] = read(g + kAhead);
                __builtin_amdgcn_sched_barrier(0);
                const uint4 r = raw[g % (kAhead + 1)];
#pragma unroll
                for (int e = 0; e < PER; ++e) {
                    const uint4 kf = !CODES ? r : e ? decode8(r.z, r.w) : decode8(r.x, r.y);
#pragma unroll
                    for (int rt = 0; rt < RT; ++rt)
                        sc[rt][g % NB] = mfma16x16x32(kf, qf[rt][g / NB * PER + e], sc[rt][g % NB]);
                }
                between(g, GROUPS);
                __builtin_amdgcn_sched_barrier(0);
            }
        };
        // Their weights, for all waves of the group: summed in fp32, rounded to bf16 (off by 2^-8 of each
        // at most) for a second product at one matrix instruction's cost, since values are bf16. Results
        // are then 0.0023 to 0.0024 of their norm off, of which the result's own rounding is 0.0017. As two
        // bf16 parts, which keep 16 bits, they would be 0.0017 off, but double the second product: 5 rows over
        // 65000 66.5 us for 64.4, 8-bit batch 152 for 139, window 45.2 for 41.7, 4 x 200 rows at D = 128 93 for
        // 83, and blocks of 128 rows at D = 256 have no LDS for them.
        auto weigh = [&](float to2, bool masked) {
            const int l = fresh(lane), col = l & 15, quad = l >> 4;
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
                if (masked) {
                    const uint32_t *mask = (const uint32_t *)(masks + (wr * RT + rt) * 16 + col);
#pragma unroll
                    for (int b = 0; b < NB; ++b) {
                        const uint32_t bits = mask[(wk * NB + b) / 2] >> (16 * ((wk * NB + b) & 1) + 4 * quad);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (!(bits >> i & 1)) sc[rt][b][i] = -INFINITY;
                    }
                }
                float high = -INFINITY;
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int i = 0; i < 4; ++i) high = fmaxf(high, sc[rt][b][i]);
                high = rows4_max(high) * to2;
                mine[rt] = top[rt];
                if (__any(high > top[rt] + kSlack)) {
                    mine[rt] = high > top[rt] + kSlack ? ceilf(high) : top[rt];
                    sum[rt] *= decay(top[rt], mine[rt]);
                }
                const float ref = mine[rt] == -INFINITY ? 0.f : mine[rt];
                float add = 0.f;
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    float e[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) add += e[i] = exp2_fast(__builtin_fmaf(sc[rt][b][i], to2, -ref));
                    weights[((wr * RT + rt) * (kTile / 16) + wk * NB + b) * 64 + l] =
                        make_uint2(pack_bf16(e[0], e[1]), pack_bf16(e[2], e[3]));
                }
                sum[rt] += add;
                if (quad == 0) refs[wk * Z::kRows + (wr * RT + rt) * 16 + col] = mine[rt];
            }
        };
        // the weights of all blocks, and one reference for all
        auto meet = [&]() {
            const int l = fresh(lane), col = l & 15;
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
                float each[WK], high = -INFINITY;
                bool other = false;
#pragma unroll
                for (int v = 0; v < WK; ++v) {
                    each[v] = refs[v * Z::kRows + (wr * RT + rt) * 16 + col];
                    high = fmaxf(high, each[v]);
                    other |= each[v] != top[rt];
                }
#pragma unroll
                for (int b = 0; b < kTile / 16; ++b) wt[rt][b] = weights[((wr * RT + rt) * (kTile / 16) + b) * 64 + l];
                if (__any(other)) {
                    sum[rt] *= decay(mine[rt], high);
                    const float down = decay(top[rt], high);
#pragma unroll
                    for (int d = 0; d < MINE; ++d) acc[rt][d] *= down;
                    top[rt] = high;
#pragma unroll
                    for (int b = 0; b < kTile / 16; ++b) {
                        const float by = decay(each[b / NB], high);
                        uint2 &x = wt[rt][b];
                        x = make_uint2(pack_bf16(bits_f32(x.x << 16) * by, bits_f32(x.x & 0xFFFF0000u) * by),
                                       pack_bf16(bits_f32(x.y << 16) * by, bits_f32(x.y & 0xFFFF0000u) * by));
                    }
                }
            }
        };
        // The weighted values of a tile in LDS: this wave's columns. A transposed read gives a lane 4
        // tokens of its column (4 quad .. 4 quad + 3 of a block), of codes those of two blocks.
        auto add_values = [&](auto codes, uint32_t values, auto between) {
            constexpr bool CODES = decltype(codes)::value;
            constexpr int BYTES = CODES ? D : 2 * D, CHUNKS = BYTES / 16, kMixed = CHUNKS < 16 ? CHUNKS - 1 : 15;
            const int l = fresh(lane), col = l & 15, quad = l >> 4;
            const int row = 4 * quad + (CODES ? (col >> 1 & 3) + (col >> 3 << 4) : col >> 2);
            const int first = wk * MINE * (CODES ? 1 : 2);  // chunk of the wave's first column
            const uint32_t from = (uint32_t)(uintptr_t)lds_opaque(
                values + row * BYTES + (((CODES ? 0 : col >> 1 & 1) ^ swizzle<CHUNKS, CODES>(row)) ^ (first & kMixed)) * 16 +
                (first & ~kMixed) * 16 + (col & 1) * 8);
            auto read = [&](int b, int chunk) {
                const lds_u8 *const at = (const lds_u8 *)(from ^ (chunk & kMixed) * 16) + (chunk & ~kMixed) * 16 + b * 16 * BYTES;
                if constexpr (CODES)
                    return __builtin_amdgcn_ds_read_tr8_b64_v2i32((__attribute__((address_space(3))) i32x2 *)at);
                else
                    return __builtin_bit_cast(
                        i32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4 *)at));
            };
            constexpr int GROUPS = kTile / 32 * MINE, READS = CODES ? 1 : 2;
            struct Raw {
                i32x2 x[READS];
            };
            auto read_group = [&](int g) {
                const int b = g / MINE * 2, d = g % MINE;
                Raw r;
#pragma unroll
                for (int k = 0; k < READS; ++k) r.x[k] = read(b + k, CODES ? d : 2 * d);
                return r;
            };
            Raw raw[kAhead + 1];
#pragma unroll
            for (int g = 0; g < kAhead && g < GROUPS; ++g) raw[g] = read_group(g);
            meet();
#pragma unroll
            for (int g = 0; g < GROUPS; ++g) {
                if (g + kAhead < GROUPS) raw[(g + kAhead) % (kAhead + 1)] = read_group(g + kAhead);
                __builtin_amdgcn_sched_barrier(0);
                const int b = g / MINE * 2, d = g % MINE;
                const Raw &r = raw[g % (kAhead + 1)];
                uint4 a;
                if constexpr (CODES) a = decode8(r.x[0][0], r.x[0][1]);
                else a = make_uint4(r.x[0][0], r.x[0][1], r.x[READS - 1][0], r.x[READS - 1][1]);
#pragma unroll
                for (int rt = 0; rt < RT; ++rt)
                    acc[rt][d] = mfma16x16x32(
                        a, make_uint4(wt[rt][b].x, wt[rt][b].y, wt[rt][b + 1].x, wt[rt][b + 1].y), acc[rt][d]);
                between(g, GROUPS);
                __builtin_amdgcn_sched_barrier(0);
            }
        };
        // In a tile that some row does not see whole, 0 * infinity must not reach the rows that do
        // not see it: infinities and NaN become zeros there, and the rows that see one get it when
        // their sums are done.
        bool any_odd = false;
        auto set_apart = [&](auto codes, char *values) {
            constexpr bool CODES = decltype(codes)::value;
            constexpr int BYTES = CODES ? D : 2 * D, CHUNKS = BYTES / 16;
            auto each = [&](auto found) {
                const uint32_t *const words = (const uint32_t *)values;
#pragma unroll 2
                for (int i = fresh(tid); i < kTile * BYTES / 4; i += Z::kThreads) {
                    const uint32_t x = words[i];
                    if (CODES) {  // 0x7F and 0xFF: all ones but the sign
                        const uint32_t y = ~x & 0x7F7F7F7Fu;
                        if ((y - 0x01010101u) & ~y & 0x80808080u) found(i, x);
                    } else if ((x & 0x7F80u) == 0x7F80u || (x & 0x7F800000u) == 0x7F800000u) {
                        found(i, x);
                    }
                }
            };
            bool here = false;
            each([&](int, uint32_t) { here = true; });
            if (!__syncthreads_or(here)) return;
            if (!any_odd)
                for (int i = fresh(tid); i < Z::kOdd / 4; i += Z::kThreads) odd[i] = 0;
            any_odd = true;
            __syncthreads();
            each([&](int word, uint32_t x) {
                constexpr int kBits = CODES ? 8 : 16;
#pragma unroll 1
                for (int e = 0; e < 32 / kBits; ++e) {
                    const uint32_t y = x >> (kBits * e) & ((1u << kBits) - 1);
                    if (CODES ? (y & 0x7F) != 0x7F : (y & 0x7F80) != 0x7F80) continue;
                    const int i = word / 4, row = i / CHUNKS;
                    const int d = (((i % CHUNKS) ^ swizzle<CHUNKS, CODES>(row)) * 4 + word % 4) * (32 / kBits) + e;
                    const bool none = CODES || (y & 0x7F);
#pragma unroll 1
                    for (int r = 0; r < Z::kRows; ++r) {
                        if (!(masks[r] >> row & 1)) continue;
                        if (none || !(y >> 15)) atomicOr(&odd[(r * D + d) / 32], 1u << (d & 31));
                        if (none || y >> 15) atomicOr(&odd[((Z::kRows + r) * D + d) / 32], 1u << (d & 31));
                    }
                    if (CODES) values[word * 4 + e] = 0;
                    else ((uint16_t *)values)[word * 2 + e] = 0;
                }
            });
            __syncthreads();
        };

        // ---- the cache's tiles (bf16: and the chunk's rows) ----
        // A tile is two halves of a step: scores and weights, then values. Keys and values have
        // SLOTS places each, and a place is filled again as soon as its tile is done with, by loads
        // between the matrix instructions. At the barrier before a tile's first half its keys are
        // there, at the one before the second its values and all weights.
        const int count = cut - t0;
        const int limit = E4M3 ? sq.cached : sq.cached + sq.n;
        auto nothing = [](int, int) {};  // (beside the chunk's tiles nothing is loaded)
        auto keys_at = [&](int i) { return area + (i & (SLOTS - 1)) * Z::kPart; };
        auto values_at = [&](int i) { return area + (SLOTS + (i & (SLOTS - 1))) * Z::kPart; };
        uint32_t masked = 0;  // of the tiles in LDS, which need a mask: bit i & (2 SLOTS - 1)
        auto find = [&](int i) {
            const int base = (t0 + i) * kTile;
            look_up(base);
            const uint64_t there = locate(base, limit);
            if (tid == 0) seen[i & (2 * SLOTS - 1)] = there;
            const uint32_t bit = 1u << (i & (2 * SLOTS - 1));
            masked = sq.needs_mask(edge, base, there) ? masked | bit : masked & ~bit;
        };
        // loads of a part, one piece at a time between `steps` groups of matrix instructions
        auto loading = [&](bool any, uint64_t from, uint32_t to) {
            return [&, any, from, to](int step, int steps) {
#pragma unroll
                for (int i = 0; i < kMine; ++i)
                    if (any && step == i * steps / kMine) fill_piece(cache_row, cache_place, from, to, i);
            };
        };
        auto first_half = [&](int i, auto between) {
            const bool mask = masked >> (i & (2 * SLOTS - 1)) & 1;
            scores(std::bool_constant<E4M3>{}, keys_at(i), between);
            weigh(ks, mask);
        };
        auto prepare = [&](int i) {  // masks of a tile that needs them, for both groups of waves
            if (masked >> (i & (2 * SLOTS - 1)) & 1) {
                make_masks((t0 + i) * kTile, seen[i & (2 * SLOTS - 1)]);
                lds_barrier();
            }
        };
        auto sift = [&](int i) {
            if (masked >> (i & (2 * SLOTS - 1)) & 1) set_apart(std::bool_constant<E4M3>{}, lds + (values_at(i) - area));
        };
        if (count > 0) {
            uint64_t vb = 0;
            // (the compiler knows of q's loads but not of the tiles': without this it would wait for
            // all of them at q's first use, in every step)
            wait_vmcnt<0>();
            // keys of SLOTS tiles ahead, values of SLOTS - 1
            for (int i = 0; i < min(SLOTS, count); ++i) {
                if (i) fill(cache_row, cache_place, vb, values_at(i - 1));
                find(i);
                vb = va;
                fill(cache_row, cache_place, ka, keys_at(i));
            }
            if (count < SLOTS) fill(cache_row, cache_place, vb, values_at(count - 1));
            for (int i = 0; i < count; ++i) {
                const int left = count - 1 - i;
                // loaded since its keys: values from its own on, keys of the tiles after it
                if (left >= SLOTS - 1) wait_vmcnt<2 * (SLOTS - 1) * kMine>();
                else wait_parts<kMine, 2 * SLOTS>(2 * left + 1);
                lds_barrier();
                prepare(i);
                first_half(i, loading(left >= SLOTS - 1, vb, values_at(i + SLOTS - 1)));
                if (left >= SLOTS) find(i + SLOTS);
                vb = va;
                if (left >= SLOTS - 1) wait_vmcnt<2 * (SLOTS - 1) * kMine>();
                else wait_parts<kMine, 2 * SLOTS>(2 * left);
                lds_barrier();
                sift(i);
                add_values(std::bool_constant<E4M3>{}, values_at(i), loading(left >= SLOTS, ka, keys_at(i)));
            }
        }
        // ---- beside an 8-bit cache, the chunk's rows ----
        if constexpr (E4M3) {
#pragma unroll
            for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                for (int d = 0; d < MINE; ++d) acc[rt][d] *= vs;
            for (int t = max(t0, sq.cache_tiles); t < t1; ++t) {
                const int base = sq.cached + (t - sq.cache_tiles) * kTile;
                const uint64_t there = locate(base, sq.cached + sq.n);
                const int2 bf16_place = place(bf16_row);
                lds_barrier();
                fill(bf16_row, bf16_place, ka, area);
                fill(bf16_row, bf16_place, va, area + kTile * 2 * D);
                make_masks(base, there);
                wait_vmcnt<0>();
                lds_barrier();
                scores(std::false_type{}, area, nothing);
                weigh(own, true);
                lds_barrier();
                set_apart(std::false_type{}, lds + kTile * 2 * D);
                add_values(std::false_type{}, area + kTile * 2 * D, nothing);
            }
        }

        // ---- the waves' sums of weights ----
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) sum[rt] = rows4_sum(sum[rt]);
        lds_barrier();
        {
            const int l = fresh(lane), row = wr * RT * 16 + (l & 15);
#pragma unroll
            for (int rt = 0; rt < RT; ++rt)
                if (l < 16) refs[wk * Z::kRows + row + rt * 16] = sum[rt];
            lds_barrier();
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
                sum[rt] = 0.f;
#pragma unroll
                for (int v = 0; v < WK; ++v) sum[rt] += refs[v * Z::kRows + row + rt * 16];
            }
        }

        // ---- out, or a part of it ----
        const Params &po = arguments();
        const bool whole = t0 == 0 && t1 == sq.tiles;
        const int64_t slot = 2 * (int64_t)w + (t0 == 0);
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
            const int l = fresh(lane), quad = l >> 4, i = (wr * RT + rt) * 16 + (l & 15), r = row0 + i, node = node_of(po, r);
            if (r >= rows) continue;
            if (whole) {
                uint16_t *o = po.out + (int64_t)(sq.first + node) * po.ld_out + (int64_t)head_of(po, r, node) * D +
                              16 * MINE * wk + 4 * quad;
                const float inv = sum[rt] == 0.f ? 0.f : 1.f / sum[rt];
#pragma unroll
                for (int d = 0; d < MINE; ++d) {
                    const f32x4 a = acc[rt][d] * inv;
                    *(uint2 *)(o + 16 * d) = make_uint2(pack_bf16(a[0], a[1]), pack_bf16(a[2], a[3]));
                }
            } else {
                float *o = po.parts + (slot * Z::kRows + i) * D + 16 * MINE * wk + 4 * quad;
#pragma unroll
                for (int d = 0; d < MINE; ++d) *(f32x4 *)(o + 16 * d) = acc[rt][d];
                if (wk == 0 && quad == 0) po.stats[slot * Z::kRows + i] = make_float2(top[rt], sum[rt]);
            }
        }
        if (any_odd) {
            // infinities and NaN that rows see
            __threadfence_block();
            __syncthreads();
            for (int i = tid; i < Z::kRows * D; i += Z::kThreads) {
                const int at = i / D, d = i % D, r = row0 + at, node = node_of(po, r);
                auto is = [&](int kind) { return odd[(kind * Z::kRows * D + i) / 32] >> (d & 31) & 1; };
                const bool up = is(0), down = is(1);
                if (r >= rows || !(up || down)) continue;
                const float add = up && down ? NAN : up ? INFINITY : -INFINITY;
                if (whole) {
                    uint16_t *o = po.out + (int64_t)(sq.first + node) * po.ld_out + (int64_t)head_of(po, r, node) * D + d;
                    *o = f32_to_bf16_rne(bits_f32((uint32_t)*o << 16) + add);
                } else {
                    po.parts[(slot * Z::kRows + at) * D + d] += add;
                }
            }
        }
        if (t0 == 0 && t1 < sq.tiles)
            // the parts that follow: one a team, up to the one with this unit's last step
            join = Join{sq.first, rows, h, row0, shares.team_of(x - t1 + sq.tiles - 1) - team};
    }
    if (tid == 0) arguments().joins[w] = join;
}

// Joins a block of rows whose first part is workgroup x's. A row takes D / 4 lanes of kSplit
// waves (few rows have many parts).
template <int D, int ROWS>
struct JoinShape {
    static constexpr int kLanes = D / 4, kSplit = ROWS >= 64 ? 1 : 64 / ROWS;
    static constexpr int kRows = 64 / kLanes * (4 / kSplit);  // of a workgroup of 4 waves
};

template <int D, int ROWS>
__global__ __launch_bounds__(256) void join_kernel(const Params p) {
    using Z = JoinShape<D, ROWS>;
    const int w = blockIdx.x;
    const Join j = p.joins[w];
    if (j.more == 0) return;
    constexpr int L = Z::kLanes, RW = Z::kSplit, kBatch = RW > 1 ? 16 : 8;
    const int lane = threadIdx.x & 63, wave = wave_id(), l = lane % L;
    __shared__ float2 stat[4][64 / L];
    __shared__ f32x4 vals[4][64];
    const int i = blockIdx.y * Z::kRows + wave / RW * (64 / L) + lane / L, r = j.row0 + i;
    float top = -INFINITY, sum = 0.f;
    f32x4 acc = f32x4{0.f, 0.f, 0.f, 0.f};
    // (rows past the last have a place in every part too: what it holds goes nowhere)
    auto slot = [&](int part) { return (part == 0 ? 2 * (int64_t)w + 1 : 2 * ((int64_t)w + part * p.members)) * ROWS + i; };
    // L parts at a time: lane l's statistics, then the values by their weights, the first ones
    // loaded beside the statistics
    for (int p0 = wave % RW; p0 <= j.more; p0 += L * RW) {
        const int part = p0 + l * RW, count = min(L, (j.more - p0) / RW + 1);
        float2 st = make_float2(-INFINITY, 0.f);
        if (part <= j.more) st = p.stats[slot(part)];
        f32x4 v[kBatch];
        auto load = [&](int k0) {
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                v[k] = f32x4{0.f, 0.f, 0.f, 0.f};
                if (k0 + k < count) v[k] = *(const f32x4 *)(p.parts + slot(p0 + (k0 + k) * RW) * D + l * 4);
            }
        };
        load(0);
        float high = fmaxf(top, st.x);
#pragma unroll
        for (int d = 1; d < L; d <<= 1) high = fmaxf(high, __shfl_xor(high, d));
        const float b = decay(st.x, high), a = decay(top, high);
        float add = st.y * b;
#pragma unroll
        for (int d = 1; d < L; d <<= 1) add += __shfl_xor(add, d);
        sum = sum * a + add;
        top = high;
        acc *= a;
        for (int k0 = 0; k0 < count; k0 += kBatch) {
            if (k0) load(k0);
#pragma unroll
            for (int k = 0; k < kBatch; ++k) acc += v[k] * (L == 64 ? bits_f32(__builtin_amdgcn_readlane(f32_bits(b), k0 + k)) : __shfl(b, k0 + k, L));
        }
    }
    if constexpr (RW > 1) {
        if (l == 0) stat[wave][lane / L] = make_float2(top, sum);
        vals[wave][lane] = acc;
        __syncthreads();
        if (wave % RW) return;
        float high = -INFINITY;
#pragma unroll
        for (int v = 0; v < RW; ++v) high = fmaxf(high, stat[wave + v][lane / L].x);
        sum = 0.f;
        acc = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int v = 0; v < RW; ++v) {
            const float2 st = stat[wave + v][lane / L];
            const float b = decay(st.x, high);
            sum += st.y * b;
            acc += vals[wave + v][lane] * b;
        }
    }
    if (r < j.rows) {
        const f32x4 o = acc * (sum == 0.f ? 0.f : 1.f / sum);
        const int node = p.by_group(r);
        *(uint2 *)(p.out + (int64_t)(j.first + node) * p.ld_out + (int64_t)(j.head * p.group + r - node * p.group) * D + l * 4) =
            make_uint2(pack_bf16(o[0], o[1]), pack_bf16(o[2], o[3]));
    }
}

}  // namespace

AttendPlan plan_tree_attention(int64_t M, int64_t S, int64_t H, int64_t KVH, int64_t D, int num_cus) {
    AttendPlan p{};
    // Blocks as tall as a sequence's rows on average, up to 128 (of two that hold them the lower):
    // 6 rows as a block of 16 / 32 take 16.6 / 17.6 us; 24 rows as 32 / 64: 154 / 156; 120 rows as
    // 32 / 64 / 128: 61 / 48.6 / 48.5; 384 rows: 914 / 553 / 381 (the tokens go through LDS once a block).
    const int64_t rows = (M * (H / KVH) + S - 1) / S;
    p.block_rows = rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 64 ? 64 : 128;
    // A sequence's blocks of rows read the same tokens: up to 8 workgroups take them side by side, so
    // that the caches keep them (3 blocks: 370 us for 396, 0.6 GB of memory traffic for 1.6). Of the
    // numbers of members that leave fewest idle the largest.
    const int64_t blocks = (rows + p.block_rows - 1) / p.block_rows;
    p.members = 1;
    for (int64_t m = 2; m <= 8 && m <= blocks; ++m) {
        auto places = [&](int64_t k) { return (blocks + k - 1) / k * k; };
        if (places(m) <= places(p.members)) p.members = (int)m;
    }
    p.teams = std::max(1, num_cus / p.members);
    const size_t groups = (size_t)p.teams * p.members;
    p.workspace_bytes = kCounterBytes + ((groups * sizeof(Join) + 255) & ~(size_t)255) + 2 * groups * p.block_rows * (D * 4 + 8);
    return p;
}

namespace {

template <int D, bool E4M3, int RT, int WR, int WK>
hipError_t launch_shape(const Params &p, hipStream_t stream) {
    using Z = Shape<D, E4M3, RT, WR, WK>;
    auto kernel = attend_kernel<D, E4M3, RT, WR, WK>;
    hipLaunchKernelGGL(kernel, dim3(p.teams * p.members), dim3(Z::kThreads), 0, stream, p);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((join_kernel<D, Z::kRows>), dim3(p.teams * p.members, Z::kRows / JoinShape<D, Z::kRows>::kRows), dim3(256), 0, stream, p);
    return hipGetLastError();
}

template <int D, bool E4M3>
hipError_t launch_rows(const Params &p, int block_rows, hipStream_t stream) {
    switch (block_rows) {
    case 16: return launch_shape<D, E4M3, 1, 1, 4>(p, stream);
    case 32: return launch_shape<D, E4M3, 1, 2, 4>(p, stream);
    case 64: return launch_shape<D, E4M3, 2, 2, 4>(p, stream);
    default: return launch_shape<D, E4M3, 2, 4, 2>(p, stream);
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
    auto side = [&](const void *cache, const int64_t *st, const float *by, const void *rows, int64_t ld) {
        return Side{(const char *)cache, (uint32_t)(st[0] * size), (uint32_t)(st[1] * size), st[2] * size, by,
                    (const uint16_t *)rows, (uint32_t)(ld * 2)};
    };
    p.k = side(c.k, c.k_strides, c.k_scale, k, ld_k);
    p.v = side(c.v, c.v_strides, c.v_scale, v, ld_v);
    p.table = c.page_table;
    p.ld_table = c.ld_table;
    p.lengths = c.lengths;
    p.starts = starts;
    p.parents = parents;
    p.pages = (uint32_t)c.pages;
    p.page_size = (uint32_t)c.page_size;
    p.by_page = Divide::by(p.page_size);
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
    p.by_group = Divide::by(p.group);
    p.teams = plan.teams;
    p.members = plan.members;
    const size_t groups = (size_t)plan.teams * plan.members;
    p.joins = (Join *)ws_partials(workspace);
    p.parts = (float *)((char *)p.joins + ((groups * sizeof(Join) + 255) & ~(size_t)255));
    p.stats = (float2 *)(p.parts + 2 * groups * plan.block_rows * D);
    switch (D) {
    case 64: return launch_type<64>(p, plan.block_rows, e4m3, stream);
    case 128: return launch_type<128>(p, plan.block_rows, e4m3, stream);
    default: return launch_type<256>(p, plan.block_rows, e4m3, stream);
    }
}

}  // namespace svq
