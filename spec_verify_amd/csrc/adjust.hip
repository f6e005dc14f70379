// Logits as the sampler takes them (svq_adjust_logits): penalties for the tokens of a
// sequence's history and of a row's path in the tree of drafts, biases, grammar masks.
//
// A workgroup takes a range of the vocabulary for some rows of one sequence. It counts the
// history's tokens of that range in LDS once (16384 words of 32 bits: two workgroups a compute
// unit). Then, row by row, it adds the row's path to the counts and takes the row before's out,
// and streams the row's logits past them; the next row's are loaded meanwhile.
//
// Bound by the logits' way in and out. Measured (V = 248320; replayed):
//   1 row behind 1500 tokens              6.0 us  latency of one workgroup: history, row, stores
//   128 rows of 32, histories of 8192    38.7 us  3.4 TB/s: each of the 16 ranges reads the history again,
//                                                 and has 4 rows to spread that over
//   512 rows of 8, histories of 4096    111 us    4.6 TB/s, 95% of a copy
#include <algorithm>

#include "svq_pack.h"
#include "svq_tree.h"

namespace svq {

namespace {

constexpr int kThreads = 512;
constexpr int kMostRange = 16384;                     // tokens of a workgroup's range
constexpr int kVectors = kMostRange / 8 / kThreads;   // of 8 logits, a thread's of one row
constexpr int kNodes = 64;                            // trees up to this size have their paths as bits
constexpr int kStaged = 1024;                         // of wider ones, parents kept in LDS
constexpr int kPath = 512;                            // and tokens of a path taken at a time
constexpr int kBiases = 128;                          // biases of a range kept in LDS

constexpr uint32_t kPrompt = 0x80000000u;  // occurs in the prompt
constexpr uint32_t kBiased = 0x40000000u;  // has biases
constexpr uint32_t kCount = 0x3FFFFFFFu;   // occurrences after it

struct Params {
    const uint16_t *logits;
    int64_t ld;
    uint16_t *out;
    int64_t ld_out;
    const int32_t *starts;
    svq_adjustments a;
    int64_t items;
    int M, S, V, range, ranges, groups;
};

__global__ __launch_bounds__(kThreads) void adjust_kernel(const Params p) {
    __shared__ __attribute__((aligned(16))) uint32_t table[kMostRange + 8];
    __shared__ uint32_t marks[kMostRange / 32 + 2];  // a bit for each word that is or was not zero
    __shared__ uint64_t lines[kNodes];  // of each node, itself and its ancestors
    __shared__ int nodes[kNodes];       // the nodes' inputs
    __shared__ int staged[kStaged], path[kPath], path_n, path_at;
    __shared__ int bias_token[kBiases], bias_n;  // of the range, in their order
    __shared__ float bias_value[kBiases];
    const int tid = threadIdx.x, lane = tid & 63, wave = wave_id();
    const svq_adjustments &a = p.a;
    for (int64_t item = blockIdx.x; item < p.items; item += gridDim.x) {
        const int c = (int)(item % p.ranges);
        const int g = (int)(item / p.ranges % p.groups), s = (int)(item / p.ranges / p.groups);
        const int first = min(max(p.starts[s], 0), p.M), n = max(min(p.starts[s + 1], p.M) - first, 0);
        if (g >= n) continue;
        const int v0 = c * p.range, v1 = min(v0 + p.range, p.V);
        const int end = min(v1 + 8, p.V);  // counted too: a vector of 8 may begin before v1 and end after it
        const int32_t *parents = a.parents ? a.parents + first : nullptr;
        // (a product with 1 / r instead of a quotient: one more rounding in fp32, 2^-16 of bf16's)
        const float rep = a.repetition ? a.repetition[s] : 1.f, inv = 1.f / rep;
        const float pres = a.presence ? a.presence[s] : 0.f, freq = a.frequency ? a.frequency[s] : 0.f;

        // ---- the first row's logits are on their way while the history is counted ----
        auto row_in = [&](int row) { return p.logits + (int64_t)(first + row) * p.ld; };
        auto lead_of = [&](const uint16_t *x) { return (int)((uintptr_t)x / 2 & 7); };
        // the first vector of 8 on a 16-byte line that begins in the range (a row's first may begin before it)
        auto first_vector = [&](int lead) { return (v0 + lead + (v0 ? 7 : 0)) / 8; };
        uint4 next[kVectors];
        uint32_t next_open[kVectors];  // the row's mask where its vectors begin
        auto mask_row = [&](int row) { return a.allowed && row < n ? a.mask_rows[first + row] : -1; };
        auto mask_of = [&](int mask) {
            return mask >= 0 && mask < a.masks ? (const uint32_t *)a.allowed + mask * a.ld_allowed : nullptr;
        };
        auto load = [&](int row, int mask) {
            const uint16_t *in = row_in(row);
            const uint32_t *allowed = mask_of(mask);
            const int lead = lead_of(in), j0 = first_vector(lead) + tid;
#pragma unroll
            for (int k = 0; k < kVectors; ++k) {
                const int v = 8 * (j0 + k * kThreads) - lead;
                next[k] = make_uint4(0, 0, 0, 0);
                next_open[k] = ~0u;
                if (v >= 0 && v < v1 && v + 8 <= p.V) {
                    next[k] = *(const uint4 *)(in + v);
                    if (allowed) next_open[k] = allowed[v >> 5];
                }
            }
        };
        int mask_now = mask_row(g), mask_next = mask_row(g + p.groups);
        load(g, mask_now);

        __syncthreads();
        for (int i = tid; i < (p.range + 8) / 4; i += kThreads) ((uint4 *)table)[i] = make_uint4(0, 0, 0, 0);
        for (int i = tid; i < p.range / 32 + 2; i += kThreads) marks[i] = 0;
        if (n <= kNodes) {
            if (wave == 0) {
                // twice as far up in every round
                int up = lane - 1;
                if (parents) up = lane < n ? parents[lane] : -1;
                if (up >= lane) up = -1;
                uint64_t line = 1ull << lane;
                for (int far = 1; far < n; far *= 2) {
                    const int from = up < 0 ? lane : up;
                    const uint64_t more = __shfl((unsigned long long)line, from);
                    const int next_up = __shfl(up, from);
                    if (up >= 0) line |= more;
                    up = up < 0 ? -1 : next_up;
                }
                lines[lane] = line;
                nodes[lane] = lane < n ? a.inputs[first + lane] : -1;
            }
        } else if (parents) {
            for (int i = tid; i < min(n, kStaged); i += kThreads) staged[i] = parents[i];
        }
        __syncthreads();
        // (a word's changes commute; marks are only ever set: a path's token may leave a zero behind)
        auto mark = [&](int v) {
            if (v < v0 || v >= end) return false;
            atomicOr(&marks[(v - v0) >> 5], 1u << ((v - v0) & 31));
            return true;
        };
        auto count = [&](int v, uint32_t by) {
            if (mark(v)) atomicAdd(&table[v - v0], by);
        };
        const int len = min(max(a.lengths[s], 0), a.max_history);
        const int prompt = a.prompt_lengths ? a.prompt_lengths[s] : 0;
        const int32_t *history = a.history + (int64_t)s * a.ld_history;
#pragma unroll 4
        for (int i = tid; i < len; i += kThreads) {
            const int v = history[i];
            if (i >= prompt) count(v, 1u);
            else if (mark(v)) atomicOr(&table[v - v0], kPrompt);
        }
        int64_t b0 = 0, b1 = 0;
        if (a.bias_starts) {
            b0 = min(max((int64_t)a.bias_starts[s], (int64_t)0), a.biases);
            b1 = min((int64_t)a.bias_starts[s + 1], a.biases);
            if (wave == 0) {
                int kept = 0;
                for (int64_t b = b0; b < b1; b += 64) {
                    const int v = b + lane < b1 ? a.bias_tokens[b + lane] : -1;
                    const bool here = mark(v);
                    const uint64_t all = __ballot(here);
                    const int at = kept + __popcll(all & ((1ull << lane) - 1));
                    if (here) {
                        atomicOr(&table[v - v0], kBiased);
                        if (at < kBiases) {
                            bias_token[at] = v;
                            bias_value[at] = a.bias_values[b + lane];
                        }
                    }
                    kept += __popcll(all);
                }
                if (lane == 0) bias_n = kept;
            }
        }
        // adds `by` to the counts of a row's path; large trees: a walk
        auto walk = [&](int row, uint32_t by) {
            if (!parents) {
                for (int i = tid; i <= row; i += kThreads) count(a.inputs[first + i], by);
                return;
            }
            int at = row;
            while (at >= 0) {
                __syncthreads();
                if (tid == 0) {
                    int k = 0;
                    while (at >= 0 && k < kPath) {
                        path[k++] = at;
                        const int up = at < kStaged ? staged[at] : parents[at];
                        at = up >= 0 && up < at ? up : -1;
                    }
                    path_n = k;
                    path_at = at;
                }
                __syncthreads();
                for (int i = tid; i < path_n; i += kThreads) count(a.inputs[first + path[i]], by);
                at = path_at;
            }
        };

        for (int row = g; row < n; row += p.groups) {
            // ---- this row's path in, the last one's out (barriers that wait for LDS alone: the
            // next row's logits stay on their way) ----
            lds_barrier();
            if (n <= kNodes) {
                if (wave == 0 && lines[row] >> lane & 1) count(nodes[lane], 1u);
                if (wave == 1 && row > g && lines[row - p.groups] >> lane & 1) count(nodes[lane], ~0u);
            } else {
                walk(row, 1u);
                if (row > g) walk(row - p.groups, ~0u);
            }
            uint4 x[kVectors];
            uint32_t open[kVectors];
#pragma unroll
            for (int k = 0; k < kVectors; ++k) x[k] = next[k], open[k] = next_open[k];
            const uint32_t *const allowed = mask_of(mask_now);
            if (row + p.groups < n) {
                load(row + p.groups, mask_next);
                mask_now = mask_next;
                mask_next = mask_row(row + 2 * p.groups);
            }
            lds_barrier();

            const int64_t m = first + row;
            const uint16_t *in = row_in(row);
            uint16_t *out = p.out + m * p.ld_out;
            auto change = [&](float x, uint32_t word, int v) {
                const uint32_t count = word & kCount;
                x *= word & ~kBiased ? (x > 0.f ? inv : rep) : 1.f;
                x = __builtin_fmaf(-freq, (float)count, x) - (count ? pres : 0.f);
                if (word & kBiased) {
                    if (bias_n <= kBiases) {
                        for (int b = 0; b < bias_n; ++b)
                            if (bias_token[b] == v) x += bias_value[b];
                    } else {
                        for (int64_t b = b0; b < b1; ++b)
                            if (a.bias_tokens[b] == v) x += a.bias_values[b];
                    }
                }
                return x;
            };
            auto single = [&](int v) {
                const uint32_t word = table[v - v0];
                uint32_t r = in[v];
                if (word) r = f32_to_bf16_rne(change(bits_f32(r << 16), word, v));
                if (allowed && !(allowed[v >> 5] >> (v & 31) & 1)) r = 0xFF80u;
                out[v] = (uint16_t)r;
            };
            const int lead = lead_of(in);
            if (lead != lead_of(out)) {
                for (int v = v0 + tid; v < v1; v += kThreads) single(v);
                continue;
            }
            // 8 bits from token v on
            auto bits_at = [](const uint32_t *words, int v, int last) {
                uint32_t b = words[v >> 5] >> (v & 31);
                if ((v & 31) > 24) b |= words[min((v >> 5) + 1, last)] << (32 - (v & 31));
                return b & 0xFFu;
            };
            auto vector = [&](uint4 x, uint32_t open, int v) {
                open = !allowed ? 0xFFu : lead == 0 ? open >> (v & 31) & 0xFFu : bits_at(allowed, v, (p.V - 1) >> 5);
                // Few logits are marked (3300 of 248320 by a history of 4096): one after the other in a
                // lane takes a wave two or three rounds (for 512 rows, then 203 us; computing all 8 takes 312
                // vector instructions, 220 us).
                uint32_t marked = bits_at(marks, v - v0, kMostRange / 32 + 1) & open;
                while (marked) {
                    const int e = __builtin_ctz(marked), k = e >> 1, shift = 16 * (e & 1);
                    marked &= marked - 1;
                    const uint32_t word = table[v - v0 + e];
                    const uint32_t pair = k & 2 ? (k & 1 ? x.w : x.z) : (k & 1 ? x.y : x.x);
                    const float y = change(bits_f32(pair >> shift << 16), word, v + e);
                    const uint32_t r = word ? pack_bf16(y, 0.f) & 0xFFFFu : pair >> shift & 0xFFFFu;
                    const uint32_t now = (pair & ~(0xFFFFu << shift)) | r << shift;
                    x.x = k == 0 ? now : x.x;
                    x.y = k == 1 ? now : x.y;
                    x.z = k == 2 ? now : x.z;
                    x.w = k == 3 ? now : x.w;
                }
                if (allowed) {
                    auto closed = [&](uint32_t pair, int e) {
                        const uint32_t keep = (open >> e & 1 ? 0xFFFFu : 0u) | (open >> e & 2 ? 0xFFFF0000u : 0u);
                        return (pair & keep) | (0xFF80FF80u & ~keep);
                    };
                    x = make_uint4(closed(x.x, 0), closed(x.y, 2), closed(x.z, 4), closed(x.w, 6));
                }
                *(uint4 *)(out + v) = x;
            };
            const int j0 = first_vector(lead) + tid;
            auto place = [&](int j, auto whole) {
                const int v = 8 * j - lead;
                if (v >= v1) return;
                if (v >= 0 && v + 8 <= p.V) whole(v);
                else
                    for (int e = max(v, 0); e < min(v + 8, p.V); ++e) single(e);
            };
#pragma unroll
            for (int k = 0; k < kVectors; ++k) place(j0 + k * kThreads, [&](int v) { vector(x[k], open[k], v); });
            // (a row that does not begin on a line may have one more)
            place(j0 + kVectors * kThreads, [&](int v) { vector(*(const uint4 *)(in + v), ~0u, v); });
        }
    }
}

}  // namespace

hipError_t launch_adjust_logits(const void *logits, int64_t ld, const int32_t *starts, const svq_adjustments &a, void *out,
                                int64_t ld_out, int64_t M, int64_t S, int64_t V, int num_cus, hipStream_t stream) {
    Params p{};
    p.logits = (const uint16_t *)logits;
    p.ld = ld;
    p.out = (uint16_t *)out;
    p.ld_out = ld_out;
    p.starts = starts;
    p.a = a;
    p.M = (int)M;
    p.S = (int)S;
    p.V = (int)V;
    // Two workgroups a compute unit, which is what LDS holds: whole ranges (every further one counts
    // the history again), fewer rows each, and shorter ranges only where there are too few rows (512
    // rows of 8 sequences: 16 ranges, 4 groups of rows 112 us, 64 ranges of all rows 182).
    const int64_t want = 2 * (int64_t)num_cus, rows = (M + S - 1) / S;
    int64_t ranges = (V + kMostRange - 1) / kMostRange;
    p.groups = (int)std::max<int64_t>(1, std::min<int64_t>(rows, (want + S * ranges - 1) / (S * ranges)));
    ranges = std::max<int64_t>(ranges, std::min<int64_t>((want + S * p.groups - 1) / (S * p.groups), (V + 1023) / 1024));
    p.range = (int)(((V + ranges - 1) / ranges + 7) & ~(int64_t)7);
    p.ranges = (int)((V + p.range - 1) / p.range);
    p.items = (int64_t)p.ranges * p.groups * S;
    hipLaunchKernelGGL(adjust_kernel, dim3((uint32_t)std::min<int64_t>(p.items, 1 << 20)), dim3(kThreads), 0, stream, p);
    return hipGetLastError();
}

}  // namespace svq
