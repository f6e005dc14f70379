// Logits as the sampler takes them (svq_adjust_logits): penalties for the tokens of a
// sequence's history and of a row's path in the tree of drafts, biases, grammar masks.
//
// A workgroup takes a range of the vocabulary for some rows of one sequence. It counts the
// history's tokens of that range in LDS once, and for each row adds its path's, streams the
// row's logits past the counts, and takes the path's out again.
#include <algorithm>

#include "svq_tree.h"

namespace svq {

namespace {

constexpr int kThreads = 256;
constexpr int kMostRange = 16384;  // tokens of a workgroup's range
constexpr int kPath = 1024;        // tokens of a path taken at a time

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
    __shared__ int path[kPath], path_n, path_at;
    const int tid = threadIdx.x;
    const svq_adjustments &a = p.a;
    for (int64_t item = blockIdx.x; item < p.items; item += gridDim.x) {
        const int c = (int)(item % p.ranges);
        const int g = (int)(item / p.ranges % p.groups), s = (int)(item / p.ranges / p.groups);
        const int first = min(max(p.starts[s], 0), p.M), n = max(min(p.starts[s + 1], p.M) - first, 0);
        if (g >= n) continue;
        const int v0 = c * p.range, v1 = min(v0 + p.range, p.V);
        const int end = min(v1 + 8, p.V);  // counted too: a vector of 8 may begin before v1 and end after it
        const int32_t *parents = a.parents ? a.parents + first : nullptr;
        const float rep = a.repetition ? a.repetition[s] : 1.f, inv = 1.f / rep;
        const float pres = a.presence ? a.presence[s] : 0.f, freq = a.frequency ? a.frequency[s] : 0.f;
        __syncthreads();
        for (int i = tid; i < (p.range + 8) / 4; i += kThreads) ((uint4 *)table)[i] = make_uint4(0, 0, 0, 0);
        __syncthreads();
        auto in_range = [&](int v) { return v >= v0 && v < end; };
        const int len = min(max(a.lengths[s], 0), a.max_history);
        const int prompt = a.prompt_lengths ? a.prompt_lengths[s] : 0;
        const int32_t *history = a.history + (int64_t)s * a.ld_history;
        for (int i = tid; i < len; i += kThreads) {
            const int v = history[i];
            if (!in_range(v)) continue;
            if (i < prompt) atomicOr(&table[v - v0], kPrompt);
            else atomicAdd(&table[v - v0], 1u);
        }
        int64_t b0 = 0, b1 = 0;
        if (a.bias_starts) {
            b0 = min(max((int64_t)a.bias_starts[s], (int64_t)0), a.biases);
            b1 = min((int64_t)a.bias_starts[s + 1], a.biases);
            for (int64_t b = b0 + tid; b < b1; b += kThreads) {
                const int v = a.bias_tokens[b];
                if (in_range(v)) atomicOr(&table[v - v0], kBiased);
            }
        }
        // adds `by` to the counts of the path of a row
        auto along_path = [&](int row, uint32_t by) {
            int at = row;
            while (at >= 0) {
                __syncthreads();
                if (tid == 0) {
                    int k = 0;
                    while (at >= 0 && k < kPath) {
                        path[k++] = a.inputs[first + at];
                        const int up = parents ? parents[at] : at - 1;
                        at = up >= 0 && up < at ? up : -1;
                    }
                    path_n = k;
                    path_at = at;
                }
                __syncthreads();
                for (int i = tid; i < path_n; i += kThreads)
                    if (in_range(path[i])) atomicAdd(&table[path[i] - v0], by);
                at = path_at;
            }
            __syncthreads();
        };
        for (int row = g; row < n; row += p.groups) {
            along_path(row, 1u);
            const int64_t m = first + row;
            const uint16_t *in = p.logits + m * p.ld;
            uint16_t *out = p.out + m * p.ld_out;
            const uint32_t *allowed = nullptr;
            if (a.allowed) {
                const int64_t mask = a.mask_rows[m];
                if (mask >= 0 && mask < a.masks) allowed = (const uint32_t *)a.allowed + mask * a.ld_allowed;
            }
            auto change = [&](uint32_t bits, uint32_t word, int v) {
                if (word == 0) return bits;
                float x = bits_f32(bits << 16);
                const uint32_t count = word & kCount;
                if (word & ~kBiased) x *= x > 0.f ? inv : rep;
                if (count) x = x - freq * (float)count - pres;
                if (word & kBiased)
                    for (int64_t b = b0; b < b1; ++b)
                        if (a.bias_tokens[b] == v) x += a.bias_values[b];
                return (uint32_t)f32_to_bf16_rne(x);
            };
            auto single = [&](int v) {
                uint32_t r = change(in[v], table[v - v0], v);
                if (allowed && !(allowed[v >> 5] >> (v & 31) & 1)) r = 0xFF80u;
                out[v] = (uint16_t)r;
            };
            const int lead = (int)((uintptr_t)in / 2 & 7);
            if (lead != (int)((uintptr_t)out / 2 & 7)) {
                for (int v = v0 + tid; v < v1; v += kThreads) single(v);
            } else {
                // vectors of 8 logits on 16-byte lines; the first of a row may begin before it
                for (int j = (v0 + lead + (v0 ? 7 : 0)) / 8 + tid; 8 * j - lead < v1; j += kThreads) {
                    const int v = 8 * j - lead;
                    if (v < 0 || v + 8 > p.V) {
                        for (int e = max(v, 0); e < min(v + 8, p.V); ++e) single(e);
                        continue;
                    }
                    uint4 x = *(const uint4 *)(in + v);
                    uint32_t *const xs = (uint32_t *)&x;
                    uint32_t bits = 0xFFu;
                    if (allowed) {
                        bits = allowed[v >> 5] >> (v & 31);
                        if ((v & 31) > 24) bits |= allowed[min((v >> 5) + 1, (p.V - 1) >> 5)] << (32 - (v & 31));
                    }
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        uint32_t r = change(xs[e / 2] >> (16 * (e & 1)) & 0xFFFFu, table[v - v0 + e], v + e);
                        if (!(bits >> e & 1)) r = 0xFF80u;
                        xs[e / 2] = e & 1 ? (xs[e / 2] & 0xFFFFu) | r << 16 : (xs[e / 2] & 0xFFFF0000u) | r;
                    }
                    *(uint4 *)(out + v) = x;
                }
            }
            along_path(row, ~0u);
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
    // enough workgroups to fill the chip: ranges of the vocabulary first, then rows
    const int64_t want = 4 * (int64_t)num_cus, rows = (M + S - 1) / S;
    int64_t ranges = std::max<int64_t>((V + kMostRange - 1) / kMostRange, std::min<int64_t>((want + S - 1) / S, (V + 1023) / 1024));
    p.range = (int)(((V + ranges - 1) / ranges + 7) & ~(int64_t)7);
    p.ranges = (int)((V + p.range - 1) / p.range);
    p.groups = (int)std::max<int64_t>(1, std::min<int64_t>(rows, (want + S * p.ranges - 1) / (S * p.ranges)));
    p.items = (int64_t)p.ranges * p.groups * S;
    hipLaunchKernelGGL(adjust_kernel, dim3((uint32_t)std::min<int64_t>(p.items, 1 << 20)), dim3(kThreads), 0, stream, p);
    return hipGetLastError();
}

}  // namespace svq
