// Acceptance along a tree of drafts (svq_accept_tree): a wave a sequence walks from the
// first row to the first child whose input is the token sampled at the current row, as
// long as there is one. The lanes look at 64 rows at a time; the rows' parents, inputs and
// samples are read once, ahead of the walk, where the sequence has at most 64 * kKept.
//
// Latency: one trip to memory for starts, one for the rows, then registers alone. 1 tree of 8
// rows 2.9 us, 32 of 64 rows 4.3, 2048 of 1 to 32 rows 5.9 (the call costs the host 11.7).
#include "svq_tree.h"

namespace svq {

namespace {

constexpr int kKept = 4;  // rows of a lane kept in registers

__global__ __launch_bounds__(256) void accept_tree_kernel(const int32_t *__restrict__ tokens,
                                                          const int32_t *__restrict__ inputs,
                                                          const int32_t *__restrict__ parents,
                                                          const int32_t *__restrict__ starts, int32_t *__restrict__ accepted,
                                                          int32_t *__restrict__ next, int32_t *__restrict__ committed,
                                                          int32_t *__restrict__ path, int M, int S) {
    const int lane = threadIdx.x & 63;
    const int64_t s = (int64_t)blockIdx.x * 4 + wave_id();
    if (s > S) return;
    auto start = [&](int64_t i) { return min(max(starts[i], 0), M); };
    auto none = [&](int i) { committed[i] = path[i] = -1; };
    if (s == S) {
        const int b = start(0), e = start(S);
        for (int i = lane; i < b; i += 64) none(i);
        for (int i = e + lane; i < M; i += 64) none(i);
        return;
    }
    const int b = start(s), n = max(start(s + 1) - b, 0);
    int up[kKept], in[kKept], tok[kKept];
#pragma unroll
    for (int k = 0; k < kKept; ++k) {
        const int i = 64 * k + lane;
        up[k] = -1;
        in[k] = tok[k] = 0;
        if (i < n) {
            up[k] = parents[b + i];
            in[k] = inputs[b + i];
            tok[k] = tokens[b + i];
        }
    }
    auto sampled = [&](int i) {
        if (i >= 64 * kKept) return __builtin_amdgcn_readfirstlane(tokens[b + i]);
        int t = 0;
#pragma unroll
        for (int k = 0; k < kKept; ++k)
            if (i >> 6 == k) t = __builtin_amdgcn_readlane(tok[k], i & 63);
        return t;
    };
    int at = 0, depth = 0, token = -1;
    while (n > 0) {
        token = sampled(at);
        if (lane == 0) {
            committed[b + depth] = token;
            path[b + depth] = at;
        }
        ++depth;
        int child = -1;
        if (token >= 0) {
#pragma unroll
            for (int k = 0; k < kKept; ++k) {
                const int i = 64 * k + lane;
                const uint64_t hit = __ballot(i > at && i < n && up[k] == at && in[k] == token);
                if (child < 0 && hit) child = 64 * k + __builtin_ctzll(hit);
            }
            for (int i0 = 64 * kKept; child < 0 && i0 < n; i0 += 64) {
                const int i = i0 + lane;
                const uint64_t hit = __ballot(i > at && i < n && parents[b + i] == at && inputs[b + i] == token);
                if (hit) child = i0 + __builtin_ctzll(hit);
            }
        }
        if (child < 0) break;
        at = child;
    }
    for (int i = depth + lane; i < n; i += 64) none(b + i);
    if (lane == 0) {
        accepted[s] = max(depth - 1, 0);
        next[s] = token;
    }
}

}  // namespace

hipError_t launch_accept_tree(const int32_t *tokens, const int32_t *inputs, const int32_t *parents,
                              const int32_t *starts, int32_t *accepted, int32_t *next, int32_t *committed,
                              int32_t *path, int64_t M, int64_t S, hipStream_t stream) {
    hipLaunchKernelGGL(accept_tree_kernel, dim3((uint32_t)((S + 1 + 3) / 4)), dim3(256), 0, stream, tokens, inputs,
                       parents, starts, accepted, next, committed, path, (int)M, (int)S);
    return hipGetLastError();
}

}  // namespace svq
