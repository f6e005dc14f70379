// C ABI of the per-request operators of a verify chunk (include/svq.h): argument
// validation and launch. Validation is pure host code that runs before any HIP call, so
// every error path is reachable without a GPU.
#include "../../include/svq.h"

#include <hip/hip_runtime.h>

#include <cstdint>

#include "svq_check.h"
#include "svq_requests.h"

using namespace svq;

namespace {

constexpr int64_t kMaxDim = int64_t(1) << 24;  // per dimension

int check_adapter_shape(int64_t M, int64_t N, int64_t K, int32_t R, int32_t slots) {
    // x and y as in the GEMMs: below 2^31 bytes each
    if (M <= 0 || N <= 0 || K <= 0 || M > kMaxDim || N > kMaxDim || K > kMaxDim || M * K >= (int64_t(1) << 30) ||
        M * N >= (int64_t(1) << 30))
        return SVQ_ERR_DIM;
    if (R <= 0 || R > SVQ_MAX_ADAPTER_RANK || slots <= 0) return SVQ_ERR_DIM;
    // the pools are addressed with 64 bits; no memory holds more than this many elements
    if (slots > (int64_t(1) << 46) / (R * (N > K ? N : K))) return SVQ_ERR_DIM;
    if (N % 16 || K % 128 || R % 8) return SVQ_ERR_DIVISIBILITY;
    return SVQ_OK;
}

int check_sample_shape(int64_t M, int64_t V) {
    return M > 0 && V > 0 && M <= kMaxDim && V <= kMaxDim ? SVQ_OK : SVQ_ERR_DIM;
}

}  // namespace

extern "C" {

size_t svq_adapter_workspace_bytes(int64_t M, int64_t N, int64_t K, int32_t R, int32_t slots) {
    if (check_adapter_shape(M, N, K, R, slots) != SVQ_OK) return (size_t)-1;
    return plan_adapter(M, N, K, R, slots).workspace_bytes;
}

int svq_adapter_add(const void *base, int64_t ld_base, const void *x, const void *a, const void *b,
                    const int32_t *rows, const float *scales, void *out, int64_t ld_out, int64_t M, int64_t N,
                    int64_t K, int32_t R, int32_t slots, void *workspace, size_t workspace_bytes, void *stream) {
    int st = check_adapter_shape(M, N, K, R, slots);
    if (st != SVQ_OK) return st;
    if (ld_base < N || ld_out < N || ld_base > (int64_t(1) << 31) || ld_out > (int64_t(1) << 31)) return SVQ_ERR_DIM;
    if (ld_base % 8 || ld_out % 8) return SVQ_ERR_DIVISIBILITY;
    if (!base || !x || !a || !b || !rows || !scales || !out) return SVQ_ERR_NULL;
    if (!aligned(base, 16) || !aligned(x, 16) || !aligned(a, 16) || !aligned(b, 16) || !aligned(rows, 4) ||
        !aligned(scales, 4) || !aligned(out, 16))
        return SVQ_ERR_ALIGN;
    const AdapterPlan plan = plan_adapter(M, N, K, R, slots);
    if (!workspace || workspace_bytes < plan.workspace_bytes || !aligned(workspace, 256)) return SVQ_ERR_WORKSPACE;
    const Span base_span = {base, ((size_t)(M - 1) * ld_base + N) * 2};
    const Span outs[] = {{out, ((size_t)(M - 1) * ld_out + N) * 2}, {workspace, plan.workspace_bytes}};
    const Span ins[] = {{x, (size_t)M * K * 2},
                        {a, (size_t)slots * R * K * 2},
                        {b, (size_t)slots * N * R * 2},
                        {rows, (size_t)M * 4},
                        {scales, (size_t)slots * 4}};
    if (any_overlap(outs, 2, ins, 5) || overlap(outs[1], base_span)) return SVQ_ERR_OVERLAP;
    // in place is the same rows in the same places, or other columns of the same matrix; anything
    // else between base and out must be apart
    if (!(out == base && ld_out == ld_base) && !(ld_out == ld_base && columns_apart(base, N, out, N, ld_base)) &&
        overlap(outs[0], base_span))
        return SVQ_ERR_OVERLAP;
    return launch_adapter_add(plan, base, ld_base, x, a, b, rows, scales, out, ld_out, M, N, K, R, slots, workspace,
                              (hipStream_t)stream) == hipSuccess
               ? SVQ_OK
               : SVQ_ERR_HIP;
}

size_t svq_sample_workspace_bytes(int64_t M, int64_t V) {
    if (check_sample_shape(M, V) != SVQ_OK) return (size_t)-1;
    return plan_sample(M, V, device_cus()).workspace_bytes;
}

int svq_sample(const void *logits, int64_t ld, const float *u, const float *temperature, const int32_t *top_k,
               const float *top_p, const float *min_p, int32_t *tokens, float *logprobs, int64_t M, int64_t V,
               void *workspace, size_t workspace_bytes, void *stream) {
    int st = check_sample_shape(M, V);
    if (st != SVQ_OK) return st;
    if (ld < V || ld > (int64_t(1) << 31)) return SVQ_ERR_DIM;
    if (!logits || !u || !tokens) return SVQ_ERR_NULL;
    if (!aligned(logits, 2) || !aligned(u, 4) || !aligned(temperature, 4) || !aligned(top_k, 4) || !aligned(top_p, 4) ||
        !aligned(min_p, 4) || !aligned(tokens, 4) || !aligned(logprobs, 4))
        return SVQ_ERR_ALIGN;
    const size_t rb = (size_t)M * 4;
    const Span io[] = {{tokens, rb}, {logprobs, rb}};
    const Span ins[] = {{logits, ((size_t)(M - 1) * ld + V) * 2}, {u, rb}, {temperature, rb}, {top_k, rb}, {top_p, rb},
                        {min_p, rb}};
    if (any_overlap(io, 2, ins, 6)) return SVQ_ERR_OVERLAP;
    // the plan needs the device's compute-unit count; the buffers are checked first
    const SamplePlan plan = plan_sample(M, V, device_cus());
    if (plan.workspace_bytes) {
        if (!workspace || workspace_bytes < plan.workspace_bytes || !aligned(workspace, 256)) return SVQ_ERR_WORKSPACE;
        const Span outs[] = {{workspace, plan.workspace_bytes}, {tokens, rb}, {logprobs, rb}};
        if (any_overlap(outs, 3, ins, 6)) return SVQ_ERR_OVERLAP;
    }
    return launch_sample(plan, logits, ld, u, temperature, top_k, top_p, min_p, tokens, logprobs, M, V, workspace,
                         (hipStream_t)stream) == hipSuccess
               ? SVQ_OK
               : SVQ_ERR_HIP;
}

int svq_accept_drafts(const int32_t *tokens, const int32_t *inputs, const int32_t *starts, int32_t *accepted,
                      int32_t *next, int32_t *committed, int64_t M, int64_t S, void *stream) {
    if (M <= 0 || S <= 0 || M > kMaxDim || S > kMaxDim) return SVQ_ERR_DIM;
    const void *all[] = {tokens, inputs, starts, accepted, next, committed};
    for (const void *p : all)
        if (!p) return SVQ_ERR_NULL;
    for (const void *p : all)
        if (!aligned(p, 4)) return SVQ_ERR_ALIGN;
    const Span outs[] = {{accepted, (size_t)S * 4}, {next, (size_t)S * 4}, {committed, (size_t)M * 4}};
    const Span ins[] = {{tokens, (size_t)M * 4}, {inputs, (size_t)M * 4}, {starts, (size_t)(S + 1) * 4}};
    if (any_overlap(outs, 3, ins, 3)) return SVQ_ERR_OVERLAP;
    return launch_accept_drafts(tokens, inputs, starts, accepted, next, committed, M, S, (hipStream_t)stream) ==
                   hipSuccess
               ? SVQ_OK
               : SVQ_ERR_HIP;
}

}  // extern "C"
