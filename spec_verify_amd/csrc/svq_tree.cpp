// C ABI of the operators of a tree of drafts (include/svq.h): argument validation and
// launch. Validation is pure host code that runs before any HIP call, so every error path
// is reachable without a GPU.
#include "svq_tree.h"

#include <hip/hip_runtime.h>

#include <cstdint>

#include "svq_check.h"
#include "svq_requests.h"

using namespace svq;

namespace {

constexpr int64_t kMaxDim = int64_t(1) << 24;     // per dimension
constexpr int64_t kMaxTokens = int64_t(1) << 30;  // of a sequence

int check_attention_shape(int64_t M, int64_t S, int32_t H, int32_t KVH, int32_t D) {
    if (M <= 0 || S <= 0 || H <= 0 || KVH <= 0 || M > kMaxDim || S > kMaxDim || H > 65536 || KVH > H ||
        M * H >= (int64_t(1) << 31))
        return SVQ_ERR_DIM;
    if (D != 64 && D != 128 && D != 256) return SVQ_ERR_UNSUPPORTED;
    if (H % KVH) return SVQ_ERR_DIVISIBILITY;
    return SVQ_OK;
}

// Strides of one side of a cache, in the dimensions that have several entries: whole 16 bytes,
// pages and tokens less than 4 GiB apart, and an extent that 63 bits hold.
int check_strides(const int64_t *st, const svq_kv_cache &c, int32_t KVH, int32_t D, int64_t size, size_t *bytes) {
    const int64_t most = int64_t(1) << 46;
    const int64_t count[3] = {c.pages, c.page_size, KVH};
    int64_t extent = D;
    for (int i = 0; i < 3; ++i) {
        if (count[i] <= 1) continue;
        if (st[i] < 0 || st[i] > most / (count[i] - 1) || (i < 2 && st[i] * size >= (int64_t(1) << 32))) return SVQ_ERR_DIM;
        if (st[i] * size % 16) return SVQ_ERR_ALIGN;
        extent += st[i] * (count[i] - 1);
    }
    *bytes = c.pages ? (size_t)(extent * size) : 0;
    return SVQ_OK;
}

}  // namespace

extern "C" {

size_t svq_tree_attention_workspace_bytes(int64_t M, int64_t S, int32_t H, int32_t KVH, int32_t D) {
    if (check_attention_shape(M, S, H, KVH, D) != SVQ_OK) return (size_t)-1;
    return plan_tree_attention(M, S, H, KVH, D, device_cus()).workspace_bytes;
}

int svq_tree_attention(const void *q, int64_t ld_q, const void *k, int64_t ld_k, const void *v, int64_t ld_v,
                       const svq_kv_cache *cache, const int32_t *starts, const int32_t *parents, float scale,
                       int32_t window, int32_t sinks, void *out, int64_t ld_out, int64_t M, int64_t S, int32_t H,
                       int32_t KVH, int32_t D, void *workspace, size_t workspace_bytes, void *stream) {
    int st = check_attention_shape(M, S, H, KVH, D);
    if (st != SVQ_OK) return st;
    if (!q || !k || !v || !cache || !starts || !out) return SVQ_ERR_NULL;
    const svq_kv_cache &c = *cache;
    // (a pool or a table of nothing has no address)
    if (((!c.k || !c.v) && c.pages != 0) || (!c.page_table && c.max_pages != 0) || !c.lengths) return SVQ_ERR_NULL;
    if (c.type != SVQ_CACHE_BF16 && c.type != SVQ_CACHE_E4M3) return SVQ_ERR_UNSUPPORTED;
    if (c.type == SVQ_CACHE_BF16 && (c.k_scale || c.v_scale)) return SVQ_ERR_UNSUPPORTED;
    const int64_t most = int64_t(1) << 31, qc = (int64_t)H * D, kc = (int64_t)KVH * D;
    if (ld_q < qc || ld_out < qc || ld_k < kc || ld_v < kc || ld_q > most || ld_k >= most || ld_v >= most || ld_out > most)
        return SVQ_ERR_DIM;
    if (ld_q % 8 || ld_k % 8 || ld_v % 8 || ld_out % 8) return SVQ_ERR_DIVISIBILITY;
    if (c.pages < 0 || c.pages > INT32_MAX || c.page_size <= 0 || c.page_size > (1 << 20) || c.max_pages < 0 ||
        (int64_t)c.max_pages * c.page_size > kMaxTokens || c.ld_table < c.max_pages || c.ld_table > most)
        return SVQ_ERR_DIM;
    // steps (a tile of 64 tokens, a run of blocks of 16 rows or more) are counted in 31 bits
    const int64_t tiles = ((int64_t)c.max_pages * c.page_size + M) / 64 + 2, runs = M * (H / KVH) / 16 + S;
    if (tiles > INT32_MAX / KVH / runs) return SVQ_ERR_DIM;
    const int64_t size = c.type == SVQ_CACHE_E4M3 ? 1 : 2;
    size_t kb, vb;
    if ((st = check_strides(c.k_strides, c, KVH, D, size, &kb)) != SVQ_OK) return st;
    if ((st = check_strides(c.v_strides, c, KVH, D, size, &vb)) != SVQ_OK) return st;
    for (const void *p : {q, k, v, c.k, c.v, (const void *)out})
        if (!aligned(p, 16)) return SVQ_ERR_ALIGN;
    for (const void *p : {(const void *)starts, (const void *)parents, (const void *)c.page_table, (const void *)c.lengths,
                          (const void *)c.k_scale, (const void *)c.v_scale})
        if (!aligned(p, 4)) return SVQ_ERR_ALIGN;
    const AttendPlan plan = plan_tree_attention(M, S, H, KVH, D, device_cus());
    if (!workspace || workspace_bytes < plan.workspace_bytes || !aligned(workspace, 256)) return SVQ_ERR_WORKSPACE;
    auto rows = [&](int64_t ld, int64_t cols) { return ((size_t)(M - 1) * ld + cols) * 2; };
    const Span outs[] = {{out, rows(ld_out, qc)}, {workspace, plan.workspace_bytes}};
    // (q, k and v may be other columns of the matrix that out is in)
    auto beside = [&](const void *p, int64_t ld, int64_t cols) {
        return Span{ld == ld_out && columns_apart(p, cols, out, qc, ld) ? nullptr : p, rows(ld, cols)};
    };
    const Span ins[] = {beside(q, ld_q, qc),
                        beside(k, ld_k, kc),
                        beside(v, ld_v, kc),
                        {c.k, kb},
                        {c.v, vb},
                        {starts, (size_t)(S + 1) * 4},
                        {parents, (size_t)M * 4},
                        {c.page_table, c.max_pages ? ((size_t)(S - 1) * c.ld_table + c.max_pages) * 4 : 0},
                        {c.lengths, (size_t)S * 4},
                        {c.k_scale, (size_t)KVH * 4},
                        {c.v_scale, (size_t)KVH * 4}};
    if (any_overlap(outs, 2, ins, 11)) return SVQ_ERR_OVERLAP;
    const Span chunk[] = {{q, rows(ld_q, qc)}, {k, rows(ld_k, kc)}, {v, rows(ld_v, kc)}};
    if (any_overlap(outs + 1, 1, chunk, 3)) return SVQ_ERR_OVERLAP;
    return launch_tree_attention(plan, q, ld_q, k, ld_k, v, ld_v, c, starts, parents, scale, window, sinks, out, ld_out, M,
                                 S, H, KVH, D, workspace, (hipStream_t)stream) == hipSuccess
               ? SVQ_OK
               : SVQ_ERR_HIP;
}

int svq_adjust_logits(const void *logits, int64_t ld, const int32_t *starts, const svq_adjustments *adjustments,
                      void *out, int64_t ld_out, int64_t M, int64_t S, int64_t V, void *stream) {
    if (M <= 0 || S <= 0 || V <= 0 || M > kMaxDim || S > kMaxDim || V > kMaxDim) return SVQ_ERR_DIM;
    if (!logits || !starts || !adjustments || !out) return SVQ_ERR_NULL;
    const svq_adjustments &a = *adjustments;
    if ((!a.history && a.max_history != 0) || !a.lengths || !a.inputs) return SVQ_ERR_NULL;
    const int64_t most = int64_t(1) << 31;
    if (ld < V || ld_out < V || ld > most || ld_out > most) return SVQ_ERR_DIM;
    // (occurrences are counted in 30 bits)
    if (a.max_history < 0 || a.max_history > (1 << 29) || a.ld_history < a.max_history || a.ld_history > most)
        return SVQ_ERR_DIM;
    if (a.bias_starts || a.bias_tokens || a.bias_values) {
        if (!a.bias_starts || (a.biases > 0 && (!a.bias_tokens || !a.bias_values))) return SVQ_ERR_NULL;
        if (a.biases < 0 || a.biases > INT32_MAX) return SVQ_ERR_DIM;
    }
    if (a.allowed || a.mask_rows) {
        if (!a.allowed || !a.mask_rows) return SVQ_ERR_NULL;
        if (a.masks <= 0 || a.masks > INT32_MAX || a.ld_allowed < (V + 31) / 32 || a.ld_allowed > most) return SVQ_ERR_DIM;
    }
    if (!aligned(logits, 2) || !aligned(out, 2)) return SVQ_ERR_ALIGN;
    const int64_t biases = a.bias_starts ? a.biases : 0;
    const Span ins[] = {{logits, ((size_t)(M - 1) * ld + V) * 2},
                        {starts, (size_t)(S + 1) * 4},
                        {a.history, a.max_history ? ((size_t)(S - 1) * a.ld_history + a.max_history) * 4 : 0},
                        {a.lengths, (size_t)S * 4},
                        {a.prompt_lengths, (size_t)S * 4},
                        {a.inputs, (size_t)M * 4},
                        {a.parents, (size_t)M * 4},
                        {a.repetition, (size_t)S * 4},
                        {a.presence, (size_t)S * 4},
                        {a.frequency, (size_t)S * 4},
                        {a.bias_starts, (size_t)(S + 1) * 4},
                        {a.bias_tokens, (size_t)biases * 4},
                        {a.bias_values, (size_t)biases * 4},
                        {a.allowed, a.allowed ? ((size_t)(a.masks - 1) * a.ld_allowed + (V + 31) / 32) * 4 : 0},
                        {a.mask_rows, (size_t)M * 4}};
    for (int i = 1; i < 15; ++i)
        if (!aligned(ins[i].p, 4)) return SVQ_ERR_ALIGN;
    const Span outs[] = {{out, ((size_t)(M - 1) * ld_out + V) * 2}};
    // (in place, or other columns of one matrix)
    const bool in_place = ld_out == ld && (out == logits || columns_apart(logits, V, out, V, ld));
    if (any_overlap(outs, 1, in_place ? ins + 1 : ins, in_place ? 14 : 15)) return SVQ_ERR_OVERLAP;
    return launch_adjust_logits(logits, ld, starts, a, out, ld_out, M, S, V, device_cus(), (hipStream_t)stream) == hipSuccess
               ? SVQ_OK
               : SVQ_ERR_HIP;
}

int svq_accept_tree(const int32_t *tokens, const int32_t *inputs, const int32_t *parents, const int32_t *starts,
                    int32_t *accepted, int32_t *next, int32_t *committed, int32_t *path, int64_t M, int64_t S,
                    void *stream) {
    if (M <= 0 || S <= 0 || M > kMaxDim || S > kMaxDim) return SVQ_ERR_DIM;
    const void *all[] = {tokens, inputs, parents, starts, accepted, next, committed, path};
    for (const void *p : all)
        if (!p) return SVQ_ERR_NULL;
    for (const void *p : all)
        if (!aligned(p, 4)) return SVQ_ERR_ALIGN;
    const Span outs[] = {
        {accepted, (size_t)S * 4}, {next, (size_t)S * 4}, {committed, (size_t)M * 4}, {path, (size_t)M * 4}};
    const Span ins[] = {
        {tokens, (size_t)M * 4}, {inputs, (size_t)M * 4}, {parents, (size_t)M * 4}, {starts, (size_t)(S + 1) * 4}};
    if (any_overlap(outs, 4, ins, 4)) return SVQ_ERR_OVERLAP;
    return launch_accept_tree(tokens, inputs, parents, starts, accepted, next, committed, path, M, S,
                              (hipStream_t)stream) == hipSuccess
               ? SVQ_OK
               : SVQ_ERR_HIP;
}

}  // extern "C"
