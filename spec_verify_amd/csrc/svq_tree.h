// Internal launch interface of the operators of a tree of drafts (svq_tree.cpp to their
// kernels). Every launcher assumes its arguments were validated by the caller.
#pragma once

#include "../../include/svq.h"
#include "svq_launch.h"

namespace svq {

// Tree attention: `teams` of workgroups share the chunk's (sequence, KV head, tile of
// tokens) steps evenly, the members of a team taking different blocks of `block_rows` rows;
// what they leave unfinished is joined by a second launch.
struct AttendPlan {
    int block_rows, teams, members;
    size_t workspace_bytes;
};
AttendPlan plan_tree_attention(int64_t M, int64_t S, int64_t H, int64_t KVH, int64_t D, int num_cus);
hipError_t launch_tree_attention(const AttendPlan &p, const void *q, int64_t ld_q, const void *k, int64_t ld_k,
                                 const void *v, int64_t ld_v, const svq_kv_cache &cache, const int32_t *starts,
                                 const int32_t *parents, float scale, int window, int sinks, void *out, int64_t ld_out,
                                 int64_t M, int64_t S, int H, int KVH, int D, void *workspace, hipStream_t stream);

hipError_t launch_adjust_logits(const void *logits, int64_t ld, const int32_t *starts, const svq_adjustments &a, void *out,
                                int64_t ld_out, int64_t M, int64_t S, int64_t V, int num_cus, hipStream_t stream);

hipError_t launch_accept_tree(const int32_t *tokens, const int32_t *inputs, const int32_t *parents,
                              const int32_t *starts, int32_t *accepted, int32_t *next, int32_t *committed,
                              int32_t *path, int64_t M, int64_t S, hipStream_t stream);

}  // namespace svq
