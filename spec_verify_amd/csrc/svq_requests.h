// Internal launch interface of the per-request operators (svq_requests.cpp to their
// kernels). Every launcher assumes its arguments were validated by the caller.
#pragma once

#include "svq_launch.h"

namespace svq {

int device_cus();  // compute units of the current device (svq_api.cpp)

// Low-rank adapters: blocks of 256 rows, in each at most `items` groups of up to 16 rows
// of one adapter. First launch: an item, rank_tiles x 16 ranks and one of `splits` K
// ranges (of tiles_per_split 128-element tiles; range_blocks block indexes) per workgroup.
// Second: an item and 256 columns (col_blocks block indexes). Or one launch for both; the
// workspace is the same for either.
struct AdapterPlan {
    int64_t row_blocks;
    int items, rank_tiles, rank_chunks, splits, tiles_per_split, range_blocks;
    int col_blocks;
    bool one_launch;
    size_t workspace_bytes;
};
AdapterPlan plan_adapter(int64_t M, int64_t N, int64_t K, int64_t R, int64_t slots);
hipError_t launch_adapter_add(const AdapterPlan &p, const void *base, int64_t ld_base, const void *x, const void *a,
                              const void *b, const int32_t *rows, const float *scales, void *out, int64_t ld_out,
                              int64_t M, int64_t N, int64_t K, int R, int slots, void *workspace, hipStream_t stream);

// Sampling: one workgroup per row, or (parts > 1) `parts` workgroups count a row's
// values and a second launch draws from their lists in the workspace.
struct SamplePlan {
    int parts, vectors_per_part;
    bool mark;  // one workgroup per row: rare rows are left to a second launch
    size_t workspace_bytes;
};
SamplePlan plan_sample(int64_t M, int64_t V, int num_cus);
hipError_t launch_sample(const SamplePlan &p, const void *logits, int64_t ld, const float *u, const float *temperature,
                         const int32_t *top_k, const float *top_p, const float *min_p, int32_t *tokens,
                         float *logprobs, int64_t M, int64_t V, void *workspace, hipStream_t stream);
hipError_t launch_accept_drafts(const int32_t *tokens, const int32_t *inputs, const int32_t *starts, int32_t *accepted,
                                int32_t *next, int32_t *committed, int64_t M, int64_t S, hipStream_t stream);

}  // namespace svq
