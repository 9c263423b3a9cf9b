// Launchers of the scored router (csrc/scored.hip).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moe {

struct ScoredPass {
    int T, H, E, k;
    int softmax, groups, keep, renorm;
    float scale;
    const void *x;
    int x_bf16;
    int64_t ldx;
    const float *w, *bias;                       // bias may be null
    int32_t *topk_idx;
    float *topk_w;
    int32_t *offsets, *perm, *inv;
    double *logits;                              // workspace: [T][E]
    int32_t *rank, *tile_counts;                 // workspace of the grouping (T > SCORED_SMALL_T)
};

// up to this many tokens one work-group groups the assignments
constexpr int SCORED_SMALL_T = 64;

size_t scored_logit_bytes(int T, int E);
void launch_scored_logits(const ScoredPass &p, hipStream_t s);
void launch_scored_topk(const ScoredPass &p, hipStream_t s);

}  // namespace moe
