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
    // workspace
    void *logits;                                // fp64 or fp32 [parts][T][E]
    void *wsplit;                                // split router: the bf16 terms of w
    float *wnorm, *xnorm;                        // split router: |w_e|^2 [E], |x_t|^2 [parts][T]
    int32_t *open;                               // split router: the tokens left to fp64, how many and, 16 bytes on, which
    int32_t *rank, *tile_counts;                 // grouping where scored_group_fits says no
};

// up to this many tokens the logits are sums of a wave each
constexpr int SCORED_SMALL_T = 128;

// The split router (see scored.hip): bf16 tokens with sigmoid scores, and enough
// of them.  Its launches have a floor (the terms of w, the open tokens) that the
// fp64 matrix instructions only reach past 640 tokens of 256 experts: H = 7168,
// T = 333 / 500 / 640 / 700 / 1000 / 1400 / 2048 take 65 / 67 / 92 / 93 / 94 / 160
// / 165 us in fp64 and 83 / 85 / 89 / 89 / 89 / 92 / 95 us split.  The border is
// that of H = 7168: with H = 1024, T = 640 takes 34 us in fp64 and 59 split; with
// H = 2048 and 64 experts T = 2560 takes 52 us either way.
inline int scored_split_above(int E) { return 640 * 256 / E > SCORED_SMALL_T ? 640 * 256 / E : SCORED_SMALL_T; }
inline bool scored_split(int T, int E, bool softmax, bool x_bf16) { return T > scored_split_above(E) && !softmax && x_bf16; }

size_t scored_logit_bytes(int T, int H, int E, bool split);
size_t scored_split_bytes(int H, int E);         // of wsplit
size_t scored_open_bytes(int T);                 // of open
int scored_split_parts(int T, int H, int E);

hipError_t launch_scored_logits(const ScoredPass &p, hipStream_t s);
hipError_t launch_scored_split(const ScoredPass &p, hipStream_t s);        // w into its terms
hipError_t launch_scored_split_logits(const ScoredPass &p, hipStream_t s);
hipError_t launch_scored_topk(const ScoredPass &p, hipStream_t s);         // T == 1: the grouping too

bool scored_group_fits(int T, int E);            // whether one work-group can group the assignments
hipError_t launch_scored_group(const ScoredPass &p, hipStream_t s);

}  // namespace moe
