// Launchers of the MoE block for a few tokens (csrc/block.hip).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "scored.h"

namespace moe {

constexpr int BLOCK_MAX_T = 16, BLOCK_MAX_K = 16, BLOCK_MAX_E = 512, BLOCK_MAX_DIM = 8192;

struct BlockPass {
    int T, H, I, E, k, sh;                       // sh: features of the shared expert, 0 for none
    // norm
    const void *x, *res;                         // res may be null
    void *sum;                                   // may be null
    int x_bf16, res_bf16, n_bf16;
    int64_t ldx, ldres, ldsum, ldy;
    const float *norm_w;
    float eps;
    // experts
    const uint8_t *gate, *up, *down;
    const int8_t *codebook;
    const int8_t *sh_up, *sh_down;
    int64_t ld_up, ld_down;
    const float *up_scale, *up_bias, *down_scale, *down_bias;
    ScoredPass route;                            // the router and the routing outputs
    float *y;
    // workspace
    uint32_t *ctl;                               // counters, a line each
    int32_t *list;                               // different experts, then a token and a weight for each position
    double *logits;                              // [T][E]
    void *s;                                     // [T][H] of the residual's type
    int8_t *planes;                              // [T][quads of H][digits of four blocks]
    float *scales;                               // [T][4 quads of H]
    int8_t *h;                                   // [T k][records] of 64 features in digits
    float *hs;                                   // [T][sh]
    // set by block_layout
    int nb, nq, nbi, nqi, nbs, nqs, records;     // blocks of 256 and quads of blocks of H, I, sh; records of a row of h
    int F, nf, rows;                             // features of a routed gate/up item, items of an expert, rows of a down item
    int experts;                                 // whose logits a work-group of the first kernel computes
    int t_shared, t_down;                        // items
    int slots, chunk;                            // tokens, and rows of h, that LDS holds
    int o_planes, o_scales, o_red, o_recs, lds;          // LDS offsets and bytes
};

void block_layout(BlockPass &p);                 // the sizes that follow from the first line
size_t block_workspace(BlockPass &p, char *base);
hipError_t launch_block_norm(const BlockPass &p, hipStream_t s);
hipError_t launch_block(const BlockPass &p, hipStream_t s);

}  // namespace moe
