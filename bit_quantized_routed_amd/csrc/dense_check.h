// Argument checks and the launch bracket shared by the C entry points of the
// operators around the routed experts.
#pragma once
#include <hip/hip_runtime.h>

#include "moe.h"
#include "rows.h"
#include "status.h"

namespace moe {

constexpr int MAX_ROWS = 1 << 22;                // rows of a call, up to 1024 threads each in a launch of fewer than 2^32

inline int hip_fail(hipError_t e, const char *what) { return set_error(MOE_ERR_HIP, "%s: %s", what, hipGetErrorString(e)); }

// Runs one launch of a call, between the caller's events if it is the profiled one.
struct Launcher {
    moe_profile *p;
    hipStream_t s;
    int n = 0;
    template <class F>
    int operator()(const char *name, F launch)
    {
        const bool timed = p && p->kernel == n;
        if (timed) {
            p->name = name;
            const hipError_t e = hipEventRecord((hipEvent_t)p->ev_start, s);
            if (e != hipSuccess) return hip_fail(e, "event record");
        }
        hipError_t e = launch();
        if (e != hipSuccess) return hip_fail(e, name);
        if (timed && (e = hipEventRecord((hipEvent_t)p->ev_stop, s)) != hipSuccess) return hip_fail(e, "event record");
        ++n;
        if (p) p->n_launches = n;
        return MOE_OK;
    }
};

inline bool act_ok(int a) { return a == MOE_ACT_F32 || a == MOE_ACT_BF16; }
inline int act_size(int a) { return a == MOE_ACT_F32 ? 4 : 2; }

// rows of T x n elements of `size` bytes, ld apart, starting at p
inline int check_rows(const char *name, const void *p, int64_t ld, int T, int n, int size)
{
    if (!p) return set_error(MOE_ERR_INVALID_ARG, "%s is NULL", name);
    if ((uintptr_t)p % size) return set_error(MOE_ERR_INVALID_ARG, "%s is not aligned to its elements", name);
    if (ld < n && T > 1) return set_error(MOE_ERR_INVALID_ARG, "%s: rows of %d elements only %lld apart", name, n, (long long)ld);
    if (ld < 0 || ld > ((int64_t)1 << 40)) return set_error(MOE_ERR_INVALID_ARG, "%s: stride %lld", name, (long long)ld);
    return MOE_OK;
}

inline int check_scored(const moe_router *R)
{
    if (!R) return set_error(MOE_ERR_INVALID_ARG, "router is NULL");
    if (R->hidden < 8 || R->hidden % 8) return set_error(MOE_ERR_INVALID_ARG, "hidden=%d must be a positive multiple of 8", R->hidden);
    if (R->n_experts < 1 || R->n_experts > 1024) return set_error(MOE_ERR_INVALID_ARG, "n_experts=%d outside [1,1024]", R->n_experts);
    if (R->score != MOE_SCORE_SIGMOID && R->score != MOE_SCORE_SOFTMAX) return set_error(MOE_ERR_INVALID_ARG, "score=%d unknown", R->score);
    if (R->n_groups < 1 || R->n_groups > 64 || R->n_experts % R->n_groups)
        return set_error(MOE_ERR_INVALID_ARG, "n_groups=%d outside [1,64] or not a divisor of n_experts=%d", R->n_groups, R->n_experts);
    if (R->keep_groups < 1 || R->keep_groups > R->n_groups)
        return set_error(MOE_ERR_INVALID_ARG, "keep_groups=%d outside [1,n_groups]", R->keep_groups);
    const int most = R->keep_groups * (R->n_experts / R->n_groups);
    if (R->top_k < 1 || R->top_k > most || R->top_k > 64)
        return set_error(MOE_ERR_INVALID_ARG, "top_k=%d outside [1,%d]", R->top_k, most < 64 ? most : 64);
    if (R->flags & ~MOE_ROUTER_RENORM) return set_error(MOE_ERR_INVALID_ARG, "flags=%#x: unknown bits", R->flags);
    if (!R->w_router) return set_error(MOE_ERR_INVALID_ARG, "w_router is NULL");
    if ((uintptr_t)R->w_router % 16 || (uintptr_t)R->bias % 4)
        return set_error(MOE_ERR_INVALID_ARG, "w_router must be 16-byte and bias 4-byte aligned");
    return MOE_OK;
}

inline int check_linear(const moe_linear *W)
{
    if (!W) return set_error(MOE_ERR_INVALID_ARG, "linear is NULL");
    if (W->in_features < 1 || W->in_features > 131071)
        return set_error(MOE_ERR_INVALID_ARG, "in_features=%d outside [1,131071]", W->in_features);
    if (W->out_features < 1) return set_error(MOE_ERR_INVALID_ARG, "out_features=%d < 1", W->out_features);
    if (!W->w || !W->w_scale) return set_error(MOE_ERR_INVALID_ARG, "linear weights are NULL");
    if ((uintptr_t)W->w % 16 || W->ldw % 16 || W->ldw < W->in_features || W->ldw > ((int64_t)1 << 40))
        return set_error(MOE_ERR_INVALID_ARG, "w must be 16-byte aligned with ldw=%lld a multiple of 16 of at least in_features",
                         (long long)W->ldw);
    if ((uintptr_t)W->w_scale % 4 || (uintptr_t)W->bias % 4)
        return set_error(MOE_ERR_INVALID_ARG, "w_scale and bias must be 4-byte aligned");
    return MOE_OK;
}

inline int check_norm(const moe_norm *N)
{
    if (!N) return set_error(MOE_ERR_INVALID_ARG, "norm is NULL");
    if (N->hidden < 1 || N->hidden > ROWS_MAX) return set_error(MOE_ERR_INVALID_ARG, "hidden=%d outside [1,%d]", N->hidden, ROWS_MAX);
    if (!(N->eps >= 0.0f)) return set_error(MOE_ERR_INVALID_ARG, "eps=%g is negative or NaN", (double)N->eps);
    if (!N->weight || (uintptr_t)N->weight % 4) return set_error(MOE_ERR_INVALID_ARG, "weight is NULL or not 4-byte aligned");
    return MOE_OK;
}

}  // namespace moe
