// C ABI of the operators around the routed experts (include/moe.h: scored
// routing, rows in 8 bits, the int8 linear layer): host-side argument
// validation and the launch sequences.
#include <hip/hip_runtime.h>

#include "linear.h"
#include "moe.h"
#include "route.h"
#include "rows.h"
#include "scored.h"
#include "status.h"

using namespace moe;

namespace {

constexpr size_t ALIGN = 256;
constexpr int MAX_ROWS = 1 << 22;                // rows of a call, up to 1024 threads each in a launch of fewer than 2^32
size_t align_up(size_t v) { return (v + ALIGN - 1) / ALIGN * ALIGN; }

int hip_fail(hipError_t e, const char *what) { return set_error(MOE_ERR_HIP, "%s: %s", what, hipGetErrorString(e)); }

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

bool act_ok(int a) { return a == MOE_ACT_F32 || a == MOE_ACT_BF16; }
int act_size(int a) { return a == MOE_ACT_F32 ? 4 : 2; }

// rows of T x n elements of `size` bytes, ld apart, starting at p
int check_rows(const char *name, const void *p, int64_t ld, int T, int n, int size)
{
    if (!p) return set_error(MOE_ERR_INVALID_ARG, "%s is NULL", name);
    if ((uintptr_t)p % size) return set_error(MOE_ERR_INVALID_ARG, "%s is not aligned to its elements", name);
    if (ld < n && T > 1) return set_error(MOE_ERR_INVALID_ARG, "%s: rows of %d elements only %lld apart", name, n, (long long)ld);
    if (ld < 0 || ld > ((int64_t)1 << 40)) return set_error(MOE_ERR_INVALID_ARG, "%s: stride %lld", name, (long long)ld);
    return MOE_OK;
}

int check_scored(const moe_router *R)
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

// Workspace of a call (p.x_bf16 and p.softmax decide the router)
size_t scored_ws(ScoredPass &p, char *base)
{
    const bool split = scored_split(p.T, p.E, p.softmax, p.x_bf16);
    size_t off = 0;
    auto take = [&](size_t bytes) {
        char *at = base + off;
        off = align_up(off + bytes);
        return (void *)at;
    };
    p.logits = take(scored_logit_bytes(p.T, p.H, p.E, split));
    if (split) {
        p.wsplit = take(scored_split_bytes(p.H, p.E));
        p.wnorm = (float *)take((size_t)p.E * sizeof(float));
        p.xnorm = (float *)take((size_t)scored_split_parts(p.T, p.H, p.E) * p.T * sizeof(float));
        p.open = (int32_t *)take(scored_open_bytes(p.T));
    }
    if (!scored_group_fits(p.T, p.E)) {
        p.rank = (int32_t *)take((size_t)p.T * p.k * sizeof(int32_t));
        p.tile_counts = (int32_t *)take((size_t)(((int64_t)p.T + 63) / 64) * p.E * sizeof(int32_t));
    }
    return off;
}

int check_linear(const moe_linear *W)
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

}  // namespace

extern "C" {

size_t moe_route_scored_workspace_bytes(const moe_router *R, int T)
{
    if (T < 0 || check_scored(R)) return 0;
    ScoredPass p{};
    p.T = T; p.H = R->hidden; p.E = R->n_experts; p.k = R->top_k;
    p.softmax = R->score == MOE_SCORE_SOFTMAX;
    size_t most = 0;
    auto count = [&](int t) {
        p.T = t;
        for (int bf16 = 0; bf16 < 2; ++bf16) {   // enough for either activation type
            p.x_bf16 = bf16;
            const size_t b = scored_ws(p, nullptr);
            most = b > most ? b : most;
        }
    };
    // ... and for every smaller batch: H is cut into parts by whole tiles of 64 and
    // 128 tokens, and not at all past 512 of the smaller ones, so what a call needs
    // grows from one multiple of 64 to the next but where the split router begins
    count(T);
    for (int t = 64; t < T && t <= 64 * 512; t += 64) count(t);
    const int last = scored_split_above(p.E);
    if (last < T) count(last);
    return most;
}

int moe_route_scored(const moe_router *R, const void *x, int act, int64_t ldx, int T, int32_t *topk_idx,
                     float *topk_w, int32_t *offsets, int32_t *perm, int32_t *inv, void *ws, size_t ws_bytes,
                     void *stream, moe_profile *prof)
{
    int rc = check_scored(R);
    if (rc) return rc;
    if (T < 0) return set_error(MOE_ERR_INVALID_ARG, "T=%d < 0", T);
    if (!act_ok(act)) return set_error(MOE_ERR_INVALID_ARG, "act=%d unknown", act);
    if (prof) prof->n_launches = 0;
    if (T == 0) return MOE_OK;
    if ((int64_t)T * R->top_k > (1 << 30)) return set_error(MOE_ERR_INVALID_ARG, "T*k too large");
    if (T >= MAX_ROWS) return set_error(MOE_ERR_UNSUPPORTED, "T=%d: more rows than one call takes", T);
    if ((rc = check_rows("x", x, ldx, T, R->hidden, act_size(act)))) return rc;
    if (!topk_idx || !topk_w || !offsets || !perm || !inv) return set_error(MOE_ERR_INVALID_ARG, "NULL tensor argument");
    if (!ws) return set_error(MOE_ERR_INVALID_ARG, "workspace is NULL");
    if ((uintptr_t)x % 16 || ldx % 8 || (uintptr_t)ws % 16)
        return set_error(MOE_ERR_INVALID_ARG, "x and the workspace must be 16-byte aligned, ldx a multiple of 8");
    ScoredPass p{};
    p.T = T; p.H = R->hidden; p.E = R->n_experts; p.k = R->top_k;
    p.softmax = R->score == MOE_SCORE_SOFTMAX; p.groups = R->n_groups; p.keep = R->keep_groups;
    p.renorm = (R->flags & MOE_ROUTER_RENORM) != 0; p.scale = R->scale;
    p.x = x; p.x_bf16 = act == MOE_ACT_BF16; p.ldx = ldx; p.w = R->w_router; p.bias = R->bias;
    p.topk_idx = topk_idx; p.topk_w = topk_w; p.offsets = offsets; p.perm = perm; p.inv = inv;
    const size_t need = scored_ws(p, (char *)ws);
    if (ws_bytes < need) return set_error(MOE_ERR_WORKSPACE, "workspace %zu < %zu bytes", ws_bytes, need);

    const hipStream_t s = (hipStream_t)stream;
    Launcher run{prof, s};
    auto plain = [](auto f) { return [f] { f(); return hipGetLastError(); }; };
    if (scored_split(T, p.E, p.softmax, p.x_bf16)) {
        if ((rc = run("scored_split", [&] { return launch_scored_split(p, s); }))) return rc;
        if ((rc = run("scored_split_logits", [&] { return launch_scored_split_logits(p, s); }))) return rc;
    } else if ((rc = run("scored_logits", [&] { return launch_scored_logits(p, s); }))) return rc;
    if ((rc = run("scored_topk", [&] { return launch_scored_topk(p, s); })) || T == 1) return rc;
    if (scored_group_fits(T, p.E)) return run("scored_group", [&] { return launch_scored_group(p, s); });
    if ((rc = run("route_rank", plain([&] { launch_route_rank(topk_idx, T, p.E, p.k, p.rank, p.tile_counts, s); })))) return rc;
    if ((rc = run("route_scan", plain([&] { launch_route_scan(T, p.E, p.k, p.tile_counts, offsets, s); })))) return rc;
    return run("route_scatter", plain([&] {
        launch_route_scatter(topk_idx, p.rank, p.tile_counts, offsets, T, p.E, p.k, perm, inv, s);
    }));
}

int moe_residual_norm(const moe_norm *N, int T, const void *x, int act_x, int64_t ldx, const void *residual,
                      int act_res, int64_t ldres, void *sum, int64_t ldsum, void *out, int act_out, int64_t ldout,
                      int8_t *q, int64_t ldq, float *q_scale, void *stream, moe_profile *prof)
{
    int rc;
    if (!N) return set_error(MOE_ERR_INVALID_ARG, "norm is NULL");
    if (N->hidden < 1 || N->hidden > ROWS_MAX) return set_error(MOE_ERR_INVALID_ARG, "hidden=%d outside [1,%d]", N->hidden, ROWS_MAX);
    if (!(N->eps >= 0.0f)) return set_error(MOE_ERR_INVALID_ARG, "eps=%g is negative or NaN", (double)N->eps);
    if (!N->weight || (uintptr_t)N->weight % 4) return set_error(MOE_ERR_INVALID_ARG, "weight is NULL or not 4-byte aligned");
    if (T < 0) return set_error(MOE_ERR_INVALID_ARG, "T=%d < 0", T);
    if (!act_ok(act_x) || (residual && !act_ok(act_res)) || (out && !act_ok(act_out)))
        return set_error(MOE_ERR_INVALID_ARG, "unknown activation type");
    if (prof) prof->n_launches = 0;
    if (T == 0) return MOE_OK;
    if (sum && !residual) return set_error(MOE_ERR_INVALID_ARG, "sum without a residual");
    if (!out && !q) return set_error(MOE_ERR_INVALID_ARG, "neither out nor q is given");
    if (!q != !q_scale) return set_error(MOE_ERR_INVALID_ARG, "q and q_scale come together");
    const int H = N->hidden;
    if (T >= MAX_ROWS) return set_error(MOE_ERR_UNSUPPORTED, "T=%d: more rows than one call takes", T);
    if ((rc = check_rows("x", x, ldx, T, H, act_size(act_x)))) return rc;
    if (residual && (rc = check_rows("residual", residual, ldres, T, H, act_size(act_res)))) return rc;
    if (sum && (rc = check_rows("sum", sum, ldsum, T, H, act_size(act_res)))) return rc;
    if (out && (rc = check_rows("out", out, ldout, T, H, act_size(act_out)))) return rc;
    if (q && (rc = check_rows("q", q, ldq, T, H, 1))) return rc;
    if ((uintptr_t)q_scale % 4) return set_error(MOE_ERR_INVALID_ARG, "q_scale is not 4-byte aligned");
    RowsPass p{};
    p.mode = ROWS_NORM; p.T = T; p.n = H;
    p.x = x; p.x_bf16 = act_x == MOE_ACT_BF16; p.ldx = ldx;
    p.res = residual; p.res_bf16 = act_res == MOE_ACT_BF16; p.ldres = ldres;
    p.sum = sum; p.ldsum = ldsum;
    p.out = out; p.out_bf16 = act_out == MOE_ACT_BF16; p.ldout = ldout;
    p.q = q; p.ldq = ldq; p.q_scale = q_scale;
    p.weight = N->weight; p.eps = N->eps;
    Launcher run{prof, (hipStream_t)stream};
    return run("residual_norm", [&] { return launch_rows(p, (hipStream_t)stream); });
}

int moe_quant_i8(const void *x, int act, int64_t ldx, int T, int K, int flags, int8_t *q, int64_t ldq, float *q_scale,
                 void *stream, moe_profile *prof)
{
    int rc;
    if (K < 1 || K > ROWS_MAX) return set_error(MOE_ERR_INVALID_ARG, "K=%d outside [1,%d]", K, ROWS_MAX);
    if (T < 0) return set_error(MOE_ERR_INVALID_ARG, "T=%d < 0", T);
    if (!act_ok(act)) return set_error(MOE_ERR_INVALID_ARG, "act=%d unknown", act);
    if (flags & ~MOE_Q8_SWIGLU) return set_error(MOE_ERR_INVALID_ARG, "flags=%#x: unknown bits", flags);
    if (prof) prof->n_launches = 0;
    if (T == 0) return MOE_OK;
    const bool swiglu = (flags & MOE_Q8_SWIGLU) != 0;
    if (T >= MAX_ROWS) return set_error(MOE_ERR_UNSUPPORTED, "T=%d: more rows than one call takes", T);
    if ((rc = check_rows("x", x, ldx, T, swiglu ? 2 * K : K, act_size(act)))) return rc;
    if ((rc = check_rows("q", q, ldq, T, K, 1))) return rc;
    if (!q_scale || (uintptr_t)q_scale % 4) return set_error(MOE_ERR_INVALID_ARG, "q_scale is NULL or not 4-byte aligned");
    RowsPass p{};
    p.mode = swiglu ? ROWS_SWIGLU : ROWS_QUANT; p.T = T; p.n = K;
    p.x = x; p.x_bf16 = act == MOE_ACT_BF16; p.ldx = ldx;
    p.q = q; p.ldq = ldq; p.q_scale = q_scale;
    Launcher run{prof, (hipStream_t)stream};
    return run("quant_i8", [&] { return launch_rows(p, (hipStream_t)stream); });
}

size_t moe_linear_i8_workspace_bytes(const moe_linear *W, int T)
{
    if (T < 0 || check_linear(W)) return 0;
    return linear_ws_bytes(T, W->out_features, W->in_features);
}

int moe_linear_i8(const moe_linear *W, int T, const int8_t *x, int64_t ldx, const float *x_scale, const void *add,
                  int64_t ldadd, void *y, int act_y, int64_t ldy, void *ws, size_t ws_bytes, void *stream,
                  moe_profile *prof)
{
    int rc = check_linear(W);
    if (rc) return rc;
    if (T < 0) return set_error(MOE_ERR_INVALID_ARG, "T=%d < 0", T);
    if (!act_ok(act_y)) return set_error(MOE_ERR_INVALID_ARG, "act_y=%d unknown", act_y);
    if (prof) prof->n_launches = 0;
    if (T == 0) return MOE_OK;
    const int K = W->in_features, N = W->out_features;
    if ((rc = check_rows("x", x, ldx, T, K, 1))) return rc;
    if ((uintptr_t)x % 16 || ldx % 16) return set_error(MOE_ERR_INVALID_ARG, "x must be 16-byte aligned with ldx a multiple of 16");
    if (!x_scale || (uintptr_t)x_scale % 4) return set_error(MOE_ERR_INVALID_ARG, "x_scale is NULL or not 4-byte aligned");
    if ((rc = check_rows("y", y, ldy, T, N, act_size(act_y)))) return rc;
    if (add && (rc = check_rows("add", add, ldadd, T, N, act_size(act_y)))) return rc;
    // a launch holds fewer than 2^32 threads: tiles of at least 32 x 64 with 256 threads, 16 channels with 1024
    if (((int64_t)T + 31) / 32 * (((int64_t)N + 63) / 64) >= ((int64_t)1 << 24) || N >= 1 << 26)
        return set_error(MOE_ERR_UNSUPPORTED, "T=%d x out_features=%d: too many tiles for one call", T, N);
    const size_t need = linear_needs_ws(T, N, K) ? linear_ws_bytes(T, N, K) : 0;
    if (need && !ws) return set_error(MOE_ERR_INVALID_ARG, "workspace is NULL");
    if ((uintptr_t)ws % 16) return set_error(MOE_ERR_INVALID_ARG, "the workspace must be 16-byte aligned");
    if (ws_bytes < need) return set_error(MOE_ERR_WORKSPACE, "workspace %zu < %zu bytes", ws_bytes, need);
    LinearPass p{};
    p.T = T; p.N = N; p.K = K;
    p.x = x; p.w = W->w; p.ldx = ldx; p.ldw = W->ldw;
    p.x_scale = x_scale; p.w_scale = W->w_scale; p.bias = W->bias;
    p.add = add; p.ldadd = ldadd; p.y = y; p.ldy = ldy; p.y_bf16 = act_y == MOE_ACT_BF16;
    p.ws = ws;
    Launcher run{prof, (hipStream_t)stream};
    return run("linear_i8", [&] { return launch_linear(p, (hipStream_t)stream); });
}

}  // extern "C"
