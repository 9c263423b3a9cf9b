// C ABI of the operators around the routed experts (include/moe.h: scored
// routing, rows in 8 bits, the int8 linear layer): host-side argument
// validation and the launch sequences.
#include <hip/hip_runtime.h>

#include "adapters.h"
#include "block.h"
#include "dense_check.h"
#include "linear.h"
#include "route.h"
#include "scored.h"

using namespace moe;

namespace {

constexpr size_t ALIGN = 256;
size_t align_up(size_t v) { return (v + ALIGN - 1) / ALIGN * ALIGN; }

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

// Checks a block, and fills in what p takes from it.
int check_block(const moe_block *B, int T, BlockPass &p)
{
    if (!B) return set_error(MOE_ERR_INVALID_ARG, "block is NULL");
    int rc;
    if ((rc = check_norm(B->norm)) || (rc = check_scored(B->router))) return rc;
    const moe_layer *L = B->layer;
    if (!L) return set_error(MOE_ERR_INVALID_ARG, "layer is NULL");
    if (!act_ok(B->act_n)) return set_error(MOE_ERR_INVALID_ARG, "act_n=%d unknown", B->act_n);
    if (!B->gate_up != !B->down) return set_error(MOE_ERR_INVALID_ARG, "gate_up and down come together");
    const int H = B->norm->hidden, E = L->n_experts, k = L->top_k;
    if (L->hidden != H || B->router->hidden != H) return set_error(MOE_ERR_INVALID_ARG, "norm, router and layer differ in hidden");
    if (B->router->n_experts != E || B->router->top_k != k) return set_error(MOE_ERR_INVALID_ARG, "router and layer differ in experts or top_k");
    if (L->inter < 8 || L->inter % 8) return set_error(MOE_ERR_INVALID_ARG, "inter=%d must be a positive multiple of 8", L->inter);
    if (!L->w_gate || !L->w_up || !L->w_down || !L->codebook) return set_error(MOE_ERR_INVALID_ARG, "layer weights are NULL");
    if (((uintptr_t)L->w_gate | (uintptr_t)L->w_up | (uintptr_t)L->w_down | (uintptr_t)L->codebook | (uintptr_t)B->norm->weight) % 16)
        return set_error(MOE_ERR_INVALID_ARG, "the norm's and the layer's weights must be 16-byte aligned");
    if (L->fmt_gate_up != MOE_FMT_CB2 || L->fmt_down != MOE_FMT_Q2K)
        return set_error(MOE_ERR_UNSUPPORTED, "formats %d and %d: CB2 gate/up and Q2K down are needed", L->fmt_gate_up, L->fmt_down);
    if (L->sh_inter || L->flags || L->expert_slot)
        return set_error(MOE_ERR_UNSUPPORTED, "a layer with a shared expert of its own, flags or an expert map");
    if (B->gate_up) {
        if ((rc = check_linear(B->gate_up)) || (rc = check_linear(B->down))) return rc;
        const int sh = B->down->in_features;
        if (B->gate_up->in_features != H || B->down->out_features != H || B->gate_up->out_features != 2 * (int64_t)sh)
            return set_error(MOE_ERR_INVALID_ARG, "shared expert: gate_up %d x %d, down %d x %d do not fit hidden %d", B->gate_up->out_features,
                             B->gate_up->in_features, B->down->out_features, sh, H);
        p.sh = sh;
        p.sh_up = B->gate_up->w; p.ld_up = B->gate_up->ldw; p.up_scale = B->gate_up->w_scale; p.up_bias = B->gate_up->bias;
        p.sh_down = B->down->w; p.ld_down = B->down->ldw; p.down_scale = B->down->w_scale; p.down_bias = B->down->bias;
    }
    if (H > BLOCK_MAX_DIM || L->inter > BLOCK_MAX_DIM || p.sh > BLOCK_MAX_DIM || E > BLOCK_MAX_E || k > BLOCK_MAX_K || T > BLOCK_MAX_T)
        return set_error(MOE_ERR_UNSUPPORTED, "hidden=%d, inter=%d, shared=%d, n_experts=%d, top_k=%d, T=%d: more than the block takes", H,
                         L->inter, p.sh, E, k, T);
    p.T = T; p.H = H; p.I = L->inter; p.E = E; p.k = k;
    p.n_bf16 = B->act_n == MOE_ACT_BF16; p.norm_w = B->norm->weight; p.eps = B->norm->eps;
    p.gate = (const uint8_t *)L->w_gate; p.up = (const uint8_t *)L->w_up; p.down = (const uint8_t *)L->w_down;
    p.codebook = L->codebook;
    const moe_router *R = B->router;
    ScoredPass &r = p.route;
    r.T = T; r.H = H; r.E = E; r.k = k;
    r.softmax = R->score == MOE_SCORE_SOFTMAX; r.groups = R->n_groups; r.keep = R->keep_groups;
    r.renorm = (R->flags & MOE_ROUTER_RENORM) != 0; r.scale = R->scale; r.w = R->w_router; r.bias = R->bias;
    return MOE_OK;
}

int check_adapters(const moe_adapter_set *W)
{
    if (!W) return set_error(MOE_ERR_INVALID_ARG, "adapter set is NULL");
    if (W->in_features < 1 || W->in_features > (1 << 24)) return set_error(MOE_ERR_INVALID_ARG, "in_features=%d outside [1,2^24]", W->in_features);
    if (W->out_features < 1 || W->out_features > (1 << 24)) return set_error(MOE_ERR_INVALID_ARG, "out_features=%d outside [1,2^24]", W->out_features);
    if (W->n_adapters < 1 || W->n_adapters > ADAPT_MAX) return set_error(MOE_ERR_INVALID_ARG, "n_adapters=%d outside [1,%d]", W->n_adapters, ADAPT_MAX);
    if (W->rank < 1 || W->rank > ADAPT_MAX_RANK) return set_error(MOE_ERR_INVALID_ARG, "rank=%d outside [1,%d]", W->rank, ADAPT_MAX_RANK);
    if (W->parts < 1 || W->out_features % W->parts || W->parts > ADAPT_MAX_WIDTH / W->rank)
        return set_error(MOE_ERR_INVALID_ARG, "parts=%d: not a divisor of out_features=%d, or parts * rank > %d", W->parts, W->out_features, ADAPT_MAX_WIDTH);
    if (!W->a || !W->b || !W->scale) return set_error(MOE_ERR_INVALID_ARG, "adapter weights are NULL");
    if (((uintptr_t)W->a | (uintptr_t)W->b) % 16 || (uintptr_t)W->scale % 4)
        return set_error(MOE_ERR_INVALID_ARG, "a and b must be 16-byte and scale 4-byte aligned");
    if (W->lda % 8 || W->lda < W->in_features || W->ldb % 8 || W->ldb < W->rank || W->lda > ((int64_t)1 << 40) || W->ldb > ((int64_t)1 << 40))
        return set_error(MOE_ERR_INVALID_ARG, "lda=%lld and ldb=%lld must be multiples of 8 of at least in_features and rank", (long long)W->lda,
                         (long long)W->ldb);
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
    int rc = check_norm(N);
    if (rc) return rc;
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

size_t moe_block_decode_workspace_bytes(const moe_block *B, int T)
{
    BlockPass p{};
    if (T < 0 || check_block(B, T, p)) return 0;
    block_layout(p);
    return block_workspace(p, nullptr) + 240;    // from any multiple of 16 to the next of 256
}

int moe_block_decode(const moe_block *B, int T, const void *x, int act_x, int64_t ldx, const void *residual, int act_res,
                     int64_t ldres, void *sum, int64_t ldsum, float *y, int64_t ldy, int32_t *topk_idx, float *topk_w,
                     int32_t *offsets, int32_t *perm, int32_t *inv, void *ws, size_t ws_bytes, void *stream,
                     moe_profile *prof)
{
    if (T < 0) return set_error(MOE_ERR_INVALID_ARG, "T=%d < 0", T);
    BlockPass p{};
    int rc = check_block(B, T, p);
    if (rc) return rc;
    if (!act_ok(act_x) || (residual && !act_ok(act_res))) return set_error(MOE_ERR_INVALID_ARG, "unknown activation type");
    if (prof) prof->n_launches = 0;
    if (T == 0) return MOE_OK;
    if (sum && !residual) return set_error(MOE_ERR_INVALID_ARG, "sum without a residual");
    if ((rc = check_rows("x", x, ldx, T, p.H, act_size(act_x)))) return rc;
    if (residual && (rc = check_rows("residual", residual, ldres, T, p.H, act_size(act_res)))) return rc;
    if (sum && (rc = check_rows("sum", sum, ldsum, T, p.H, act_size(act_res)))) return rc;
    if ((rc = check_rows("y", y, ldy, T, p.H, 4))) return rc;
    if (!topk_idx || !topk_w || !offsets || !perm || !inv) return set_error(MOE_ERR_INVALID_ARG, "NULL tensor argument");
    if (!ws) return set_error(MOE_ERR_INVALID_ARG, "workspace is NULL");
    if (((uintptr_t)x | (uintptr_t)residual | (uintptr_t)sum | (uintptr_t)ws) % 16 || (ldx | (residual ? ldres : 0) | (sum ? ldsum : 0)) % 8)
        return set_error(MOE_ERR_INVALID_ARG, "x, residual, sum and the workspace must be 16-byte aligned, their strides multiples of 8");
    block_layout(p);
    const size_t need = block_workspace(p, (char *)ws);
    if (ws_bytes < need) return set_error(MOE_ERR_WORKSPACE, "workspace %zu < %zu bytes", ws_bytes, need);
    p.x = x; p.x_bf16 = act_x == MOE_ACT_BF16; p.ldx = ldx;
    p.res = residual; p.res_bf16 = act_res == MOE_ACT_BF16; p.ldres = ldres;
    p.sum = sum; p.ldsum = ldsum;
    p.y = y; p.ldy = ldy;
    ScoredPass &r = p.route;
    r.topk_idx = topk_idx; r.topk_w = topk_w; r.offsets = offsets; r.perm = perm; r.inv = inv;
    const hipStream_t s = (hipStream_t)stream;
    Launcher run{prof, s};
    if ((rc = run("block_norm", [&] { return launch_block_norm(p, s); }))) return rc;
    return run("block", [&] { return launch_block(p, s); });
}

int moe_adapter_tiles(int T, int n_adapters)
{
    return T < 1 || T > ADAPT_MAX_T || n_adapters < 1 || n_adapters > ADAPT_MAX ? 0 : adapter_tiles(T, n_adapters);
}

int moe_adapter_plan(const int32_t *ids, int T, int n_adapters, int32_t *order, int32_t *offsets, int32_t *tiles, void *stream,
                     moe_profile *prof)
{
    if (T < 0) return set_error(MOE_ERR_INVALID_ARG, "T=%d < 0", T);
    if (n_adapters < 1 || n_adapters > ADAPT_MAX) return set_error(MOE_ERR_INVALID_ARG, "n_adapters=%d outside [1,%d]", n_adapters, ADAPT_MAX);
    if (prof) prof->n_launches = 0;
    if (T == 0) return MOE_OK;
    if (T > ADAPT_MAX_T) return set_error(MOE_ERR_UNSUPPORTED, "T=%d: more tokens than one plan takes", T);
    if (!ids || !order || !offsets || !tiles) return set_error(MOE_ERR_INVALID_ARG, "NULL tensor argument");
    if (((uintptr_t)ids | (uintptr_t)order | (uintptr_t)offsets) % 4 || (uintptr_t)tiles % 8)
        return set_error(MOE_ERR_INVALID_ARG, "ids, order and offsets must be 4-byte, tiles 8-byte aligned");
    Launcher run{prof, (hipStream_t)stream};
    return run("adapter_plan", [&] {
        return launch_adapter_plan(ids, T, n_adapters, order, offsets, (AdapterTile *)tiles, (hipStream_t)stream);
    });
}

size_t moe_adapters_workspace_bytes(const moe_adapter_set *W, int T)
{
    if (T < 0 || T > ADAPT_MAX_T || check_adapters(W)) return 0;
    return align_up(adapter_low_bytes(T, W->in_features, W->parts * ((W->rank + 7) & ~7), W->n_adapters));
}

int moe_adapters(const moe_adapter_set *W, int T, const int32_t *order, const int32_t *offsets, const int32_t *tiles,
                 const void *x, int kind_x, int64_t ldx, const float *x_scale, const void *add, int64_t ldadd, void *y,
                 int act_y, int64_t ldy, void *ws, size_t ws_bytes, void *stream, moe_profile *prof)
{
    int rc = check_adapters(W);
    if (rc) return rc;
    if (T < 0) return set_error(MOE_ERR_INVALID_ARG, "T=%d < 0", T);
    if (kind_x != MOE_ADAPT_F32 && kind_x != MOE_ADAPT_BF16 && kind_x != MOE_ADAPT_I8) return set_error(MOE_ERR_INVALID_ARG, "kind_x=%d unknown", kind_x);
    if (!act_ok(act_y)) return set_error(MOE_ERR_INVALID_ARG, "act_y=%d unknown", act_y);
    if (prof) prof->n_launches = 0;
    if (T == 0) return MOE_OK;
    if (T > ADAPT_MAX_T) return set_error(MOE_ERR_UNSUPPORTED, "T=%d: more tokens than one plan takes", T);
    const size_t need = (size_t)adapter_k_parts(T, W->in_features, W->n_adapters) * T * W->parts * ((W->rank + 7) & ~7) * sizeof(float);
    if (!ws || (uintptr_t)ws % 16) return set_error(MOE_ERR_INVALID_ARG, "the workspace is NULL or not 16-byte aligned");
    if (ws_bytes < need) return set_error(MOE_ERR_WORKSPACE, "workspace %zu < %zu bytes", ws_bytes, need);
    if (!order || !offsets || !tiles) return set_error(MOE_ERR_INVALID_ARG, "the plan is NULL");
    if (((uintptr_t)order | (uintptr_t)offsets) % 4 || (uintptr_t)tiles % 8) return set_error(MOE_ERR_INVALID_ARG, "the plan is not aligned");
    if ((rc = check_rows("x", x, ldx, T, W->in_features, kind_x == MOE_ADAPT_F32 ? 4 : kind_x == MOE_ADAPT_BF16 ? 2 : 1))) return rc;
    if (!x_scale != (kind_x != MOE_ADAPT_I8) || (uintptr_t)x_scale % 4)
        return set_error(MOE_ERR_INVALID_ARG, "x_scale comes with codes, and only with them, 4-byte aligned");
    if ((rc = check_rows("y", y, ldy, T, W->out_features, act_size(act_y)))) return rc;
    if ((rc = check_rows("add", add, ldadd, T, W->out_features, act_size(act_y)))) return rc;
    AdapterPass p{};
    p.T = T; p.K = W->in_features; p.N = W->out_features; p.n = W->n_adapters; p.rank = W->rank; p.parts = W->parts;
    p.kind = kind_x == MOE_ADAPT_F32 ? ADAPT_F32 : kind_x == MOE_ADAPT_BF16 ? ADAPT_BF16 : ADAPT_I8;
    p.x = x; p.x_scale = x_scale; p.ldx = ldx;
    p.a = (const uint16_t *)W->a; p.b = (const uint16_t *)W->b; p.lda = W->lda; p.ldb = W->ldb; p.scale = W->scale;
    p.add = add; p.ldadd = ldadd; p.y = y; p.ldy = ldy; p.y_bf16 = act_y == MOE_ACT_BF16;
    p.order = order; p.offsets = offsets; p.tiles = (const AdapterTile *)tiles; p.low = (float *)ws;
    const hipStream_t s = (hipStream_t)stream;
    Launcher run{prof, s};
    if ((rc = run("adapter_down", [&] { return launch_adapter_down(p, s); }))) return rc;
    return run("adapter_up", [&] { return launch_adapter_up(p, s); });
}

}  // extern "C"
