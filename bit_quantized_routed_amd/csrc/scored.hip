// Scored router on gfx950: sigmoid or softmax scores, a selection-only bias,
// group-limited top-k and the weights of the chosen experts.  Scores and their
// comparisons are fp64, as in the plain router (route.hip).
#include "common.h"
#include "route_dev.h"
#include "scored.h"

namespace moe {

namespace {

// One wave per (expert, 8 tokens): each lane strides over h, a fixed butterfly
// adds the 64 partial sums.
template <bool XBF16>
__global__ __launch_bounds__(64) void scored_logits(ScoredPass p)
{
    const int e = blockIdx.x, t0 = blockIdx.y * 8, lane = threadIdx.x;
    const int nt = min(8, p.T - t0);
    double acc[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = 0.0;
    const float *w = p.w + (size_t)e * p.H;
    for (int h = lane; h < p.H; h += 64) {
        const double wv = (double)w[h];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int64_t at = (int64_t)(t0 + min(i, nt - 1)) * p.ldx + h;
            const double xv = XBF16 ? (double)bf16_bits_to_f32(((const uint16_t *)p.x)[at]) : (double)((const float *)p.x)[at];
            acc[i] = fma(xv, wv, acc[i]);
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
#pragma unroll
        for (int off = 32; off > 0; off >>= 1) acc[i] += __shfl_xor(acc[i], off, 64);
        if (lane == i && i < nt) p.logits[(int64_t)(t0 + i) * p.E + e] = acc[i];
    }
}

__device__ __forceinline__ double wave_sum_f64(double v)
{
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, 64);
    return v;
}

// Scores of one token, one wave: lane l holds experts l, l + 64, ...  On
// return pr holds the scores p (0 for NaN logits and past E) and c the
// selection values p + bias (-inf for NaN and past E).
template <int MAXPL>
__device__ __forceinline__ void token_scores(const ScoredPass &p, const double *l, int lane, double pr[MAXPL],
                                             double c[MAXPL])
{
    double lg[MAXPL], top = -INFINITY;
#pragma unroll
    for (int i = 0; i < MAXPL; ++i) {
        const int e = lane + 64 * i;
        const double v = e < p.E ? l[e] : -INFINITY;
        c[i] = v != v ? -INFINITY : 0.0;
        lg[i] = v != v ? -INFINITY : v;
        top = fmax(top, lg[i]);
    }
    if (p.softmax) {
        top = wave_max_f64(top);
        double sum = 0.0;
#pragma unroll
        for (int i = 0; i < MAXPL; ++i) {
            // the largest logit's term is 1, also where it is infinite
            pr[i] = lg[i] == -INFINITY ? 0.0 : lg[i] == top ? 1.0 : exp(lg[i] - top);
            sum += pr[i];
        }
        sum = wave_sum_f64(sum);
        const double inv = sum > 0.0 ? 1.0 / sum : 0.0;
#pragma unroll
        for (int i = 0; i < MAXPL; ++i) pr[i] *= inv;
    } else {
#pragma unroll
        for (int i = 0; i < MAXPL; ++i) pr[i] = lg[i] == -INFINITY ? 0.0 : 1.0 / (1.0 + exp(-lg[i]));
    }
#pragma unroll
    for (int i = 0; i < MAXPL; ++i) {
        const int e = lane + 64 * i;
        if (e >= p.E) { c[i] = -INFINITY; continue; }
        const double b = p.bias ? (double)p.bias[e] : 0.0;
        const double v = c[i] + pr[i] + b;       // c[i] is -inf for a NaN logit
        c[i] = v != v ? -INFINITY : v;
    }
}

// Group limit of one token, one wave: selection values of the groups that are
// not among the `keep` best become -inf.  cs: this wave's LDS copy of c, [E];
// gs: its group scores, [groups].
template <int MAXPL>
__device__ __forceinline__ void limit_groups(const ScoredPass &p, int lane, double c[MAXPL], double *cs, double *gs)
{
    const int G = p.groups, size = p.E / G;
#pragma unroll
    for (int i = 0; i < MAXPL; ++i)
        if (lane + 64 * i < p.E) cs[lane + 64 * i] = c[i];
    __builtin_amdgcn_wave_barrier();
    for (int g = lane; g < G; g += 64) {
        double a = -INFINITY, b = -INFINITY;     // the two largest
        for (int j = 0; j < size; ++j) {
            const double v = cs[g * size + j];
            b = fmax(b, fmin(a, v));
            a = fmax(a, v);
        }
        gs[g] = size > 1 ? a + b : a;
    }
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int i = 0; i < MAXPL; ++i) {
        const int e = lane + 64 * i;
        if (e >= p.E) continue;
        const int g = e / size;
        const double mine = gs[g];
        int r = 0;
        for (int o = 0; o < G; ++o) r += gs[o] > mine || (gs[o] == mine && o < g);
        if (r >= p.keep) c[i] = -INFINITY;
    }
}

// WAVES tokens per work-group, a wave each: k rounds of a wave-wide arg-max
// over (c descending, expert ascending); lane j keeps slot j's expert and score.
constexpr int WAVES = 4;
template <int MAXPL>
__global__ __launch_bounds__(64 * WAVES) void scored_topk(ScoredPass p)
{
    extern __shared__ double lds[];              // groups > keep: [WAVES][E + groups]
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int t = blockIdx.x * WAVES + wave;
    if (t >= p.T) return;
    double pr[MAXPL], c[MAXPL];
    token_scores<MAXPL>(p, p.logits + (int64_t)t * p.E, lane, pr, c);
    if (p.keep < p.groups) {
        double *cs = lds + (size_t)wave * (p.E + p.groups);
        limit_groups<MAXPL>(p, lane, c, cs, cs + p.E);
    }
    uint32_t taken = 0;
    int my_e = 0;
    double my_p = 0.0;
    for (int j = 0; j < p.k; ++j) {
        double bv = -INFINITY, bp = 0.0;
        int be = 0x7fffffff;
#pragma unroll
        for (int i = 0; i < MAXPL; ++i) {
            const int e = lane + 64 * i;
            // e grows with i, so a strict '>' keeps the lowest expert among equals
            if (e < p.E && !((taken >> i) & 1u) && (be == 0x7fffffff || c[i] > bv)) { bv = c[i]; bp = pr[i]; be = e; }
        }
        const int mine = be;
        wave_argmax(bv, be);
        const uint64_t owner = __ballot(mine == be);
        const double sel = readlane_f64(bp, __ffsll((unsigned long long)owner) - 1);
        if (mine == be) taken |= 1u << (be >> 6);
        if (lane == j) { my_e = be; my_p = bv == -INFINITY ? 0.0 : sel; }
    }
    double w = lane < p.k ? my_p : 0.0;
    if (p.renorm) {
        const double sum = wave_sum_f64(w);
        w = sum > 0.0 ? w / sum : 0.0;
    }
    if (lane < p.k) {
        p.topk_idx[(int64_t)t * p.k + lane] = my_e;
        p.topk_w[(int64_t)t * p.k + lane] = (float)(w * (double)p.scale);
    }
}

}  // namespace

size_t scored_logit_bytes(int T, int E) { return (size_t)T * E * sizeof(double); }

void launch_scored_logits(const ScoredPass &p, hipStream_t s)
{
    const dim3 grid((unsigned)p.E, (unsigned)((p.T + 7) / 8));
    if (p.x_bf16) scored_logits<true><<<grid, 64, 0, s>>>(p);
    else scored_logits<false><<<grid, 64, 0, s>>>(p);
}

void launch_scored_topk(const ScoredPass &p, hipStream_t s)
{
    const size_t lds = p.keep < p.groups ? (size_t)WAVES * (p.E + p.groups) * sizeof(double) : 0;
    const unsigned grid = (unsigned)((p.T + WAVES - 1) / WAVES);
    // unrolled for the experts each lane holds (E <= 64 * MAXPL)
#define MOE_TOPK(pl) scored_topk<pl><<<grid, 64 * WAVES, lds, s>>>(p)
    if (p.E <= 64) MOE_TOPK(1);
    else if (p.E <= 128) MOE_TOPK(2);
    else if (p.E <= 256) MOE_TOPK(4);
    else if (p.E <= 512) MOE_TOPK(8);
    else MOE_TOPK(16);
#undef MOE_TOPK
}

}  // namespace moe
