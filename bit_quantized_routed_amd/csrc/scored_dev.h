// Device pieces of the scored router's selection, one wave a token: scores,
// groups, top k and weights.  The router's launches (scored.hip) and the MoE block
// for a few tokens (block.hip) share them, so that both choose alike.
#pragma once
#include "common.h"
#include "route_dev.h"
#include "scored.h"

namespace moe {

__device__ __forceinline__ double wave_sum_f64(double v)
{
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, 64);
    return v;
}

__device__ __forceinline__ double sigmoid64(double l) { return l == -INFINITY ? 0.0 : 1.0 / (1.0 + exp(-l)); }

// score + bias, or -inf where the logit or the sum is NaN
__device__ __forceinline__ double with_bias(double l, double pr, float bias)
{
    const double v = l != l ? -INFINITY : pr + (double)bias;
    return v != v ? -INFINITY : v;
}

__device__ __forceinline__ double biased(const ScoredPass &p, int e, double l, double pr)
{
    return with_bias(l, pr, p.bias ? p.bias[e] : 0.0f);
}

// Scores of one token, one wave: lane l holds experts l, l + 64, ...  On
// return pr holds the scores p (0 for NaN logits and past E) and c the
// selection values p + bias (-inf for NaN and past E).
template <int MAXPL>
__device__ __forceinline__ void token_scores(const ScoredPass &p, const double l[MAXPL], int lane, double pr[MAXPL],
                                             double c[MAXPL])
{
    double top = -INFINITY;
    float bias[MAXPL];                           // on their way during the scores' arithmetic
#pragma unroll
    for (int i = 0; i < MAXPL; ++i) bias[i] = p.bias ? p.bias[min(lane + 64 * i, p.E - 1)] : 0.0f;
#pragma unroll
    for (int i = 0; i < MAXPL; ++i) {
        pr[i] = l[i] != l[i] ? -INFINITY : l[i]; // for now the logit, NaN as none
        top = fmax(top, pr[i]);
    }
    if (p.softmax) {
        top = wave_max_f64(top);
        double sum = 0.0;
#pragma unroll
        for (int i = 0; i < MAXPL; ++i) {
            // the largest logit's term is 1, also where it is infinite
            pr[i] = pr[i] == -INFINITY ? 0.0 : pr[i] == top ? 1.0 : exp(pr[i] - top);
            sum += pr[i];
        }
        sum = wave_sum_f64(sum);
        const double inv = sum > 0.0 ? 1.0 / sum : 0.0;
#pragma unroll
        for (int i = 0; i < MAXPL; ++i) pr[i] *= inv;
    } else {
#pragma unroll
        for (int i = 0; i < MAXPL; ++i) pr[i] = sigmoid64(pr[i]);
    }
#pragma unroll
    for (int i = 0; i < MAXPL; ++i) {
        const int e = lane + 64 * i;
        c[i] = e < p.E ? with_bias(l[i], pr[i], bias[i]) : -INFINITY;
    }
}

// Wave-wide maximum of floats by DPP (see wave_max_f64); no NaN among them.
__device__ __forceinline__ float wave_max_f32(float v)
{
    auto step = [](float a, int b) { return fmaxf(a, __uint_as_float((uint32_t)b)); };
    v = step(v, __builtin_amdgcn_mov_dpp((int)__float_as_uint(v), 0xB1, 0xF, 0xF, false));
    v = step(v, __builtin_amdgcn_mov_dpp((int)__float_as_uint(v), 0x4E, 0xF, 0xF, false));
    v = step(v, __builtin_amdgcn_mov_dpp((int)__float_as_uint(v), 0x141, 0xF, 0xF, false));
    v = step(v, __builtin_amdgcn_mov_dpp((int)__float_as_uint(v), 0x140, 0xF, 0xF, false));
    auto row = [&](int l) { return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v), l)); };
    return fmaxf(fmaxf(row(0), row(16)), fmaxf(row(32), row(48)));
}

__device__ __forceinline__ float wave_max(float v) { return wave_max_f32(v); }
__device__ __forceinline__ double wave_max(double v) { return wave_max_f64(v); }

// LDS written before is read after, within one wave: its LDS operations run in
// order, so only the compiler has to keep it.
__device__ __forceinline__ void wave_sync()
{
    asm volatile("" ::: "memory");
    __builtin_amdgcn_wave_barrier();
    asm volatile("" ::: "memory");
}

// The parts of a token's logits added in part order, the parts' loads in
// batches of four.  V: the logits' type; -inf past E.
template <int MAXPL, typename V>
__device__ __forceinline__ void load_logits(const ScoredPass &p, int t, int parts, int lane, V l[MAXPL])
{
    const V *in = (const V *)p.logits + (int64_t)t * p.E;
    const int64_t stride = (int64_t)p.T * p.E;
#pragma unroll
    for (int i = 0; i < MAXPL; ++i) l[i] = 0;
    for (int q0 = 0; q0 < parts; q0 += 4) {
        V v[4][MAXPL];
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int i = 0; i < MAXPL; ++i) {
                v[q][i] = 0;
                if (q0 + q < parts && lane + 64 * i < p.E) v[q][i] = in[(q0 + q) * stride + lane + 64 * i];
            }
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int i = 0; i < MAXPL; ++i) l[i] += v[q][i];
    }
#pragma unroll
    for (int i = 0; i < MAXPL; ++i)
        if (lane + 64 * i >= p.E) l[i] = -INFINITY;
}

// Groups of one token (p.keep < p.groups <= 64), one wave: lane g's group has
// `score`, the sum of its two largest c, and `second`, the second of them (the
// only one where groups hold one expert; then score is it too); bit g of
// `kept` says whether group g is among the keep best (score descending, group
// ascending).  cs: this wave's LDS, [E].
template <typename V>
struct Groups {
    V score, second;
    uint64_t kept;
};

// group of expert e, by a reciprocal: exact for e < 1024
__device__ __forceinline__ int group_of(int e, float inv_size) { return (int)(((float)e + 0.5f) * inv_size); }

__device__ __forceinline__ float lane_value(float v, int l)
{
    return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v), l));
}
__device__ __forceinline__ double lane_value(double v, int l) { return readlane_f64(v, l); }

template <int MAXPL, typename V>
__device__ __forceinline__ Groups<V> rank_groups(const ScoredPass &p, int lane, const V c[MAXPL], V *cs)
{
    const int G = p.groups, size = p.E / G;
    wave_sync();
#pragma unroll
    for (int i = 0; i < MAXPL; ++i)
        if (lane + 64 * i < p.E) cs[lane + 64 * i] = c[i];
    wave_sync();
    Groups<V> g;
    V a = -INFINITY, b = -INFINITY;              // the two largest
    if (G <= 8) {                                // 8 lanes a group, then their two largest together
        if ((lane >> 3) < G)
            for (int j = lane & 7; j < size; j += 8) {
                const V v = cs[(lane >> 3) * size + j];
                b = fmax(b, fmin(a, v));
                a = fmax(a, v);
            }
#pragma unroll
        for (int off = 1; off < 8; off <<= 1) {
            const V oa = __shfl_xor(a, off, 64), ob = __shfl_xor(b, off, 64);
            b = fmax(fmin(a, oa), fmax(b, ob));
            a = fmax(a, oa);
        }
        a = __shfl(a, (lane & 7) * 8, 64);       // group g's to lane g
        b = __shfl(b, (lane & 7) * 8, 64);
    } else if (lane < G) {
        for (int j = 0; j < size; ++j) {
            const V v = cs[lane * size + j];
            b = fmax(b, fmin(a, v));
            a = fmax(a, v);
        }
    }
    // inf - inf would be a NaN, which no score outranks
    g.score = size == 1 ? a : b == -INFINITY ? b : a + b;
    g.second = size > 1 ? b : a;
    int r = 0;
    for (int o = 0; o < G; ++o) {
        const V s = lane_value(g.score, o);
        r += s > g.score || (s == g.score && o < lane);
    }
    g.kept = __ballot(lane < G && r < p.keep);
    return g;
}

// k rounds of a wave-wide arg-max over (c descending, expert ascending): lane
// j < k keeps slot j's expert, value and score
template <int MAXPL>
__device__ __forceinline__ void select64(const ScoredPass &p, int lane, const double c[MAXPL], const double pr[MAXPL], int &my_e,
                                         double &my_c, double &my_p, uint32_t &taken)
{
    taken = 0;
    my_e = 0;
    my_c = my_p = 0.0;
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
        const double sel = readlane_f64(bp, be & 63);   // expert be is lane be % 64's
        if (mine == be) taken |= 1u << (be >> 6);
        if (lane == j) { my_e = be; my_c = bv; my_p = sel; }
    }
}

// Slot `slot` of token t (slot < k in k lanes of the wave) gets expert e, whose
// score is w (0 in the other lanes and for c = -inf).  Returns the slot's weight.
__device__ __forceinline__ float write_token(const ScoredPass &p, int t, int slot, int e, double w)
{
    if (p.renorm) {
        const double sum = wave_sum_f64(w);
        w = sum > 0.0 ? w / sum : 0.0;
    }
    const float weight = (float)(w * (double)p.scale);
    if (slot < p.k) {
        p.topk_idx[(int64_t)t * p.k + slot] = e;
        p.topk_w[(int64_t)t * p.k + slot] = weight;
    }
    return weight;
}

}  // namespace moe
