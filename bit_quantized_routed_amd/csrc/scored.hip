// Scored router on gfx950: sigmoid or softmax scores, a selection-only bias,
// group-limited top-k and the weights of the chosen experts.
//
//   l = x W_r^T;  p = sigmoid(l) or softmax(l);  c = p + bias
//   groups: score = sum of the two largest c; the `keep` best stay
//   the k largest c are chosen; w = p (/ sum p) * scale
//
// The chosen experts are those of fp64 scores.  Two ways to them:
//
// - fp64 logits and scores throughout, as in the plain router (route.hip).
// - The split router, for many bf16 tokens with sigmoid scores.  Each weight is
//   three bf16 terms that add up to it exactly, so that the logits are fp32 sums
//   of exact products on the bf16 matrix instructions, 16 times the rate of the
//   fp64 ones for 3 times the products.  A bound on the sums' rounding goes with
//   every token; where it leaves the order of two experts or groups open, the
//   experts in question are summed again in fp64 by the wave that selects.
//   Softmax stays in fp64: there every score hangs on the sum over all experts.
#include "common.h"
#include "devcache.h"
#include "route.h"
#include "route_dev.h"
#include "scored.h"

#include <algorithm>

namespace moe {

namespace {

typedef double f64x4 __attribute__((ext_vector_type(4)));

// ---------------------------------------------------------------- fp64 logits
// More than 64 tokens on the fp64 matrix instructions: 64 tokens x 64 experts
// and one part of H per work-group, partial sums [part][T][E].  Chunks of 32 of
// H pass through LDS as fp64, the next one's values on their way into
// registers meanwhile; rows of 33 doubles put the 16 lanes of a read on
// different bank pairs.  Each wave owns 16 experts and four 16-token products.
constexpr int PARTS64 = 8;

int parts64(int T, int H, int E)
{
    const int64_t tiles = ((int64_t)T + 63) / 64 * ((E + 63) / 64);
    return (int)std::max<int64_t>(1, std::min<int64_t>({(512 + tiles - 1) / tiles, (H + 127) / 128, PARTS64}));
}

template <bool XBF16>
__global__ __launch_bounds__(256) void scored_logits64(ScoredPass p, int parts)
{
    constexpr int HC = 32, LD = HC + 1;
    __shared__ double xs[64][LD], ws[64][LD];
    const int t0 = blockIdx.x * 64, e0 = blockIdx.y * 64, part = blockIdx.z;
    const int chunks = (p.H + HC - 1) / HC;
    const int begin = chunks * part / parts * HC, end = min(p.H, chunks * (part + 1) / parts * HC);
    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, fr = lane & 15, fk = lane >> 4;
    f64x4 acc[4];
#pragma unroll
    for (int m = 0; m < 4; ++m) acc[m] = f64x4{0.0, 0.0, 0.0, 0.0};
    // 8 values of x and of w per thread and chunk; rows past T or E, and columns
    // past H, load something in bounds and count as zero
    const int sr = tid >> 2, sk = (tid & 3) * 8;
    const bool xok = t0 + sr < p.T, wok = e0 + sr < p.E;
    const int64_t xrow = (int64_t)(xok ? t0 + sr : 0) * p.ldx, wrow = (int64_t)(wok ? e0 + sr : 0) * p.H;
    u32x4 xraw[XBF16 ? 1 : 2];
    f32x4 wraw[2];
    auto load = [&](int h0) {
        const int h = min(h0 + sk, p.H - 8);
        if (XBF16) xraw[0] = *(const u32x4 *)((const uint16_t *)p.x + xrow + h);
        else {
#pragma unroll
            for (int i = 0; i < 2; ++i) xraw[i] = *(const u32x4 *)((const float *)p.x + xrow + h + 4 * i);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) wraw[i] = *(const f32x4 *)(p.w + wrow + h + 4 * i);
    };
    load(begin);
    for (int h0 = begin; h0 < end; h0 += HC) {
        const bool in = h0 + sk < p.H;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            double v;
            if (XBF16) v = (double)bf16_bits_to_f32((xraw[0][i >> 1] >> (16 * (i & 1))) & 0xffffu);
            else v = (double)__uint_as_float(xraw[i >> 2][i & 3]);
            xs[sr][sk + i] = xok && in ? v : 0.0;
            ws[sr][sk + i] = wok && in ? (double)wraw[i >> 2][i & 3] : 0.0;
        }
        __syncthreads();
        load(h0 + HC);
#pragma unroll
        for (int kk = 0; kk < HC / 4; ++kk) {
            const double b = ws[wave * 16 + fr][4 * kk + fk];
#pragma unroll
            for (int m = 0; m < 4; ++m)
                acc[m] = __builtin_amdgcn_mfma_f64_16x16x4f64(xs[m * 16 + fr][4 * kk + fk], b, acc[m], 0, 0, 0);
        }
    }
    // D: lane (fr, fk) holds tokens fk + 4 i of expert fr
    const int e = e0 + wave * 16 + fr;
    if (e >= p.E) return;
#pragma unroll
    for (int m = 0; m < 4; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = t0 + m * 16 + fk + 4 * i;
            if (t < p.T) ((double *)p.logits)[((int64_t)part * p.T + t) * p.E + e] = acc[m][i];
        }
}

// ---------------------------------------------------------------- split logits
// The terms of w: w1 = bf16(w), w2 = bf16(w - w1), w3 = bf16(w - w1 - w2), each
// difference exact, w1 + w2 + w3 = w (but for bits below the smallest bf16).
// They are laid out as the logits kernel's LDS images: [expert block][step of
// 32 of H][term][64 NG rows][4 chunks of 8 at chunk ^ key(row)], zeros past E
// and H.
constexpr int BM = 128;                          // tokens of a work-group
constexpr int STEP = 32, CHUNK = 128;            // of H: a matrix instruction's depth, a short sum's

int expert_waves(int E) { return E <= 64 ? 1 : E <= 128 ? 2 : 4; }    // NG: columns of 64 experts a work-group has
__host__ __device__ inline int split_steps(int H) { return (H + CHUNK - 1) / CHUNK * (CHUNK / STEP); }
__device__ __forceinline__ int key(int r) { return (r >> 2) & 3; }

__device__ __forceinline__ uint32_t bf16_of(float f) { return __builtin_bit_cast(uint16_t, (__bf16)f); }

__global__ __launch_bounds__(256) void scored_split_w(ScoredPass p, int rows)
{
    __shared__ float part[4];
    const int e = blockIdx.x, blk = e / rows, r = e % rows, tid = threadIdx.x;
    const int steps = split_steps(p.H);
    float ss = 0.0f;
    for (int c = tid; c < steps * 4; c += 256) { // chunks of 8
        const int h = 8 * c;
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = 0.0f;
        if (e < p.E && h < p.H) {
            const f32x4 a = *(const f32x4 *)(p.w + (int64_t)e * p.H + h), b = *(const f32x4 *)(p.w + (int64_t)e * p.H + h + 4);
#pragma unroll
            for (int i = 0; i < 4; ++i) { v[i] = a[i]; v[4 + i] = b[i]; }
        }
        u32x4 *o = (u32x4 *)p.wsplit + (((int64_t)blk * steps + c / 4) * 3 * rows + r) * 4 + ((c & 3) ^ key(r));
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(v[i], v[i], ss);
#pragma unroll
        for (int term = 0; term < 3; ++term) {
            u32x4 u;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t lo = bf16_of(v[2 * i]), hi = bf16_of(v[2 * i + 1]);
                u[i] = lo | (hi << 16);
                v[2 * i] -= bf16_bits_to_f32(lo);
                v[2 * i + 1] -= bf16_bits_to_f32(hi);
            }
            o[(int64_t)term * rows * 4] = u;
        }
    }
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) ss += __shfl_xor(ss, off, 64);
    if ((tid & 63) == 0) part[tid >> 6] = ss;
    __syncthreads();
    if (tid == 0 && e < p.E) p.wnorm[e] = part[0] + part[1] + part[2] + part[3];
}

// Logits of 128 tokens x 64 NG experts over one part of H, fp32 [part][T][E],
// and the tokens' sums of squares [part][T].  2 NG waves of 64 tokens x 64
// experts.  x and the three terms of a step of 32 go to LDS without passing
// registers, one step ahead; the smallest term's products are added first, sums
// run over 128 of H and are then added to the totals, so that a logit has been
// rounded 12 times in its short sum and H / 128 times after it.  Parts of H are
// dealt so that an XCD sees few of them: its share of the terms stays in its L2.
template <int NG>
__global__ __launch_bounds__(128 * NG) void scored_split_logits(ScoredPass p, int parts)
{
    constexpr int ROWS = 64 * NG, NW = 2 * NG, XB = BM * 64, TERM = ROWS * 64, SLOT = XB + 3 * TERM;
    constexpr int LX = BM / 16 / NW, LW = 3 * ROWS / 16 / NW;          // loads of a wave in a step
    extern __shared__ __align__(16) int8_t ring[];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int fr = lane & 15, fg = lane >> 4;
    const int part = blockIdx.x % parts, t0 = (int)(blockIdx.x / parts) * BM, blk = blockIdx.y;
    const int chunks = (p.H + CHUNK - 1) / CHUNK;
    const int begin = chunks * part / parts * (CHUNK / STEP), steps = chunks * (part + 1) / parts * (CHUNK / STEP) - begin;

    const int lr = lane >> 2, lc = lane & 3;
    const uint16_t *xp[LX];
    int xc[LX];
#pragma unroll
    for (int i = 0; i < LX; ++i) {
        const int r = (wave * LX + i) * 16 + lr;
        xp[i] = (const uint16_t *)p.x + (int64_t)min(t0 + r, p.T - 1) * p.ldx;
        xc[i] = 8 * (lc ^ key(r));
    }
    const int8_t *wp = (const int8_t *)p.wsplit + ((int64_t)blk * split_steps(p.H) + begin) * 3 * TERM + wave * LW * 1024 + lane * 16;
    auto fetch = [&](int s) {
        int8_t *const buf = ring + (s & 1) * SLOT;
#pragma unroll
        for (int i = 0; i < LX; ++i) {
            // past H: the row's last chunk again, the terms are zero there
            const int h = min((begin + s) * STEP + xc[i], p.H - 8);
            __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)(xp[i] + h),
                                             (__attribute__((address_space(3))) void *)(buf + (wave * LX + i) * 1024), 16, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < LW; ++i)
            __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)(wp + (int64_t)s * 3 * TERM + i * 1024),
                                             (__attribute__((address_space(3))) void *)(buf + XB + (wave * LW + i) * 1024), 16, 0, 0);
    };
    const int wa = wave % NG, wt = wave / NG;
    const int x0 = 64 * wt + fr, w0 = 64 * wa + fr;
    const int xo = x0 * 64 + 16 * (fg ^ key(x0)), wo = XB + w0 * 64 + 16 * (fg ^ key(w0));  // + 1024 a fragment
    f32x4 total[4][4], acc[4][4];
    float ss[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        ss[i] = 0.0f;
#pragma unroll
        for (int j = 0; j < 4; ++j) total[i][j] = acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }
    fetch(0);
    for (int s = 0; s < steps; ++s) {
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_waitcnt(0x0070);      // vmcnt(0) lgkmcnt(0)
        __builtin_amdgcn_s_barrier();            // step s has landed for everybody, and step s - 1 is read
        asm volatile("" ::: "memory");
        if (s + 1 < steps) fetch(s + 1);
        const int8_t *buf = ring + (s & 1) * SLOT;
        bf16x8 b[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) b[j] = *(const bf16x8 *)(buf + xo + 1024 * j);
#pragma unroll
        for (int term = 2; term >= 0; --term) {
            bf16x8 a[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) a[i] = *(const bf16x8 *)(buf + wo + term * TERM + 1024 * i);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = mfma16x16x32(a[i], b[j], acc[i][j]);
        }
        // sums of squares of x, the four fragments shared out over the NG waves
        // that hold the same tokens
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (j % NG == wa && blk == 0 && (begin + s) * STEP + 8 * fg < p.H) {
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    const float v = (float)b[j][q];
                    ss[j] = fmaf(v, v, ss[j]);
                }
            }
        if ((s & 3) == 3) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    total[i][j] += acc[i][j];
                    acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
                }
        }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        float v = ss[j];
        v += __shfl_xor(v, 16, 64);
        v += __shfl_xor(v, 32, 64);
        const int t = t0 + x0 + 16 * j;
        if (t >= p.T) continue;
        if (j % NG == wa && blk == 0 && fg == 0) p.xnorm[(int64_t)part * p.T + t] = v;
        // D: lane (fr, fg) holds experts 4 fg .. 4 fg + 3 of token fr
        float *o = (float *)p.logits + ((int64_t)part * p.T + t) * p.E;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int e = ROWS * blk + 64 * wa + 16 * i + 4 * fg;
            if (p.E % 4 == 0) {
                if (e < p.E) *(f32x4 *)(o + e) = total[i][j];
            } else {
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    if (e + q < p.E) o[e + q] = total[i][j][q];
            }
        }
    }
}

// ---------------------------------------------------------------- selection
__device__ __forceinline__ double wave_sum_f64(double v)
{
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, 64);
    return v;
}

__device__ __forceinline__ double sigmoid64(double l) { return l == -INFINITY ? 0.0 : 1.0 / (1.0 + exp(-l)); }

// p + bias, or -inf where the logit or the sum is NaN
__device__ __forceinline__ double biased(const ScoredPass &p, int e, double l, double pr)
{
    const double v = l != l ? -INFINITY : p.bias ? pr + (double)p.bias[e] : pr;
    return v != v ? -INFINITY : v;
}

// Scores of one token, one wave: lane l holds experts l, l + 64, ...  On
// return pr holds the scores p (0 for NaN logits and past E) and c the
// selection values p + bias (-inf for NaN and past E).
template <int MAXPL>
__device__ __forceinline__ void token_scores(const ScoredPass &p, const double l[MAXPL], int lane, double pr[MAXPL],
                                             double c[MAXPL])
{
    double top = -INFINITY;
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
        c[i] = e < p.E ? biased(p, e, l[i], pr[i]) : -INFINITY;
    }
}

// LDS written before is read after, within one wave: its LDS operations run in
// order, so only the compiler has to keep it.
__device__ __forceinline__ void wave_sync()
{
    asm volatile("" ::: "memory");
    __builtin_amdgcn_wave_barrier();
    asm volatile("" ::: "memory");
}

// This wave's LDS: its token's selection values [E] and group scores [groups],
// of type V.
template <typename V>
struct Groups {
    V *c, *score, *second;                       // second: the second largest c of a group, -inf for groups of one
};

// Group scores of one token from c, one wave (p.groups > 1).
template <int MAXPL, typename V>
__device__ __forceinline__ void group_scores(const ScoredPass &p, int lane, const V c[MAXPL], const Groups<V> &g)
{
    const int G = p.groups, size = p.E / G;
#pragma unroll
    for (int i = 0; i < MAXPL; ++i)
        if (lane + 64 * i < p.E) g.c[lane + 64 * i] = c[i];
    wave_sync();
    if (G <= 8) {                                // 8 lanes a group, then their two largest together
        const int gr = lane >> 3;
        V a = -INFINITY, b = -INFINITY;
        if (gr < G)
            for (int j = lane & 7; j < size; j += 8) {
                const V v = g.c[gr * size + j];
                b = fmax(b, fmin(a, v));
                a = fmax(a, v);
            }
#pragma unroll
        for (int off = 1; off < 8; off <<= 1) {
            const V oa = __shfl_xor(a, off, 64), ob = __shfl_xor(b, off, 64);
            b = fmax(fmin(a, oa), fmax(b, ob));
            a = fmax(a, oa);
        }
        if (gr < G && (lane & 7) == 0) {
            g.score[gr] = size > 1 ? a + b : a;
            g.second[gr] = b;
        }
    } else {
        for (int gr = lane; gr < G; gr += 64) {
            V a = -INFINITY, b = -INFINITY;
            for (int j = 0; j < size; ++j) {
                const V v = g.c[gr * size + j];
                b = fmax(b, fmin(a, v));
                a = fmax(a, v);
            }
            g.score[gr] = size > 1 ? a + b : a;
            g.second[gr] = b;
        }
    }
    wave_sync();
}

// whether group g is among the `keep` best
template <typename V>
__device__ __forceinline__ bool group_kept(const ScoredPass &p, const V *score, int g)
{
    const V mine = score[g];
    int r = 0;
    for (int o = 0; o < p.groups; ++o) r += score[o] > mine || (score[o] == mine && o < g);
    return r < p.keep;
}

// k rounds of a wave-wide arg-max over (c descending, expert ascending): lane
// j < k keeps slot j's expert and value
template <int MAXPL>
__device__ __forceinline__ void select64(const ScoredPass &p, int lane, const double c[MAXPL], int &my_e, double &my_c,
                                         uint32_t &taken)
{
    taken = 0;
    my_e = 0;
    my_c = 0.0;
    for (int j = 0; j < p.k; ++j) {
        double bv = -INFINITY;
        int be = 0x7fffffff;
#pragma unroll
        for (int i = 0; i < MAXPL; ++i) {
            const int e = lane + 64 * i;
            // e grows with i, so a strict '>' keeps the lowest expert among equals
            if (e < p.E && !((taken >> i) & 1u) && (be == 0x7fffffff || c[i] > bv)) { bv = c[i]; be = e; }
        }
        const int mine = be;
        wave_argmax(bv, be);
        if (mine == be) taken |= 1u << (be >> 6);
        if (lane == j) { my_e = be; my_c = bv; }
    }
}

// value i = be / 64 of lane be % 64
template <int MAXPL>
__device__ __forceinline__ double value_of(const double v[MAXPL], int be)
{
    double r = 0.0;
#pragma unroll
    for (int i = 0; i < MAXPL; ++i) {
        const double s = __shfl(v[i], be & 63, 64);
        if (i == be >> 6) r = s;
    }
    return r;
}

// the weights of the chosen experts, w the score of lane j's (0 past k and for c = -inf)
__device__ __forceinline__ void write_token(const ScoredPass &p, int t, int lane, int my_e, double w)
{
    if (p.renorm) {
        const double sum = wave_sum_f64(w);
        w = sum > 0.0 ? w / sum : 0.0;
    }
    if (lane < p.k) {
        p.topk_idx[(int64_t)t * p.k + lane] = my_e;
        p.topk_w[(int64_t)t * p.k + lane] = (float)(w * (double)p.scale);
    }
}

constexpr int WAVES = 4;                         // tokens of a work-group, a wave each

// fp64 selection; a single token is grouped here too (the sorted selection:
// offsets from ballots of the taken flags)
template <int MAXPL>
__global__ __launch_bounds__(64 * WAVES) void scored_topk(ScoredPass p, int parts)
{
    extern __shared__ double lds[];              // keep < groups: [WAVES][E + 2 groups]
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int t = blockIdx.x * (blockDim.x >> 6) + wave;
    if (t >= p.T) return;
    double l[MAXPL], pr[MAXPL], c[MAXPL];
    const double *in = (const double *)p.logits + (int64_t)t * p.E;
#pragma unroll
    for (int i = 0; i < MAXPL; ++i) l[i] = lane + 64 * i < p.E ? in[lane + 64 * i] : -INFINITY;
    for (int q = 1; q < parts; ++q) {
        in += (int64_t)p.T * p.E;
#pragma unroll
        for (int i = 0; i < MAXPL; ++i)
            if (lane + 64 * i < p.E) l[i] += in[lane + 64 * i];
    }
    token_scores<MAXPL>(p, l, lane, pr, c);
    if (p.keep < p.groups) {
        double *mine = lds + (size_t)wave * (p.E + 2 * p.groups);
        const Groups<double> g{mine, mine + p.E, mine + p.E + p.groups};
        group_scores<MAXPL, double>(p, lane, c, g);
        const int size = p.E / p.groups;
#pragma unroll
        for (int i = 0; i < MAXPL; ++i)
            if (lane + 64 * i < p.E && !group_kept(p, g.score, (lane + 64 * i) / size)) c[i] = -INFINITY;
    }
    int my_e;
    double my_c;
    uint32_t taken;
    select64<MAXPL>(p, lane, c, my_e, my_c, taken);
    const double mine = value_of<MAXPL>(pr, my_e);
    write_token(p, t, lane, my_e, lane < p.k && my_c != -INFINITY ? mine : 0.0);
    if (p.T > 1) return;
    uint64_t mk[MAXPL];
    int below = 0, base = 0;
#pragma unroll
    for (int i = 0; i < MAXPL; ++i) {
        mk[i] = __ballot((taken >> i) & 1u);
        below += i < my_e >> 6 ? __popcll(mk[i]) : i == my_e >> 6 ? __popcll(mk[i] & ((1ull << (my_e & 63)) - 1ull)) : 0;
        if (lane + 64 * i < p.E) p.offsets[lane + 64 * i] = base + __popcll(mk[i] & ((1ull << lane) - 1ull));
        base += __popcll(mk[i]);
    }
    if (lane == 0) p.offsets[p.E] = base;
    if (lane < p.k) {
        p.perm[below] = lane;
        p.inv[lane] = below;
    }
}

// One expert's logit of one token in fp64 by a whole wave, always in the same
// order: equal rows of w give equal logits.
__device__ __forceinline__ double exact_logit(const ScoredPass &p, int t, int e, int lane)
{
    const uint16_t *x = (const uint16_t *)p.x + (int64_t)t * p.ldx;
    const float *w = p.w + (int64_t)e * p.H;
    double s = 0.0;
    for (int h = 8 * lane; h < p.H; h += 512) {
        const u32x4 u = *(const u32x4 *)(x + h);
        const f32x4 a = *(const f32x4 *)(w + h), b = *(const f32x4 *)(w + h + 4);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            s = fma((double)bf16_bits_to_f32((u[i >> 1] >> (16 * (i & 1))) & 0xffffu), (double)(i < 4 ? a[i & 3] : b[i & 3]), s);
    }
    return wave_sum_f64(s);
}

// replaces the logits of the flagged experts (bit i: expert lane + 64 i) by
// their fp64 values, and with them pr and c
template <int MAXPL>
__device__ __forceinline__ void refine(const ScoredPass &p, int t, int lane, uint32_t flags, uint32_t &done, double pr[MAXPL],
                                       double c[MAXPL])
{
#pragma unroll
    for (int i = 0; i < MAXPL; ++i) {
        uint64_t todo = __ballot((flags & ~done) >> i & 1u);
        while (todo) {
            const int o = __ffsll((unsigned long long)todo) - 1;
            todo &= todo - 1;
            const double l = exact_logit(p, t, o + 64 * i, lane);
            if (lane == o) {
                pr[i] = l != l ? 0.0 : sigmoid64(l);
                c[i] = biased(p, o + 64 * i, l, pr[i]);
                done |= 1u << i;
            }
        }
    }
}

// Selection from the split router's logits.  A logit is off by at most d =
// rounding |x| max |w_e|: 12 roundings in a short sum, of 2^-23 each (a matrix
// instruction's own sum included), and up to H / 128 + 8 of 2^-24 after it, all of
// values that |x| |w| bounds piece by piece.  (In practice the sums' random signs
// keep it some hundred times smaller.)  A selection value is off by at most eps =
// d / 4, the sigmoid's steepest slope, and fp32's roundings.  Groups whose scores
// lie within 4 eps of the border between kept and not, and experts within 2 eps
// of each other down to the first that is not chosen, are decided on fp64 logits.
template <int MAXPL>
__global__ __launch_bounds__(64 * WAVES) void scored_split_topk(ScoredPass p, int parts, float rounding)
{
    extern __shared__ double lds[];              // keep < groups: [WAVES][E + 2 groups]
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int t = blockIdx.x * WAVES + wave;
    if (t >= p.T) return;
    float l[MAXPL], c[MAXPL];
    float wmax = 0.0f, bmax = 0.0f, xn = lane < parts ? p.xnorm[(int64_t)lane * p.T + t] : 0.0f;
    const float *in = (const float *)p.logits + (int64_t)t * p.E;
#pragma unroll
    for (int i = 0; i < MAXPL; ++i) {
        const int e = lane + 64 * i;
        l[i] = -INFINITY;
        c[i] = 0.0f;                             // the bias for now
        if (e < p.E) {
            l[i] = in[e];
            wmax = fmaxf(wmax, p.wnorm[e]);
            if (p.bias) c[i] = p.bias[e];
            if (fabsf(c[i]) < INFINITY) bmax = fmaxf(bmax, fabsf(c[i]));
        }
    }
    for (int q = 1; q < parts; ++q) {
        in += (int64_t)p.T * p.E;
#pragma unroll
        for (int i = 0; i < MAXPL; ++i)
            if (lane + 64 * i < p.E) l[i] += in[lane + 64 * i];
    }
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) {
        wmax = fmaxf(wmax, __shfl_xor(wmax, off, 64));
        bmax = fmaxf(bmax, __shfl_xor(bmax, off, 64));
        xn += __shfl_xor(xn, off, 64);
    }
    const float d = rounding * sqrtf(xn) * sqrtf(wmax);
    const bool sure = d < 1e-2f;                 // no overflow near, no NaN; else everything in fp64
    const float eps = 0.25f * d + 0x1p-21f * (1.0f + bmax);
#pragma unroll
    for (int i = 0; i < MAXPL; ++i) {
        const float v = l[i] == -INFINITY ? c[i] : 1.0f / (1.0f + expf(-l[i])) + c[i];
        c[i] = lane + 64 * i < p.E && v == v ? v : -INFINITY;
    }
    const int size = p.E / p.groups;
    const bool limit = p.keep < p.groups;
    double *mine64 = lds + (size_t)wave * (p.E + 2 * p.groups);
    float *mine32 = (float *)mine64;
    const Groups<float> g{mine32, mine32 + p.E, mine32 + p.E + p.groups};
    bool open = !sure;
    float in_least = INFINITY, out_most = -INFINITY;      // scores on both sides of the border
    float cs[MAXPL];
#pragma unroll
    for (int i = 0; i < MAXPL; ++i) cs[i] = c[i];
    if (limit) {
        group_scores<MAXPL, float>(p, lane, c, g);
        for (int gr = lane; gr < p.groups; gr += 64) {
            const float s = g.score[gr];
            if (group_kept(p, g.score, gr)) in_least = fminf(in_least, s);
            else out_most = fmaxf(out_most, s);
        }
#pragma unroll
        for (int off = 32; off > 0; off >>= 1) {
            in_least = fminf(in_least, __shfl_xor(in_least, off, 64));
            out_most = fmaxf(out_most, __shfl_xor(out_most, off, 64));
        }
        open = open || !(in_least - out_most > 4.0f * eps);
#pragma unroll
        for (int i = 0; i < MAXPL; ++i)
            if (lane + 64 * i < p.E && !group_kept(p, g.score, (lane + 64 * i) / size)) cs[i] = -INFINITY;
    }
    // the k + 1 largest; lane j keeps slot j
    int my_e = 0;
    float my_l = -INFINITY, my_c = -INFINITY;
    if (!open) {
        uint32_t taken = 0;
        float last = INFINITY;
        for (int j = 0; j <= p.k && j < p.E; ++j) {
            float bv = -INFINITY, bl = -INFINITY;
            int be = 0x7fffffff;
#pragma unroll
            for (int i = 0; i < MAXPL; ++i) {
                const int e = lane + 64 * i;
                if (e < p.E && !((taken >> i) & 1u) && (be == 0x7fffffff || cs[i] > bv)) { bv = cs[i]; be = e; bl = l[i]; }
            }
            float m = bv;
#pragma unroll
            for (int off = 32; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor(m, off, 64));
            // values this close are told apart in fp64; equal ones too
            if (!(last - m > 2.0f * eps)) { open = true; break; }
            if (m == -INFINITY) {                // nothing left: the k-th lies above, or it does not and fp64 says which
                open = j < p.k;
                break;
            }
            last = m;
            const uint64_t at = __ballot(bv == m);
            if (__popcll(at) != 1) { open = true; break; }
            const int o = __ffsll((unsigned long long)at) - 1;
            const int e = __builtin_amdgcn_readlane(be, o);
            const float el = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(bl), o));
            if (lane == o) taken |= 1u << (e >> 6);
            if (lane == j) { my_e = e; my_l = el; my_c = m; }
        }
    }
    if (!open) {
        write_token(p, t, lane, my_e, lane < p.k && my_c != -INFINITY ? sigmoid64((double)my_l) : 0.0);
        return;
    }
    // ---- in doubt: fp64 for the experts that matter
    double pr[MAXPL], c64[MAXPL];
    uint32_t done = 0, flags = 0;
#pragma unroll
    for (int i = 0; i < MAXPL; ++i) {
        pr[i] = l[i] != l[i] ? 0.0 : sigmoid64((double)l[i]);
        c64[i] = (double)c[i];
        if (lane + 64 * i >= p.E) continue;
        const int gr = (lane + 64 * i) / size;
        const bool near = limit && g.score[gr] <= out_most + 4.0f * eps && g.score[gr] >= in_least - 4.0f * eps &&
                          c[i] >= g.second[gr] - 2.0f * eps;
        if (!sure || near) flags |= 1u << i;
    }
    refine<MAXPL>(p, t, lane, flags, done, pr, c64);
    if (limit) {
        wave_sync();                             // the fp32 scores are read
        const Groups<double> g64{mine64, mine64 + p.E, mine64 + p.E + p.groups};
        group_scores<MAXPL, double>(p, lane, c64, g64);
#pragma unroll
        for (int i = 0; i < MAXPL; ++i)
            if (lane + 64 * i < p.E && !group_kept(p, g64.score, (lane + 64 * i) / size)) {
                c64[i] = -INFINITY;
                done |= 1u << i;
            }
    }
    double slot_c;
    uint32_t taken;
    select64<MAXPL>(p, lane, c64, my_e, slot_c, taken);
    const double least = __shfl(slot_c, p.k - 1, 64) - 2.0 * (double)eps;
    flags = 0;
#pragma unroll
    for (int i = 0; i < MAXPL; ++i)
        if (lane + 64 * i < p.E && c64[i] >= least) flags |= 1u << i;
    refine<MAXPL>(p, t, lane, flags, done, pr, c64);
    select64<MAXPL>(p, lane, c64, my_e, slot_c, taken);
    const double w = value_of<MAXPL>(pr, my_e);
    write_token(p, t, lane, my_e, lane < p.k && slot_c != -INFINITY ? w : 0.0);
}

}  // namespace

size_t scored_logit_bytes(int T, int H, int E, bool split)
{
    if (split) return (size_t)scored_split_parts(T, H, E) * T * E * sizeof(float);
    return (size_t)(T <= SCORED_SMALL_T ? route_decode_chunks(T, H) : parts64(T, H, E)) * T * E * sizeof(double);
}

size_t scored_split_bytes(int H, int E)
{
    const int rows = 64 * expert_waves(E);
    return (size_t)((E + rows - 1) / rows) * split_steps(H) * 3 * rows * 64;
}

int scored_split_parts(int T, int H, int E)
{
    // enough work-groups for the 256 CUs, parts of at least four chunks
    const int rows = 64 * expert_waves(E);
    const int64_t tiles = ((int64_t)T + BM - 1) / BM * ((E + rows - 1) / rows);
    return (int)std::max<int64_t>(1, std::min<int64_t>({256 / tiles, (H + CHUNK - 1) / CHUNK / 4, 8}));
}

hipError_t launch_scored_logits(const ScoredPass &p, hipStream_t s)
{
    if (p.T <= SCORED_SMALL_T) {
        launch_route_partial(p.x, p.x_bf16, p.ldx, p.w, p.T, p.H, p.E, (double *)p.logits, s);
        return hipGetLastError();
    }
    const int parts = parts64(p.T, p.H, p.E);
    const dim3 grid((unsigned)(((int64_t)p.T + 63) / 64), (unsigned)((p.E + 63) / 64), (unsigned)parts);
    if (p.x_bf16) scored_logits64<true><<<grid, 256, 0, s>>>(p, parts);
    else scored_logits64<false><<<grid, 256, 0, s>>>(p, parts);
    return hipGetLastError();
}

hipError_t launch_scored_split(const ScoredPass &p, hipStream_t s)
{
    const int rows = 64 * expert_waves(p.E);
    scored_split_w<<<dim3((unsigned)((p.E + rows - 1) / rows * rows)), 256, 0, s>>>(p, rows);
    return hipGetLastError();
}

hipError_t launch_scored_split_logits(const ScoredPass &p, hipStream_t s)
{
    const int ng = expert_waves(p.E), rows = 64 * ng, parts = scored_split_parts(p.T, p.H, p.E);
    const dim3 grid((unsigned)(((int64_t)p.T + BM - 1) / BM * parts), (unsigned)((p.E + rows - 1) / rows));
    const size_t lds = 2 * (BM * 64 + 3 * rows * 64);
#define MOE_SPLIT(n)                                                                              \
    do {                                                                                          \
        static DevSlots slots{};                                                                  \
        const hipError_t e = lds_limit((const void *)scored_split_logits<n>, slots, lds);         \
        if (e != hipSuccess) return e;                                                            \
        scored_split_logits<n><<<grid, 128 * n, lds, s>>>(p, parts);                              \
    } while (0)
    if (ng == 1) MOE_SPLIT(1);
    else if (ng == 2) MOE_SPLIT(2);
    else MOE_SPLIT(4);
#undef MOE_SPLIT
    return hipGetLastError();
}

hipError_t launch_scored_topk(const ScoredPass &p, hipStream_t s)
{
    const bool split = scored_split(p.T, p.softmax, p.x_bf16);
    const int parts = split ? scored_split_parts(p.T, p.H, p.E)
                            : p.T <= SCORED_SMALL_T ? route_decode_chunks(p.T, p.H) : parts64(p.T, p.H, p.E);
    const int waves = p.T == 1 ? 1 : WAVES;
    const size_t lds = p.keep < p.groups ? (size_t)waves * (p.E + 2 * p.groups) * sizeof(double) : 0;
    const unsigned grid = (unsigned)(((int64_t)p.T + waves - 1) / waves);
    // the short sums' 12 roundings and those after them, in units of 2^-23 of the bound
    const float rounding = 0x1p-23f * (12.0f + 0.5f * ((float)p.H / CHUNK + 8.0f));
    // unrolled for the experts each lane holds (E <= 64 * MAXPL)
#define MOE_TOPK(pl)                                                                              \
    do {                                                                                          \
        static DevSlots slots[2]{};                                                               \
        const void *k = split ? (const void *)scored_split_topk<pl> : (const void *)scored_topk<pl>; \
        const hipError_t e = lds > 65536 ? lds_limit(k, slots[split], lds) : hipSuccess;          \
        if (e != hipSuccess) return e;                                                            \
        if (split) scored_split_topk<pl><<<grid, 64 * WAVES, lds, s>>>(p, parts, rounding);       \
        else scored_topk<pl><<<grid, 64 * waves, lds, s>>>(p, parts);                             \
    } while (0)
    if (p.E <= 64) MOE_TOPK(1);
    else if (p.E <= 128) MOE_TOPK(2);
    else if (p.E <= 256) MOE_TOPK(4);
    else if (p.E <= 512) MOE_TOPK(8);
    else MOE_TOPK(16);
#undef MOE_TOPK
    return hipGetLastError();
}

}  // namespace moe
