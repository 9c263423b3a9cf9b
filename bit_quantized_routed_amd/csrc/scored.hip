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
//   every token; where it leaves the order of two experts or groups open, a
//   work-group of a later launch sums the experts in question again in fp64.
//   Softmax stays in fp64: there every score hangs on the sum over all experts.
#include "common.h"
#include "devcache.h"
#include "scored.h"
#include "scored_dev.h"

#include <algorithm>

namespace moe {

namespace {

typedef double f64x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// ---------------------------------------------------------------- fp64 logits
// Up to 128 tokens: a wave sums EW experts x TB tokens over one part of H, 8
// values a lane and step, every load of two steps on its way before the first
// product; a fixed butterfly adds the lanes.  Partial sums [part][T][E].
constexpr int PARTS_SMALL = 4;

int parts_small(int H) { return std::min(PARTS_SMALL, (H + 511) / 512); }

template <int EW, int TB, bool XBF16>
__global__ __launch_bounds__(256) void scored_partial(ScoredPass p, int parts)
{
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int tgroups = (p.T + TB - 1) / TB, item = blockIdx.x * 4 + wave;
    if (item >= (p.E + EW - 1) / EW * tgroups * parts) return;
    const int part = item % parts, t0 = item / parts % tgroups * TB, e0 = item / (parts * tgroups) * EW;
    const int steps = (p.H + 511) / 512;
    const int begin = steps * part / parts * 512, end = min(p.H, steps * (part + 1) / parts * 512);
    double acc[EW][TB];
#pragma unroll
    for (int a = 0; a < EW; ++a)
#pragma unroll
        for (int b = 0; b < TB; ++b) acc[a][b] = 0.0;
    constexpr int B = TB == 1 ? 4 : 1;           // steps loaded together
    for (int h0 = begin + 8 * lane; h0 < end; h0 += 512 * B) {
        f32x4 w[B][EW][2];
        u32x4 x[B][TB][XBF16 ? 1 : 2];
#pragma unroll
        for (int s = 0; s < B; ++s) {
            const int h = min(h0 + 512 * s, p.H - 8);
#pragma unroll
            for (int a = 0; a < EW; ++a)
#pragma unroll
                for (int q = 0; q < 2; ++q) w[s][a][q] = *(const f32x4 *)(p.w + (int64_t)min(e0 + a, p.E - 1) * p.H + h + 4 * q);
#pragma unroll
            for (int b = 0; b < TB; ++b) {
                const int64_t at = (int64_t)min(t0 + b, p.T - 1) * p.ldx + h;
                if (XBF16) x[s][b][0] = *(const u32x4 *)((const uint16_t *)p.x + at);
                else {
#pragma unroll
                    for (int q = 0; q < 2; ++q) x[s][b][q] = *(const u32x4 *)((const float *)p.x + at + 4 * q);
                }
            }
        }
#pragma unroll
        for (int s = 0; s < B; ++s)
            if (h0 + 512 * s < end) {
#pragma unroll
                for (int b = 0; b < TB; ++b)
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        double xv;
                        if (XBF16) xv = (double)bf16_bits_to_f32((x[s][b][0][i >> 1] >> (16 * (i & 1))) & 0xffffu);
                        else xv = (double)__uint_as_float(x[s][b][i >> 2][i & 3]);
#pragma unroll
                        for (int a = 0; a < EW; ++a) acc[a][b] = fma(xv, (double)w[s][a][i >> 2][i & 3], acc[a][b]);
                    }
            }
    }
#pragma unroll
    for (int a = 0; a < EW; ++a)
#pragma unroll
        for (int b = 0; b < TB; ++b) {
#pragma unroll
            for (int off = 32; off > 0; off >>= 1) acc[a][b] += __shfl_xor(acc[a][b], off, 64);
            if (lane == a * TB + b && t0 + b < p.T && e0 + a < p.E)
                ((double *)p.logits)[((int64_t)part * p.T + t0 + b) * p.E + e0 + a] = acc[a][b];
        }
}

// More tokens on the fp64 matrix instructions: 64 tokens x 64 experts
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
// 32 of H][w3, w2, w1][64 NG rows][4 chunks of 8 at chunk ^ key(row)], zeros past
// E and H.
constexpr int BM = 128;                          // tokens of a work-group
constexpr int STEP = 32, CHUNK = 128;            // of H: a matrix instruction's depth, a short sum's

int expert_waves(int E) { return E <= 64 ? 1 : E <= 128 ? 2 : 4; }    // NG: columns of 64 experts a work-group has
__host__ __device__ inline int split_steps(int H) { return (H + CHUNK - 1) / CHUNK * (CHUNK / STEP); }
__device__ __forceinline__ int key(int r) { return (r >> 2) & 3; }

__device__ __forceinline__ uint32_t bf16_of(float f) { return __builtin_bit_cast(uint16_t, (__bf16)f); }

__global__ __launch_bounds__(256) void scored_split_w(ScoredPass p, int rows)
{
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.open = 0;
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
            o[(int64_t)(2 - term) * rows * 4] = u;
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
// experts.  x and the terms go to LDS without passing registers, through rings of
// three steps of x and eight terms: at the start of step s, whose three terms
// have landed, those of step s - 1 are free, and the three terms after the five
// that are there or on their way are requested, with x of step s + 2.  The
// smallest term's products are added first, sums run over 128 of H (12
// instructions) and are then added to the totals, which keeps their roundings
// few (value_error).  Parts of H are dealt so that an XCD sees few of
// them: its share of the terms stays in its L2.  8192 x 7168 x 256: 92 us for 90
// Gflop of products (a large library product runs at 1.37 Pflop/s here, 66 us);
// loads alone 50 us, products and LDS reads 75.  Alternating the waves of a SIMD
// between reading and multiplying, as the int8 linear layer does, took 105 us.
constexpr int XRING = 3, TRING = 8;

template <int NG>
__global__ __launch_bounds__(128 * NG) void scored_split_logits(ScoredPass p, int parts)
{
    constexpr int ROWS = 64 * NG, NW = 2 * NG, XB = BM * 64, TERM = ROWS * 64;
    constexpr int LX = BM / 16 / NW, LT = ROWS / 16 / NW;              // loads of a wave: x of a step, a term
    extern __shared__ __align__(16) int8_t ring[];                     // x [XRING][XB], terms [TRING][TERM]
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
    const int8_t *wp = (const int8_t *)p.wsplit + ((int64_t)blk * split_steps(p.H) + begin) * 3 * TERM + wave * LT * 1024 + lane * 16;
    // past the end: the last step again, into slots that nobody reads
    auto fetch_x = [&](int s) {
        int8_t *const buf = ring + s % XRING * XB;
#pragma unroll
        for (int i = 0; i < LX; ++i) {
            // past H: the row's last chunk again, the terms are zero there
            const int h = min((begin + min(s, steps - 1)) * STEP + xc[i], p.H - 8);
            __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)(xp[i] + h),
                                             (__attribute__((address_space(3))) void *)(buf + (wave * LX + i) * 1024), 16, 0, 0);
        }
    };
    auto fetch_term = [&](int u) {               // term u % 3 of step u / 3
        int8_t *const buf = ring + XRING * XB + u % TRING * TERM;
        const int8_t *const at = wp + (int64_t)min(u, 3 * steps - 1) * TERM;
#pragma unroll
        for (int i = 0; i < LT; ++i)
            __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)(at + i * 1024),
                                             (__attribute__((address_space(3))) void *)(buf + (wave * LT + i) * 1024), 16, 0, 0);
    };
    const int wa = wave % NG, wt = wave / NG;
    const int x0 = 64 * wt + fr, w0 = 64 * wa + fr;
    const int xo = x0 * 64 + 16 * (fg ^ key(x0)), wo = w0 * 64 + 16 * (fg ^ key(w0));       // + 1024 a fragment
    f32x4 total[4][4], acc[4][4];
    float ss[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        ss[i] = 0.0f;
#pragma unroll
        for (int j = 0; j < 4; ++j) total[i][j] = acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }
    fetch_x(0);
#pragma unroll
    for (int u = 0; u < 3; ++u) fetch_term(u);
    fetch_term(3);
    fetch_term(4);
    fetch_x(1);
    for (int s = 0; s < steps; ++s) {
        asm volatile("" ::: "memory");
        // vmcnt: the newest two terms and x may be on their way; lgkmcnt(0)
        __builtin_amdgcn_s_waitcnt((2 * LT + LX) | 0x70);
        __builtin_amdgcn_s_barrier();            // step s has landed for everybody, and step s - 1 is read
        asm volatile("" ::: "memory");
        const int8_t *xbuf = ring + s % XRING * XB;
        bf16x8 b[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) b[j] = *(const bf16x8 *)(xbuf + xo + 1024 * j);
        bf16x8 a[3][4];
#pragma unroll
        for (int term = 0; term < 3; ++term)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                a[term][i] = *(const bf16x8 *)(ring + XRING * XB + (3 * s + term) % TRING * TERM + wo + 1024 * i);
        __builtin_amdgcn_sched_barrier(0);       // the reads first
#pragma unroll
        for (int u = 5; u < 8; ++u) fetch_term(3 * s + u);
        fetch_x(s + 2);
#pragma unroll
        for (int term = 0; term < 3; ++term)     // smallest first
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = mfma16x16x32(a[term][i], b[j], acc[i][j]);
        // sums of squares of x, the four fragments shared out over the NG waves
        // that hold the same tokens
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (j % NG == wa && blk == 0 && (begin + s) * STEP + 8 * fg < p.H) {
#pragma unroll
                for (int q = 0; q < 8; q += 2) {
                    const bf16x2 v = {b[j][q], b[j][q + 1]};
                    ss[j] = __builtin_amdgcn_fdot2_f32_bf16(v, v, ss[j], false);
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
    __builtin_amdgcn_s_waitcnt(0x0f70);          // no load may be in flight when the LDS is freed
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
// (a token's scores, groups and top k: scored_dev.h)
constexpr int WAVES = 4;                         // tokens of a work-group, a wave each
constexpr int EXACT_WAVES = 4;                   // waves of a work-group that share a token

// A token left to fp64: `slots` experts in order around the top k with their
// logits, bit j of close where slot j may not be below slot j - 1; 0 slots: the
// whole token.
struct OpenToken {
    int32_t t, slots;
    uint64_t close;
    float logit[64];
    int16_t expert[64];
};

// fp64 selection; a single token is grouped here too (the sorted selection:
// offsets from ballots of the taken flags).  One token of 256 experts: 7.6 us, the
// latency of the scores' exp, the groups' exchanges and k rounds of the maximum.
template <int MAXPL>
__global__ __launch_bounds__(64 * WAVES) void scored_topk(ScoredPass p, int parts)
{
    extern __shared__ double lds[];              // keep < groups: [WAVES][E]
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int t = blockIdx.x * (blockDim.x >> 6) + wave;
    if (t >= p.T) return;
    double l[MAXPL], pr[MAXPL], c[MAXPL];
    load_logits<MAXPL, double>(p, t, parts, lane, l);
    token_scores<MAXPL>(p, l, lane, pr, c);
    if (p.keep < p.groups) {
        const Groups<double> g = rank_groups<MAXPL, double>(p, lane, c, lds + (size_t)wave * p.E);
        const float inv = 1.0f / (float)(p.E / p.groups);
#pragma unroll
        for (int i = 0; i < MAXPL; ++i)
            if (!(g.kept >> group_of(min(lane + 64 * i, p.E - 1), inv) & 1)) c[i] = -INFINITY;
    }
    int my_e;
    double my_c, my_p;
    uint32_t taken;
    select64<MAXPL>(p, lane, c, pr, my_e, my_c, my_p, taken);
    write_token(p, t, lane, my_e, lane < p.k && my_c != -INFINITY ? my_p : 0.0);
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
// order: equal rows of w give equal logits.  The loads go in batches of seven
// stretches of 512 of H: their latency is the cost.
__device__ __forceinline__ double exact_logit(const ScoredPass &p, int t, int e, int lane)
{
    const uint16_t *x = (const uint16_t *)p.x + (int64_t)t * p.ldx;
    const float *w = p.w + (int64_t)e * p.H;
    double s = 0.0;
    constexpr int B = 7;
    for (int h0 = 8 * lane; h0 < p.H; h0 += 512 * B) {
        u32x4 u[B];
        f32x4 a[B], b[B];
#pragma unroll
        for (int i = 0; i < B; ++i) {
            const int h = min(h0 + 512 * i, p.H - 8);
            u[i] = *(const u32x4 *)(x + h);
            a[i] = *(const f32x4 *)(w + h);
            b[i] = *(const f32x4 *)(w + h + 4);
        }
#pragma unroll
        for (int i = 0; i < B; ++i)
            if (h0 + 512 * i < p.H) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    s = fma((double)bf16_bits_to_f32((u[i][j >> 1] >> (16 * (j & 1))) & 0xffffu),
                            (double)(j < 4 ? a[i][j & 3] : b[i][j & 3]), s);
            }
    }
    return wave_sum_f64(s);
}

// replaces the scores and selection values of the flagged experts (bit i:
// expert lane + 64 i) that are not done by those of their fp64 logits, shared
// out over the work-group's waves, which all hold the same token and flags.  ex:
// LDS [E].
template <int MAXPL>
__device__ __forceinline__ void refine(const ScoredPass &p, int t, int wave, int lane, uint32_t flags, uint32_t &done,
                                       double pr[MAXPL], double c[MAXPL], double *ex)
{
    int n = 0;
    __syncthreads();                             // ex is read
#pragma unroll
    for (int i = 0; i < MAXPL; ++i) {
        uint64_t todo = __ballot((flags & ~done) >> i & 1u);
        while (todo) {
            const int o = __ffsll((unsigned long long)todo) - 1;
            todo &= todo - 1;
            if (n++ % EXACT_WAVES == wave) {
                const double l = exact_logit(p, t, o + 64 * i, lane);
                if (lane == 0) ex[o + 64 * i] = l;
            }
        }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < MAXPL; ++i)
        if ((flags & ~done) >> i & 1u) {
            const double l = ex[lane + 64 * i];
            pr[i] = l != l ? 0.0 : sigmoid64(l);
            c[i] = biased(p, lane + 64 * i, l, pr[i]);
        }
    done |= flags;
}

// A bound on the error of a token's selection values from the split router's
// logits.  A logit is off by at most d = rounding |x| max |w_e|.  The matrix
// instruction adds its 32 products to the sum in four groups of 8 (in order of k):
// within a group each product loses what lies below 2^-24 of the largest one (of
// the power of two under it), as the sum before it does, and each of the four
// additions rounds to nearest (and drops 2^-31 of the larger side; an emulation of
// this differs from the instruction in 4 of a million sums, all next to a tie).  In
// units u = 2^-24: 8 u of the products' magnitudes and 4.1 u of the running sum an
// instruction.  A short sum has 12 of them: 49.2 u + 8 u, with 0.5% for the terms
// of w, which add up to that much more than |w|: 58 u.  Then u for each short sum
// of a part and for each part.  All of values that |x| |w| bounds piece by piece (the
// pieces' bounds add up to at most the whole's).  In practice the random signs
// keep it some hundred times smaller.  A selection value is off by at most d / 4,
// the sigmoid's steepest slope, and fp32's roundings.  Infinite where there is no
// bound: NaN, or overflow near.
// c: the experts' biases on return.
template <int MAXPL>
__device__ __forceinline__ float value_error(const ScoredPass &p, int t, int parts, float rounding, int lane, float c[MAXPL])
{
    float wmax = 0.0f, bmax = 0.0f, xn = 0.0f;
#pragma unroll
    for (int i = 0; i < MAXPL; ++i) {
        const int e = min(lane + 64 * i, p.E - 1);
        const float n = p.wnorm[e];
        c[i] = p.bias ? p.bias[e] : 0.0f;
        wmax = n >= 0.0f ? fmaxf(wmax, n) : INFINITY;
        if (fabsf(c[i]) < INFINITY) bmax = fmaxf(bmax, fabsf(c[i]));
    }
    for (int q = 0; q < parts; ++q) xn += p.xnorm[(int64_t)q * p.T + t];
    wmax = wave_max_f32(wmax);
    bmax = wave_max_f32(bmax);
    // squares below fp32's smallest are missing from both sums, of less than 2^-126 each even where they are flushed
    const float lost = 0x1p-126f * (float)p.H;
    const float d = rounding * sqrtf(xn + lost) * sqrtf(wmax + lost);
    return d < 1e30f ? 0.25f * d + 0x1p-21f * (1.0f + bmax) : INFINITY;
}

// The experts around the top k in order, lane j slot j with its expert, value c
// and companion v (a logit or a score): down to the first past k that is more than
// 2 eps below its predecessor, at most 64.  Bit j of close: slot j is not.  Returns
// whether that first one was found (or nothing was left) with at least k slots.
template <int MAXPL, typename V>
__device__ __forceinline__ bool order_slots(const ScoredPass &p, int lane, const V c[MAXPL], const V v[MAXPL], V eps, int &my_e,
                                            V &my_c, V &my_v, int &n, uint64_t &close)
{
    uint32_t taken = 0;
    V last = INFINITY;
    my_e = 0;
    my_c = -INFINITY;
    my_v = 0;
    n = 0;
    close = 0;
    while (true) {
        V bc = -INFINITY, bv = 0;
        int bi = 0;
#pragma unroll
        for (int i = 0; i < MAXPL; ++i)
            if (!((taken >> i) & 1u) && c[i] > bc) { bc = c[i]; bv = v[i]; bi = i; }
        const V m = wave_max(bc);
        const bool near = !(last - m > 2 * eps);
        if (m == -INFINITY || (n >= p.k && !near)) return n >= p.k;
        if (n == 64) return false;
        const int o = __ffsll((unsigned long long)__ballot(bc == m)) - 1;
        if (near) close |= 1ull << n;
        if (lane == o) taken |= 1u << bi;
        const int e = o + 64 * __builtin_amdgcn_readlane(bi, o);
        const V ev = lane_value(bv, o);
        if (lane == n) { my_e = e; my_c = m; my_v = ev; }
        last = m;
        ++n;
    }
}

// Puts the slots (lane j: expert e, score pr, value c) in their fp64 order and
// writes token t: the experts of close slots are summed again, shared out over the
// work-group's waves.  ex: LDS [64].
__device__ __forceinline__ void settle(const ScoredPass &p, int t, int wave, int lane, int slots, uint64_t close, int e, double pr,
                                       double c, double *ex)
{
    uint64_t todo = close | close >> 1;
    __syncthreads();                             // ex is read: by refine for this token, by this function or refine for the last
    for (int i = 0; todo; ++i) {
        const int j = __ffsll((unsigned long long)todo) - 1;
        todo &= todo - 1;
        if (i % EXACT_WAVES != wave) continue;
        const double v = exact_logit(p, t, __builtin_amdgcn_readlane(e, j), lane);
        if (lane == 0) ex[j] = v;
    }
    __syncthreads();
    if (wave == 0) {
        if ((close | close >> 1) >> lane & 1) {
            pr = sigmoid64(ex[lane]);
            c = biased(p, e, ex[lane], pr);
        }
        int slot = lane < slots ? 0 : p.k;
        for (int j = 0; j < slots; ++j) {
            const double v = readlane_f64(c, j);
            const int oe = __builtin_amdgcn_readlane(e, j);
            if (lane < slots) slot += v > c || (v == c && oe < e);
        }
        write_token(p, t, slot, e, slot < p.k ? pr : 0.0);
    }
}

// The tokens that scored_split_topk left open, a work-group each.  Mostly it
// names the experts around the top k in order, and which of them are too close to
// their neighbours: those are settled in fp64.  Otherwise every wave holds the
// whole token and goes the same way: groups around the border are decided on fp64
// values first, then the slots; without a bound, or with more than 64 slots,
// every expert that may be among the k largest is summed again.  8192 tokens of
// 256 experts leave about 900 open, some 100 of them for their groups.
template <int MAXPL>
__global__ __launch_bounds__(64 * EXACT_WAVES) void scored_split_exact(ScoredPass p, int parts, float rounding)
{
    __shared__ double ex[64 * MAXPL], cs[EXACT_WAVES][64 * MAXPL];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int n = *p.open;
    for (int at = blockIdx.x; at < n; at += gridDim.x) {
        const OpenToken &o = ((const OpenToken *)(p.open + 4))[at];
        const int t = o.t, slots = o.slots;
        if (slots > 0) {
            const int e = lane < slots ? o.expert[lane] : 0;
            const double l = lane < slots ? (double)o.logit[lane] : -INFINITY, q = sigmoid64(l);
            settle(p, t, wave, lane, slots, o.close, e, q, lane < slots ? biased(p, e, l, q) : -INFINITY, ex);
            continue;
        }
        double pr[MAXPL], c[MAXPL];
        uint32_t done = 0, flags = 0;
        float l[MAXPL], bias[MAXPL];
        load_logits<MAXPL, float>(p, t, parts, lane, l);
        const double eps = (double)value_error<MAXPL>(p, t, parts, rounding, lane, bias);
#pragma unroll
        for (int i = 0; i < MAXPL; ++i) {
            pr[i] = l[i] != l[i] ? 0.0 : sigmoid64((double)l[i]);
            c[i] = lane + 64 * i < p.E ? biased(p, lane + 64 * i, (double)l[i], pr[i]) : -INFINITY;
            if (!(eps < INFINITY) && lane + 64 * i < p.E) flags |= 1u << i;
        }
        if (!(eps < INFINITY)) refine<MAXPL>(p, t, wave, lane, flags, done, pr, c, ex);
        if (p.keep < p.groups) {
            const float inv = 1.0f / (float)(p.E / p.groups);
            Groups<double> g = rank_groups<MAXPL, double>(p, lane, c, cs[wave]);
            const bool in = g.kept >> lane & 1;
            const double least = -wave_max_f64(in ? -g.score : -INFINITY);
            const double most = wave_max_f64(!in && lane < p.groups ? g.score : -INFINITY);
            flags = 0;
#pragma unroll
            for (int i = 0; i < MAXPL; ++i) {
                const int gr = group_of(min(lane + 64 * i, p.E - 1), inv);
                const double s = __shfl(g.score, gr, 64), b = __shfl(g.second, gr, 64);
                if (lane + 64 * i < p.E && !(least - most > 4.0 * eps) && s <= most + 4.0 * eps && s >= least - 4.0 * eps &&
                    c[i] >= b - 2.0 * eps)
                    flags |= 1u << i;
            }
            refine<MAXPL>(p, t, wave, lane, flags, done, pr, c, ex);
            g = rank_groups<MAXPL, double>(p, lane, c, cs[wave]);
#pragma unroll
            for (int i = 0; i < MAXPL; ++i)
                if (!(g.kept >> group_of(min(lane + 64 * i, p.E - 1), inv) & 1)) {
                    c[i] = -INFINITY;
                    done |= 1u << i;
                }
        }
        int my_e, n_slots;
        double my_c, my_p;
        uint64_t close;
        if (eps < INFINITY && order_slots<MAXPL, double>(p, lane, c, pr, eps, my_e, my_c, my_p, n_slots, close)) {
            settle(p, t, wave, lane, n_slots, close, my_e, my_p, my_c, ex);
            continue;
        }
        uint32_t taken;
        select64<MAXPL>(p, lane, c, pr, my_e, my_c, my_p, taken);
        const double least = readlane_f64(my_c, p.k - 1) - 2.0 * eps;
        flags = 0;
#pragma unroll
        for (int i = 0; i < MAXPL; ++i)
            if (lane + 64 * i < p.E && c[i] >= least) flags |= 1u << i;
        refine<MAXPL>(p, t, wave, lane, flags, done, pr, c, ex);
        select64<MAXPL>(p, lane, c, pr, my_e, my_c, my_p, taken);
        if (wave == 0) write_token(p, t, lane, my_e, lane < p.k && my_c != -INFINITY ? my_p : 0.0);
    }
}

// Selection from the split router's logits where their error leaves no doubt:
// the scores of kept and other groups more than 4 errors apart, and each of the
// k largest values, and the next one, more than 2 from its predecessor.  Other
// tokens go on the list of open ones.
template <int MAXPL>
__global__ __launch_bounds__(64 * WAVES) void scored_split_topk(ScoredPass p, int parts, float rounding)
{
    extern __shared__ double lds[];              // keep < groups: [WAVES][E] floats
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int t = blockIdx.x * WAVES + wave;
    if (t >= p.T) return;
    float l[MAXPL], c[MAXPL];
    load_logits<MAXPL, float>(p, t, parts, lane, l);
    const float eps = value_error<MAXPL>(p, t, parts, rounding, lane, c);
    bool open = !(eps < INFINITY);
#pragma unroll
    for (int i = 0; i < MAXPL; ++i) {
        const float v = 1.0f / (1.0f + expf(-l[i])) + c[i];
        c[i] = lane + 64 * i < p.E && v == v ? v : -INFINITY;
    }
    if (p.keep < p.groups) {
        const Groups<float> g = rank_groups<MAXPL, float>(p, lane, c, (float *)lds + (size_t)wave * p.E);
        const bool in = g.kept >> lane & 1;
        const float least = -wave_max_f32(in ? -g.score : -INFINITY);
        const float most = wave_max_f32(!in && lane < p.groups ? g.score : -INFINITY);
        open = open || !(least - most > 4.0f * eps);
        const float inv = 1.0f / (float)(p.E / p.groups);
#pragma unroll
        for (int i = 0; i < MAXPL; ++i)
            if (!(g.kept >> group_of(min(lane + 64 * i, p.E - 1), inv) & 1)) c[i] = -INFINITY;
    }
    int my_e = 0, n = 0;
    float my_c, my_l = 0.0f;
    uint64_t close = 0;
    // else open: groups, no bound, too many close ones, too few experts
    open = open || !order_slots<MAXPL, float>(p, lane, c, l, eps, my_e, my_c, my_l, n, close);
    if (!open && !close) {
        write_token(p, t, lane, my_e, lane < p.k ? sigmoid64((double)my_l) : 0.0);
        return;
    }
    int at = 0;
    if (lane == 0) at = atomicAdd(p.open, 1);
    OpenToken &o = ((OpenToken *)(p.open + 4))[__builtin_amdgcn_readfirstlane(at)];
    if (lane == 0) {
        o.t = t;
        o.slots = open ? 0 : n;
        o.close = close;
    }
    if (!open && lane < n) {
        o.expert[lane] = (int16_t)my_e;
        o.logit[lane] = my_l;
    }
}

// ---------------------------------------------------------------- grouping
// offsets, perm and inv in one launch, by one work-group, where a bit for every
// token and expert fits LDS with a running count for every 32 tokens: the
// position of (t, e) is e's offset, the count before t's word and the bits below
// t's.  333 tokens of 160 experts: 4 us where the three launches of larger
// batches take 10.
constexpr int GROUP_LDS = 60000, GROUP_T = 4096;

int group_words(int T) { return ((T + 31) / 32) | 1; }                // words of an expert's row, odd: rows on different banks
bool group_fits(int T, int E) { return T <= GROUP_T && (int64_t)E * group_words(T) * 6 <= GROUP_LDS; }

__global__ __launch_bounds__(1024) void scored_group(const int32_t *topk_idx, int T, int E, int k, int words, int32_t *offsets,
                                                     int32_t *perm, int32_t *inv)
{
    extern __shared__ uint32_t mask[];           // [E][words]
    __shared__ int32_t first[1024], sums[16];
    uint16_t *const before = (uint16_t *)(mask + E * words);           // [E][words]
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    for (int i = tid; i < E * words; i += 1024) mask[i] = 0;
    __syncthreads();
    for (int a = tid; a < T * k; a += 1024) {
        const int t = a / k;
        atomicOr(&mask[topk_idx[a] * words + (t >> 5)], 1u << (t & 31));
    }
    __syncthreads();
    int run = 0;
    if (tid < E)
        for (int w = 0; w < words; ++w) {
            before[tid * words + w] = (uint16_t)run;
            run += __popc(mask[tid * words + w]);
        }
    int upto = run;                              // inclusive sum over the experts of the wave, then of those before it
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const int v = __shfl_up(upto, off, 64);
        if (lane >= off) upto += v;
    }
    if (lane == 63) sums[wave] = upto;
    __syncthreads();
    for (int w = 0; w < wave; ++w) upto += sums[w];
    first[tid] = upto - run;
    if (tid < E) offsets[tid] = upto - run;
    if (tid == 0) offsets[E] = T * k;
    __syncthreads();
    for (int a = tid; a < T * k; a += 1024) {
        const int t = a / k, e = topk_idx[a], at = e * words + (t >> 5);
        const int pos = first[e] + before[at] + __popc(mask[at] & ((1u << (t & 31)) - 1u));
        perm[pos] = a;
        inv[a] = pos;
    }
}

}  // namespace

size_t scored_logit_bytes(int T, int H, int E, bool split)
{
    if (split) return (size_t)scored_split_parts(T, H, E) * T * E * sizeof(float);
    return (size_t)(T <= SCORED_SMALL_T ? parts_small(H) : parts64(T, H, E)) * T * E * sizeof(double);
}

size_t scored_open_bytes(int T) { return 4 * sizeof(int32_t) + (size_t)T * sizeof(OpenToken); }

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
        // one token: a wave per expert; more: eight tokens and two experts a wave share what they load
        const int parts = parts_small(p.H), tb = p.T == 1 ? 1 : 8, ew = p.T == 1 ? 1 : 2;
        const int items = (p.E + ew - 1) / ew * ((p.T + tb - 1) / tb) * parts;
        const unsigned grid = (unsigned)((items + 3) / 4);
        if (p.T == 1) {
            if (p.x_bf16) scored_partial<1, 1, true><<<grid, 256, 0, s>>>(p, parts);
            else scored_partial<1, 1, false><<<grid, 256, 0, s>>>(p, parts);
        } else {
            if (p.x_bf16) scored_partial<2, 8, true><<<grid, 256, 0, s>>>(p, parts);
            else scored_partial<2, 8, false><<<grid, 256, 0, s>>>(p, parts);
        }
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
    const size_t lds = XRING * BM * 64 + TRING * rows * 64;
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
    const bool split = scored_split(p.T, p.E, p.softmax, p.x_bf16);
    const int parts = split ? scored_split_parts(p.T, p.H, p.E)
                            : p.T <= SCORED_SMALL_T ? parts_small(p.H) : parts64(p.T, p.H, p.E);
    const int waves = p.T == 1 ? 1 : WAVES;
    const size_t lds = p.keep < p.groups ? (size_t)waves * p.E * sizeof(double) : 0;
    const unsigned grid = (unsigned)(((int64_t)p.T + waves - 1) / waves);
    // see value_error: a short sum, the short sums of a part, the parts; and the roundings of the norms' own sums
    // (H / 8 additions of up to 4 units, half of it in the root)
    const float rounding = 0x1p-24f * (58.0f + (float)((p.H + CHUNK - 1) / CHUNK / parts + 1) + (float)parts) *
                           (1.001f + 0x1p-26f * (float)p.H);
    // a work-group for each of so many open tokens (those without one end at once), more in turns
    const unsigned exact = (unsigned)std::min(p.T, 2048);
    // unrolled for the experts each lane holds (E <= 64 * MAXPL)
#define MOE_TOPK(pl)                                                                              \
    do {                                                                                          \
        if (split) {                                                                              \
            scored_split_topk<pl><<<grid, 64 * WAVES, lds, s>>>(p, parts, rounding);              \
            scored_split_exact<pl><<<exact, 64 * EXACT_WAVES, 0, s>>>(p, parts, rounding);        \
        } else scored_topk<pl><<<grid, 64 * waves, lds, s>>>(p, parts);                           \
    } while (0)
    if (p.E <= 64) MOE_TOPK(1);
    else if (p.E <= 128) MOE_TOPK(2);
    else if (p.E <= 256) MOE_TOPK(4);
    else if (p.E <= 512) MOE_TOPK(8);
    else MOE_TOPK(16);
#undef MOE_TOPK
    return hipGetLastError();
}

bool scored_group_fits(int T, int E) { return group_fits(T, E); }

hipError_t launch_scored_group(const ScoredPass &p, hipStream_t s)
{
    const int words = group_words(p.T);
    scored_group<<<1, 1024, (size_t)p.E * words * 6, s>>>(p.topk_idx, p.T, p.E, p.k, words, p.offsets, p.perm, p.inv);
    return hipGetLastError();
}

}  // namespace moe
