// One MoE block for a few tokens in two kernels.
//
//   s = x + res;  n = rms_norm(s);  scored routing of n;
//   y = sum_j w_j FFN_{e_j}(n) + FFN_shared(n)
//
// The first kernel is the norm and the router's logits.  The second does everything
// else: its work is cut into items (the selection, 8 features of the shared
// gate/up, F features of a routed expert's gate/up, some rows of y) that
// work-groups draw by ticket, in that order, and an item waits only for items of
// lower tickets: for the selection, for h of all experts.  Tickets are drawn by
// running work-groups only, so the lowest unfinished item is always being worked
// on and every wait ends, however many work-groups are resident and whatever else
// runs on the device.  (A bound on the polls ends a wait all the same, should a
// second call overwrite the workspace; y is NaN then.)
//
// Data that a work-group hands to others goes past its XCD's cache (agent-scope
// stores; the arrival counter is raised after they are acknowledged).
//
// Arithmetic.  An activation block of 256 is x = scale * q with integers |q| <= 127
// * 2^16 (23 bits and a sign below the block's largest value), written in three
// int8 digits, so that dot products with integer weights run on the int8 matrix
// instructions exactly: CB2's s_j C and Q2_K's sc_j q are at most 45, the shared
// expert's weights are int8 as they are.  A block's sums leave as fp32, times its
// scales, and are added in fp32.  An activation is off by at most 1.5 units of its
// block's largest value / (127 * 2^16), 1.8e-7 of that value (half a unit for the
// integer, the rest for the reciprocal and the product before it), and its scale by
// an fp32 rounding.  A block whose largest value is below 2^-100 counts as zero: its
// reciprocal would not be finite.
//
// A lane streams a quantized block of its own (a row's four consecutive blocks are
// read by one load, lanes r + 16 g, g = 0..3); the matrix instruction's 16 rows are
// four blocks x (three digits and a spare), zero where a lane's block is another
// one: sums of different blocks never mix, and each arrives in the lane that holds
// the block's scale.
//
// What bounds it.  Its floor is the weights of the experts that the tokens chose,
// but the parts stand in a row and each has its latency: one token, H 7168, I 2048,
// 8 of 256 experts and a shared one, 125 MB: 50 us (2.5 TB/s; a large copy reaches
// 5.1): 10 until the experts are known (the shared gate/up runs beside it), 10 of
// routed gate/up (6 without its arithmetic, 8 without its loads), 9 until every h is
// there, 9 of rows of y, and the drain.  Four such tokens, 332 MB: 127 us (2.6 TB/s;
// the SIMDs issue vector instructions 44% of the time).  Sixteen of a small layer (H
// 2048, I 768, 6 of 64), 60 MB: 95 us, of which the rows of y are 41, on half of the
// CUs and in six passes over h, and the routed gate/up 10 to 25, whose tokens' digits
// are staged for every pair (vector instructions 23% of the time).  The norm before
// it: 7, 12 and 9 us.  One work-group a CU of eight waves, because the tables and
// digits take most of the LDS and the products up to 256 registers (the same with 12
// waves 65 us and with 16, which spill, 80, when this took 62).
#include "block.h"
#include "common.h"
#include "devcache.h"
#include "scored_dev.h"

#include <algorithm>

namespace moe {

namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4u __attribute__((ext_vector_type(4), aligned(4)));
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x2u __attribute__((ext_vector_type(2), aligned(4)));

constexpr int NORM_NT = 1024, NORM_NW = NORM_NT / 64;
constexpr int NT = 512, NW = NT / 64;
constexpr int QUAD = 16 * 4 * 3 * 16;            // bytes of four blocks' digits: [16 steps][4 blocks][3 digits][16]
constexpr float QMAX = 127.0f * 65536.0f;
// 64 features of a row of h: [4 steps][3 digits][16] in the order of Q2_K's codes (dword i of a step = features i, i + 4, i + 8,
// i + 12), the sums of the four steps (fp32) and the scale.  A record has lines of its own in the workspace; in LDS four
// records are a block's, a little apart from the next block's for the banks' sake.
constexpr int REC = 224, REC_SUMS = 192, REC_SCALE = 208, REC_LINES = 256, REC_BLOCK = 4 * REC + 48;
constexpr int LINE = 32;                         // uint32s of a counter's line
enum { C_TICKET = 0, C_LIST = LINE, C_SHARED = 2 * LINE, C_ROUTED = 3 * LINE, C_WORDS = 4 * LINE };
constexpr int TABLE = 32768;                     // LDS: [256 codewords][16 copies]
constexpr int O_ZERO = TABLE;                    // zeros for the lanes whose rows of the matrix instruction are empty
constexpr int O_SMALL = TABLE + QUAD;            // the parts' small arrays

struct Small {
    union {
        struct {
            uint32_t mask[BLOCK_MAX_E];          // tokens of an expert
            float weight[BLOCK_MAX_T * BLOCK_MAX_K];
            int32_t sums[2][NW];
            int16_t chosen[BLOCK_MAX_T * BLOCK_MAX_K], first[BLOCK_MAX_E];
        } select;
        struct {
            int16_t token[2], slot[2], row[2];   // of the tokens in hand: their slots of digits, their rows of h
        } routed;
    };
    // the list: different experts (expert, first position, tokens), and each position's token, weight and expert's number
    int32_t entry[BLOCK_MAX_T * BLOCK_MAX_K];
    float weight[BLOCK_MAX_T * BLOCK_MAX_K];
    int16_t tok[BLOCK_MAX_T * BLOCK_MAX_K], seg[BLOCK_MAX_T * BLOCK_MAX_K];
};
constexpr int O_END = O_SMALL + (sizeof(Small) + 15) / 16 * 16;

__device__ __forceinline__ float to_f32(const uint32_t w, int hi) { return __uint_as_float(hi ? w & 0xffff0000u : w << 16); }

template <class T>
__device__ __forceinline__ T peek(const T *p) { return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); }
template <class T>
__device__ __forceinline__ void post(T *p, T v) { __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); }

// The kernel's parts are functions of their own, so that none's loop invariants and registers weigh on another's (one body
// took 10 us before its first item, with 1500 instructions on spilled scalars).  Each finds the arguments in the kernel's
// argument segment and loads what it needs into scalar registers.
struct Args { uint32_t lo, hi; };

__device__ __forceinline__ const BlockPass &args_of(Args a)
{
    const uint64_t at = (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)a.hi) << 32 |
                        (uint32_t)__builtin_amdgcn_readfirstlane((int)a.lo);
    return *(const BlockPass *)(const __attribute__((address_space(4))) BlockPass *)at;
}

// three signed digits of base 256, least first
__device__ __forceinline__ void digits(int q, int &d0, int &d1, int &d2)
{
    d0 = (int)(int8_t)q;
    q = (q - d0) >> 8;
    d1 = (int)(int8_t)q;
    d2 = (q - d1) >> 8;
}

__device__ __forceinline__ uint32_t bytes4(int a, int b, int c, int d)
{
    return (uint32_t)(a & 255) | (uint32_t)(b & 255) << 8 | (uint32_t)(c & 255) << 16 | (uint32_t)d << 24;
}

// sum over the lanes r, r + 16, r + 32, r + 48
__device__ __forceinline__ float sum_rows(float v)
{
    uint32_t u = __float_as_uint(v);
    auto a = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    u = __float_as_uint(__uint_as_float(a[0]) + __uint_as_float(a[1]));
    a = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    return __uint_as_float(a[0]) + __uint_as_float(a[1]);
}

// largest of the wave's non-negative integers: four steps within rows of 16 lanes, then across them
__device__ __forceinline__ uint32_t max_bits(uint32_t v)
{
    v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, false));      // quad_perm [1,0,3,2]
    v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, false));      // quad_perm [2,3,0,1]
    v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x141, 0xF, 0xF, false));     // row_half_mirror
    v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x140, 0xF, 0xF, false));     // row_mirror
    auto a = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    v = max(a[0], a[1]);
    a = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    return max(a[0], a[1]);
}

// scale and its reciprocal for a block whose largest magnitude has the bits m (an infinity or a NaN wins, and makes the scale NaN)
__device__ __forceinline__ float block_scale(uint32_t m, float &inv)
{
    const float amax = __uint_as_float(m);
    const bool finite = m < 0x7f800000u, some = amax >= 0x1p-100f;
    inv = finite && some ? QMAX / amax : 0.0f;
    return !finite ? __uint_as_float(0x7fc00000u) : some ? amax / QMAX : 0.0f;
}

// ---------------------------------------------------------------- norm and logits
// A work-group a token and a few experts, 8 elements of the token a thread: the
// operations of the row kernels' norm, in their order, in every work-group of the
// token; the first of them leaves s and the digits of n.  s goes to the
// workspace, and where the caller wants it by the second kernel: it may replace
// the residual, which other work-groups still read here.  Clears the counters.
__device__ __forceinline__ void load8(const void *p, int bf16, int64_t at, float v[8])
{
    if (bf16) {
        const u32x4 u = *(const u32x4 *)((const uint16_t *)p + at);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = to_f32(u[j >> 1], j & 1);
    } else {
        const f32x4 a = *(const f32x4 *)((const float *)p + at), b = *(const f32x4 *)((const float *)p + at + 4);
#pragma unroll
        for (int j = 0; j < 4; ++j) { v[j] = a[j]; v[4 + j] = b[j]; }
    }
}

__device__ __forceinline__ uint32_t bf16_bits(float f) { return __builtin_bit_cast(uint16_t, (__bf16)f); }

__global__ __launch_bounds__(NORM_NT) void block_norm(BlockPass p)
{
    __shared__ double part[NORM_NW], logit[NORM_NW][4];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, t = blockIdx.x, c = 8 * tid;
    const bool lead = blockIdx.y == 0;
    if (t == 0 && lead && tid < C_WORDS) p.ctl[tid] = 0;
    const bool in = c < p.H;
    const int at = in ? c : 0;                   // something in bounds
    const int e0 = blockIdx.y * p.experts, e1 = min(e0 + p.experts, p.E);
    float v[8], g[8], w[4][8];                   // up to four experts' weights are on their way during the norm
    auto load_w = [&](int e, float o[8]) {
        if (e < e1) load8(p.route.w, 0, (int64_t)e * p.H + at, o);
    };
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) w[i][j] = 0.0f;
    load8(p.x, p.x_bf16, (int64_t)t * p.ldx + at, v);
    load8(p.norm_w, 0, at, g);
    if (p.res) {
        float r[8];
        load8(p.res, p.res_bf16, (int64_t)t * p.ldres + at, r);
#pragma unroll
        for (int i = 0; i < 4; ++i) load_w(e0 + i, w[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            v[j] = v[j] + r[j];
            if (p.res_bf16) v[j] = __uint_as_float(bf16_bits(v[j]) << 16);
        }
        if (p.sum && lead && in) {
            const int64_t o = (int64_t)t * p.H + c;
            if (p.res_bf16) {
                u32x4 u;
#pragma unroll
                for (int j = 0; j < 4; ++j) u[j] = bf16_bits(v[2 * j]) | bf16_bits(v[2 * j + 1]) << 16;
                *(u32x4 *)((uint16_t *)p.s + o) = u;
            } else {
                *(f32x4 *)((float *)p.s + o) = f32x4{v[0], v[1], v[2], v[3]};
                *(f32x4 *)((float *)p.s + o + 4) = f32x4{v[4], v[5], v[6], v[7]};
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) load_w(e0 + i, w[i]);
    }
    double ss = 0.0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        v[j] = in ? v[j] : 0.0f;
        ss = fma((double)v[j], (double)v[j], ss);
    }
    ss = wave_sum_f64(ss);
    if (lane == 0) part[wave] = ss;
    __syncthreads();
    ss = part[0];
#pragma unroll
    for (int q = 1; q < NORM_NW; ++q) ss += part[q];
    const float r = (float)(1.0 / sqrt(ss / (double)p.H + (double)p.eps));
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        v[j] = in ? (v[j] * r) * g[j] : 0.0f;
        if (p.n_bf16) v[j] = __uint_as_float(bf16_bits(v[j]) << 16);
        m = max(m, __float_as_uint(v[j]) & 0x7fffffffu);
    }
    if (lead) {
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, off, 64));  // the 32 threads of a block
        if (c < p.nq * 1024) {
            float inv;
            const float scale = block_scale(m, inv);
            if ((tid & 31) == 0) p.scales[t * 4 * p.nq + (tid >> 5)] = scale;
            int d[8][3];
#pragma unroll
            for (int j = 0; j < 8; ++j) digits((int)rintf(v[j] * inv), d[j][2], d[j][1], d[j][0]);
            // block tid / 32, step tid / 2 % 16, half tid % 2
            int8_t *o = p.planes + ((int64_t)t * p.nq + (tid >> 7)) * QUAD + ((tid >> 1) & 15) * 192 + ((tid >> 5) & 3) * 48 + (tid & 1) * 8;
#pragma unroll
            for (int q = 0; q < 3; ++q)
                *(uint2 *)(o + 16 * q) = uint2{bytes4(d[0][q], d[1][q], d[2][q], d[3][q]), bytes4(d[4][q], d[5][q], d[6][q], d[7][q])};
        }
    }
    // fp64 logits, four experts at a time
    for (int e = e0; e < e1; e += 4) {
        if (e > e0) {
            __syncthreads();                     // the sums are read
#pragma unroll
            for (int i = 0; i < 4; ++i) load_w(e + i, w[i]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (e + i >= e1) break;
            double l = 0.0;
#pragma unroll
            for (int j = 0; j < 8; ++j) l = fma((double)v[j], in ? (double)w[i][j] : 0.0, l);
            l = wave_sum_f64(l);
            if (lane == 0) logit[wave][i] = l;
        }
        __syncthreads();
        if (tid < 4 && e + tid < e1) {
            double l = logit[0][tid];
            for (int q = 1; q < NORM_NW; ++q) l += logit[q][tid];
            p.logits[(int64_t)t * p.E + e + tid] = l;
        }
    }
}

// ---------------------------------------------------------------- the rest
__device__ __forceinline__ i32x4 mfma_i8(const i32x4 &a, const i32x4 &b, const i32x4 &c)
{
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, c, 0, 0, 0);
}

// the sum that three digits' sums (most significant first) stand for
__device__ __forceinline__ float joined(const i32x4 &a) { return fmaf((float)a[0], 65536.0f, (float)(a[1] * 256 + a[2])); }

extern __shared__ __align__(16) int8_t smem[];
__device__ __forceinline__ Small &small() { return *(Small *)(smem + O_SMALL); }

// Thread 0 waits until *p is at least n; false if that does not come (two seconds or more).
constexpr int POLLS = 1 << 21;

__device__ bool wait_for(const uint32_t *p, uint32_t n)
{
    for (int i = 0; i < POLLS; ++i) {
        if (peek(p) >= n) return true;
        __builtin_amdgcn_s_sleep(1);
    }
    return false;
}

// All of a work-group's posts are acknowledged before thread 0 raises the counter (and draws the next ticket with it).
__device__ __forceinline__ uint32_t draw(uint32_t *ctl)
{
    return __hip_atomic_fetch_add(ctl + C_TICKET, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

__device__ __forceinline__ void arrive(uint32_t *ctl, int counter, uint32_t &next)
{
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    if (threadIdx.x == 0) {
        __hip_atomic_fetch_add(ctl + counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        next = draw(ctl);
    }
}

// digits and scales of tokens t0 .. t0 + n - 1 (list: of the tokens in it) into LDS slots
__device__ __noinline__ void stage_tokens(Args pa, int t0, const int16_t *tokens, int n)
{
    const BlockPass &p = args_of(pa);
    const int per = p.nq * (QUAD / 16);
    for (int i = threadIdx.x; i < n * per; i += NT) {
        const int j = i / per, t = tokens ? tokens[j] : t0 + j;
        ((u32x4 *)(smem + p.o_planes))[i] = ((const u32x4 *)p.planes)[(int64_t)t * per + (i - j * per)];
    }
    float *const sc = (float *)(smem + p.o_scales);
    for (int i = threadIdx.x; i < n * 4 * p.nq; i += NT) {
        const int j = i / (4 * p.nq), t = tokens ? tokens[j] : t0 + j;
        sc[i] = p.scales[t * 4 * p.nq + (i - j * 4 * p.nq)];
    }
}

// ---- the selection: a wave a token, then the grouping and the list of experts
template <int MAXPL>
__device__ __noinline__ void select(Args pa)
{
    const BlockPass &p = args_of(pa);
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int E = p.E, k = p.k, n = p.T * k;
    auto &mask = small().select.mask;
    auto &weight = small().select.weight;
    auto &sums = small().select.sums;
    auto &chosen = small().select.chosen;
    auto &first = small().select.first;
    double *const cs = (double *)(smem + p.o_planes);                  // [T][E]
    if (tid < BLOCK_MAX_E) mask[tid] = 0;
    for (int t = wave; t < p.T; t += NW) {
        double l[MAXPL], pr[MAXPL], c[MAXPL];
#pragma unroll
        for (int i = 0; i < MAXPL; ++i)
            l[i] = lane + 64 * i < E ? p.logits[(int64_t)t * E + lane + 64 * i] : -INFINITY;
        token_scores<MAXPL>(p.route, l, lane, pr, c);
        if (p.route.keep < p.route.groups) {
            const Groups<double> g = rank_groups<MAXPL, double>(p.route, lane, c, cs + t * E);
            const float inv = 1.0f / (float)(E / p.route.groups);
#pragma unroll
            for (int i = 0; i < MAXPL; ++i)
                if (!(g.kept >> group_of(min(lane + 64 * i, E - 1), inv) & 1)) c[i] = -INFINITY;
        }
        int my_e;
        double my_c, my_p;
        uint32_t taken;
        select64<MAXPL>(p.route, lane, c, pr, my_e, my_c, my_p, taken);
        const float w = write_token(p.route, t, lane, my_e, lane < k && my_c != -INFINITY ? my_p : 0.0);
        if (lane < k) {
            chosen[t * k + lane] = (int16_t)my_e;
            weight[t * k + lane] = w;
        }
    }
    __syncthreads();
    if (tid < n) atomicOr(&mask[chosen[tid]], 1u << (tid / k));
    __syncthreads();
    // positions and numbers of the experts, by an inclusive sum over waves and then their totals
    const uint32_t m = tid < E ? mask[tid] : 0;
    int upto = __popc(m), used = m != 0;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const int a = __shfl_up(upto, off, 64), b = __shfl_up(used, off, 64);
        if (lane >= off) { upto += a; used += b; }
    }
    if (lane == 63) { sums[0][wave] = upto; sums[1][wave] = used; }
    __syncthreads();
    int all = 0;
    for (int w = 0; w < NW; ++w) {
        if (w < wave) { upto += sums[0][w]; used += sums[1][w]; }
        all += sums[1][w];
    }
    const int begin = upto - __popc(m);
    if (tid < E) {
        first[tid] = (int16_t)begin;
        p.route.offsets[tid] = begin;
        if (m) post(p.list + used - 1, (int32_t)(tid | begin << 10 | (int)__popc(m) << 20));
    }
    if (tid == 0) p.route.offsets[E] = n;
    __syncthreads();
    if (tid < n) {
        const int t = tid / k, e = chosen[tid], pos = first[e] + __popc(mask[e] & ((1u << t) - 1u));
        p.route.perm[pos] = tid;
        p.route.inv[tid] = pos;
        post(p.list + 256 + pos, t);
        post((float *)p.list + 512 + pos, weight[tid]);
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    if (tid == 0) post(p.ctl + C_LIST, (uint32_t)all);
}

// ---- 8 features of the shared gate/up: a tile of rows gate f .. f + 7, up f .. f + 7; the waves take the blocks of K in turn
__device__ __forceinline__ const int8_t *digit_base(const BlockPass &p, bool in, int slot, int stride, int at)
{
    return in ? smem + p.o_planes + slot * stride + at : smem + O_ZERO;
}

__device__ __forceinline__ i32x4 load_row16(const int8_t *row, int at, int K)
{
    i32x4 v = {0, 0, 0, 0};
    if (at < K) v = *(const i32x4 *)(row + at);
    return v;
}

__device__ __noinline__ void shared_item(Args pa, int item, int t0, int nt)
{
    const BlockPass &p = args_of(pa);
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, r = lane & 15, g = lane >> 4;
    const int f = 8 * item + (r & 7);
    const int8_t *const row = p.sh_up + (int64_t)((r < 8 ? 0 : p.sh) + min(f, p.sh - 1)) * p.ld_up;
    const int slot = r >> 2, digit = r & 3;                            // this lane's row of the instruction
    const bool in = digit < 3 && slot < nt;
    const float *const sc = (const float *)(smem + p.o_scales) + min(g, nt - 1) * 4 * p.nq;
    float v = 0.0f;
    for (int b = wave; b < p.nb; b += NW) {
        i32x4 w[4];
#pragma unroll
        for (int s = 0; s < 4; ++s) w[s] = load_row16(row, 256 * b + 64 * s + 16 * g, p.H);
        const int8_t *const a = digit_base(p, in, slot, p.nq * QUAD, (b >> 2) * QUAD + g * 192 + ((b & 3) * 3 + digit) * 16);
        i32x4 acc = {0, 0, 0, 0};
#pragma unroll
        for (int s = 0; s < 4; ++s) acc = mfma_i8(*(const i32x4 *)(a + s * 768), w[s], acc);
        v = fmaf(joined(acc), sc[b], v);                               // lane (r, g): row r, token g
    }
    float *const red = (float *)(smem + p.o_red);
    red[wave * 64 + lane] = v;
    __syncthreads();
    if (tid < 32 && (tid >> 3) < nt && 8 * item + (tid & 7) < p.sh) {
        const int fo = tid & 7, t = tid >> 3, ff = 8 * item + fo;
        float a = 0.0f, u = 0.0f;
        for (int w = 0; w < NW; ++w) {
            a += red[w * 64 + 16 * t + fo];
            u += red[w * 64 + 16 * t + 8 + fo];
        }
        a *= p.up_scale[ff];
        u *= p.up_scale[p.sh + ff];
        if (p.up_bias) { a += p.up_bias[ff]; u += p.up_bias[p.sh + ff]; }
        post(p.hs + (int64_t)(t0 + t) * p.sh + ff, a / (1.0f + expf(-a)) * u);
    }
}

// ---- F features of a routed expert's gate/up, N tokens (their digits in slots s0 ..): a unit is 16 features and a quad of blocks
struct Window { uint32_t w[10]; };

__device__ __forceinline__ Window load_window(const uint8_t *at)
{
    const uint32_t *const q = (const uint32_t *)((uintptr_t)at & ~(uintptr_t)3);
    const u32x4u a = *(const u32x4u *)q, b = *(const u32x4u *)(q + 4);
    const u32x2u c = *(const u32x2u *)(q + 8);
    return Window{{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3], c[0], c[1]}};
}

// Fields of a block whose first byte is byte 0 (odd = 0) or 2 of its window.
struct Cb2 {
    uint32_t idx[8], scales;
    float d;
    __device__ __forceinline__ Cb2(const Window &v, bool odd)
    {
        const uint32_t sel = odd ? 0x07060504u : 0x05040302u;
#pragma unroll
        for (int j = 0; j < 8; ++j) idx[j] = __builtin_amdgcn_perm(v.w[2 + j], v.w[1 + j], sel);
        scales = __builtin_amdgcn_perm(v.w[1], v.w[0], sel);
        d = f16_bits_to_f32((odd ? v.w[0] >> 16 : v.w[0]) & 0xffffu);
    }
    __device__ __forceinline__ int scale(int j) const { return (int)(scales >> (4 * j) & 15u); }
};

// The codewords go to the matrix instructions as they are, the sums of a sub-block are multiplied by its s_j: three products
// a token instead of eight permuted dwords of scaled weights.
template <int N>
__device__ __forceinline__ void routed_unit(const Cb2 &gb, const Cb2 &ub, const int8_t *const a[N], i32x4 ag[N], i32x4 au[N])
{
    const uint32_t copy = (threadIdx.x & 15) * 8;
    auto codes = [&](uint32_t idx, int q) {      // codewords 2 q and 2 q + 1 of a sub-block
        const uint32_t at0 = ((q == 0 ? idx << 7 : idx >> 9) & 0x7f80u) | copy, at1 = (idx >> (16 * q + 1) & 0x7f80u) | copy;
        const uint2 x = *(const uint2 *)(smem + at0), y = *(const uint2 *)(smem + at1);
        return i32x4{(int)x.x, (int)x.y, (int)y.x, (int)y.y};
    };
#pragma unroll
    for (int n = 0; n < N; ++n) ag[n] = au[n] = i32x4{0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        if (N > 1) __builtin_amdgcn_sched_barrier(0);                  // few sub-blocks' LDS reads in registers at once
        const i32x4 g0 = codes(gb.idx[j], 0), g1 = codes(gb.idx[j], 1), u0 = codes(ub.idx[j], 0), u1 = codes(ub.idx[j], 1);
        const int gs = gb.scale(j), us = ub.scale(j);
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const i32x4 x0 = *(const i32x4 *)(a[n] + 2 * j * 192), x1 = *(const i32x4 *)(a[n] + (2 * j + 1) * 192);
            const i32x4 g = mfma_i8(x1, g1, mfma_i8(x0, g0, i32x4{0, 0, 0, 0})), u = mfma_i8(x1, u1, mfma_i8(x0, u0, i32x4{0, 0, 0, 0}));
#pragma unroll
            for (int i = 0; i < 3; ++i) {
                ag[n][i] += __mul24(g[i], gs);
                au[n][i] += __mul24(u[i], us);
            }
        }
    }
}

template <int N>
__device__ __forceinline__ void routed_units(const BlockPass &p, int e, int f0, int n)
{
    const auto &slots = small().routed.slot;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), r = lane & 15, g = lane >> 4;
    const int units = p.F / 16 * p.nq;
    const bool in = (r & 3) < 3 && (r >> 2) == g;
    const float *const sc = (const float *)(smem + p.o_scales);
    float *const red = (float *)(smem + p.o_red);                      // [units][N][gate, up][16]
    auto block_at = [&](const uint8_t *w, int u) {
        const int row = min(f0 + u / p.nq * 16 + r, p.I - 1), b = min(4 * (u % p.nq) + g, p.nb - 1);
        return w + (((int64_t)e * p.I + row) * p.nb + b) * 38;
    };
    struct Pair { Window g, u; };
    auto load = [&](int u, Pair &w) {
        if (u < units) {
            w.g = load_window(block_at(p.gate, u));
            w.u = load_window(block_at(p.up, u));
        }
    };
    // the next unit's blocks are requested before this one's arithmetic
    auto unit = [&](int u, Pair &w) {
        const Cb2 gb(w.g, (uintptr_t)block_at(p.gate, u) & 2), ub(w.u, (uintptr_t)block_at(p.up, u) & 2);
        load(u + NW, w);
        const int q = u % p.nq, b = 4 * q + g;
        const int8_t *a[N];
        i32x4 ag[N], au[N];
#pragma unroll
        for (int j = 0; j < N; ++j)
            a[j] = digit_base(p, in && j < n, slots[min(j, n - 1)], p.nq * QUAD, q * QUAD + ((r >> 2) * 3 + (r & 3)) * 16);
        routed_unit<N>(gb, ub, a, ag, au);
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const float s = b < p.nb && j < n ? sc[slots[min(j, n - 1)] * 4 * p.nq + b] : 0.0f;
            float x = b < p.nb ? joined(ag[j]) * (gb.d * s) : 0.0f, y = b < p.nb ? joined(au[j]) * (ub.d * s) : 0.0f;
            x = sum_rows(x);
            y = sum_rows(y);
            if (g < 2) red[(u * N + j) * 32 + lane] = g ? y : x;
        }
    };
    Pair next;
    load(wave, next);
    for (int u = wave; u < units; u += NW) unit(u, next);
    __syncthreads();
    // a wave finishes 64 features of a token: SwiGLU, digits, sums
    const int groups = p.F / 64;
    for (int i = wave; i < n * groups; i += NW) {
        const int j = i / groups, f = i % groups * 64 + lane;
        float a = 0.0f, u = 0.0f;
        for (int q = 0; q < p.nq; ++q) {
            const float *const x = red + ((f / 16 * p.nq + q) * N + j) * 32 + f % 16;
            a += x[0];
            u += x[16];
        }
        const float h = f0 + f < p.I ? a / (1.0f + expf(-a)) * u : 0.0f;
        float inv;
        const float scale = block_scale(max_bits(__float_as_uint(h) & 0x7fffffffu), inv);
        int x = (int)rintf(h * inv), d0, d1, d2;
        digits(x, d2, d1, d0);
        // bytes to their places by way of LDS
        int8_t *const rec = smem + p.o_recs + wave * REC;
        int8_t *const o = rec + (lane >> 4) * 48 + 4 * (lane & 3) + (lane >> 2 & 3);
        o[0] = (int8_t)d0;
        o[16] = (int8_t)d1;
        o[32] = (int8_t)d2;
        x += __builtin_amdgcn_mov_dpp(x, 0xB1, 0xF, 0xF, false);       // the 16 lanes of a step
        x += __builtin_amdgcn_mov_dpp(x, 0x4E, 0xF, 0xF, false);
        x += __builtin_amdgcn_mov_dpp(x, 0x141, 0xF, 0xF, false);
        x += __builtin_amdgcn_mov_dpp(x, 0x140, 0xF, 0xF, false);
        if ((lane & 15) == 0) ((float *)(rec + REC_SUMS))[lane >> 4] = (float)x * scale;
        if (lane == 0) *(float *)(rec + REC_SCALE) = scale;
        wave_sync();
        if (lane < REC / 4)
            post((uint32_t *)(p.h + ((int64_t)small().routed.row[j] * p.records + (f0 + f) / 64) * REC_LINES) + lane, ((const uint32_t *)rec)[lane]);
        wave_sync();
    }
}

__device__ __forceinline__ void routed_item(const BlockPass &p, Args pa, int item)
{
    auto &now = small().routed;
    const int d = item / p.nf, f0 = item % p.nf * p.F;
    const int entry = small().entry[d], e = entry & 1023, first = entry >> 10 & 1023, n = entry >> 20;
    for (int j0 = 0; j0 < n; j0 += 2) {
        const int m = min(2, n - j0);
        __syncthreads();
        if (threadIdx.x < m) {
            const int i = threadIdx.x, t = small().tok[first + j0 + i];
            now.token[i] = (int16_t)t;
            now.slot[i] = (int16_t)(p.T <= p.slots ? t : i);
            now.row[i] = (int16_t)(first + j0 + i);
        }
        __syncthreads();
        if (p.T > p.slots) {
            stage_tokens(pa, 0, now.token, m);
            __syncthreads();
        }
        if (m == 1) routed_units<1>(p, e, f0, m);
        else routed_units<2>(p, e, f0, m);
    }
}

// ---- some rows of y: the shared expert's down rows and every chosen expert's
// Digits of rows of the shared expert's h into LDS.
__device__ __forceinline__ void stage_shared(const BlockPass &p, int t0, int count)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int nb = 4 * p.nqs;
    int8_t *const planes = smem + p.o_planes;
    float *const sc = (float *)(planes + count * p.nqs * QUAD);
    for (int i = wave; i < count * nb; i += NW) {
        const int row = i / nb, b = i - row * nb, at = 256 * b + 4 * lane;
        float v[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) v[c] = at + c < p.sh ? peek(p.hs + (int64_t)(t0 + row) * p.sh + at + c) : 0.0f;
        uint32_t m = 0;
#pragma unroll
        for (int c = 0; c < 4; ++c) m = max(m, __float_as_uint(v[c]) & 0x7fffffffu);
        float inv;
        const float scale = block_scale(max_bits(m), inv);
        int d[4][3];
#pragma unroll
        for (int c = 0; c < 4; ++c) digits((int)rintf(v[c] * inv), d[c][2], d[c][1], d[c][0]);
        int8_t *const o = planes + (row * p.nqs + (b >> 2)) * QUAD + (lane >> 2) * 192 + (b & 3) * 48 + 4 * (lane & 3);
#pragma unroll
        for (int c = 0; c < 3; ++c) *(uint32_t *)(o + 16 * c) = bytes4(d[0][c], d[1][c], d[2][c], d[3][c]);
        if (lane == 0) sc[i] = scale;
    }
}

// Records of `count` rows of h from c0 on into LDS; what no item has written (past inter) is zero.  Plain loads: a record's lines
// hold nothing else (block_workspace), and no cache can have an older copy, since this kernel reads them here alone, after their
// item has counted itself in, and the caches were emptied at its start.
__device__ __forceinline__ void stage_h(const BlockPass &p, int c0, int count)
{
    constexpr int PIECES = REC / 16;
    const int per_row = p.nqi * 16;              // records of a row in LDS
    int8_t *const planes = smem + p.o_planes;
    // a record is shared out over 16 threads, the last two idle
    for (int i = threadIdx.x; i < count * per_row * 16; i += NT) {
        const int rec = i >> 4, piece = i & 15, row = rec / per_row, at = rec - row * per_row;
        if (piece >= PIECES) continue;
        u32x4 v = {0, 0, 0, 0};
        if (at < p.records) v = *(const u32x4 *)(p.h + ((int64_t)(c0 + row) * p.records + at) * REC_LINES + 16 * piece);
        *(u32x4 *)(planes + (row * p.nqi * 4 + (at >> 2)) * REC_BLOCK + (at & 3) * REC + 16 * piece) = v;
    }
}

// N rows of h from i0 on (LDS rows) with 16 rows of one expert's down matrix and a quad of its blocks, times the rows' weights,
// onto this wave's sums
template <int N>
__device__ __forceinline__ void down_rows(const BlockPass &p, const uint32_t c[21], int c0, int i0, int n, int quad, float *ya)
{
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4, b = 4 * quad + g;
    const int8_t *const planes = smem + p.o_planes;
    const int beta = r >> 2, digit = r & 3;
    const int8_t *a[N], *rec[N];
    float v[N], off[N];
#pragma unroll
    for (int j = 0; j < N; ++j) {
        const int row = (i0 + min(j, n - 1)) * p.nqi * 4;
        a[j] = beta == g && digit < 3 ? planes + (row + 4 * quad + beta) * REC_BLOCK + digit * 16 : smem + O_ZERO;
        rec[j] = planes + (row + b) * REC_BLOCK;
        v[j] = off[j] = 0.0f;
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {                // 64 features with a scale of their own
        i32x4 acc[N];
#pragma unroll
        for (int j = 0; j < N; ++j) acc[j] = i32x4{0, 0, 0, 0};
        const uint32_t sc = c[1 + q] & 0x0f0f0f0fu;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t code = c[5 + 4 * q + i];
            asm volatile("" : "+v"(code));       // expanded here, not once for all rows: the registers are not there
            // four codes of 2 bits in the bytes, times the scale in both halves: at most 45, no carry between bytes
            const u16x2 s = __builtin_bit_cast(u16x2, __builtin_amdgcn_perm(sc, sc, 0x0c000c00u | 0x00010001u * i));
            i32x4 w;
#pragma unroll
            for (int k = 0; k < 4; ++k) w[k] = __builtin_bit_cast(int, (u16x2)(__builtin_bit_cast(u16x2, code >> (2 * k) & 0x03030303u) * s));
#pragma unroll
            for (int j = 0; j < N; ++j) acc[j] = mfma_i8(*(const i32x4 *)(a[j] + q * REC + i * 48), w, acc[j]);
        }
        const uint32_t m = c[1 + q] >> 4 & 0x0f0f0f0fu;
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const f32x4 s = *(const f32x4 *)(rec[j] + q * REC + REC_SUMS);
#pragma unroll
            for (int i = 0; i < 4; ++i) off[j] = fmaf((float)(m >> (8 * i) & 255u), s[i], off[j]);
            v[j] = fmaf(joined(acc[j]), *(const float *)(rec[j] + q * REC + REC_SCALE), v[j]);
        }
    }
    const float d = f16_bits_to_f32(c[0] & 0xffffu), dmin = f16_bits_to_f32(c[0] >> 16);
#pragma unroll
    for (int j = 0; j < N; ++j) {
        const float x = sum_rows(b < p.nbi && j < n ? v[j] * d - off[j] * dmin : 0.0f);
        if (g == 0 && j < n) ya[small().tok[c0 + i0 + j] * 32 + r] += small().weight[c0 + i0 + j] * x;
    }
}

struct DownBlock { uint32_t c[21]; };

// The down phase of a work-group, item after item; false if a wait was given up.  An item is p.rows rows of y.  Its weights
// do not hang on h: a wave's first blocks are on their way before the waits.
__device__ __forceinline__ bool down_items(const BlockPass &p, int item, int base, int n_list, uint32_t &next, uint32_t &word)
{
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), r = lane & 15, g = lane >> 4;
    const int tiles = (p.rows + 15) / 16, n = p.T * p.k, units = p.nqi * tiles;
    float *const ya_all = (float *)(smem + p.o_red), *const ya = ya_all + wave * p.T * 32;     // [NW][T][32]
    bool first = true;                           // the waits are still to come
    while (item < p.t_down) {
        const int r0 = item * p.rows;
        auto load_down = [&](int v, int lo, int total, DownBlock &x) { // unit v: expert lo + v / units, quad of blocks, tile
            if (v >= total) return;
            const int u = v % units, e = small().entry[lo + v / units] & 1023;
            const int row = min(r0 + u % tiles * 16 + r, p.H - 1), b = min(4 * (u / tiles) + g, p.nbi - 1);
            const uint32_t *const at = (const uint32_t *)(p.down + (((int64_t)e * p.H + row) * p.nbi + b) * 84);
#pragma unroll
            for (int i = 0; i < 5; ++i) {
                const u32x4u q = *(const u32x4u *)(at + 4 * i);
#pragma unroll
                for (int j = 0; j < 4; ++j) x.c[4 * i + j] = q[j];
            }
            x.c[20] = at[20];
        };
        for (int i = lane; i < p.T * 32; i += 64) ya[i] = 0.0f;
        int count = min(p.chunk, n), lo = 0, total = (small().seg[count - 1] + 1) * units;
        DownBlock even, odd;
        if (p.sh) {
            struct Rows { i32x4 w[4]; float scale; };
            auto load_shared = [&](int u, Rows &x) {                   // unit u: tile, block
                if (u >= tiles * p.nbs) return;
                const int row = min(r0 + u % tiles * 16 + r, p.H - 1);
                x.scale = p.down_scale[row];
#pragma unroll
                for (int s = 0; s < 4; ++s) x.w[s] = load_row16(p.sh_down + (int64_t)row * p.ld_down, 256 * (u / tiles) + 64 * s + 16 * g, p.sh);
            };
            Rows x0, x1;
            load_shared(wave, x0);
            load_shared(wave + NW, x1);
            load_down(wave, lo, total, even);
            load_down(wave + NW, lo, total, odd);
            if (first) {
                if (tid == 0) word = wait_for(p.ctl + C_SHARED, (uint32_t)p.t_shared);
                __syncthreads();
                if (!word) return false;
            }
            const int rows_max = min(p.chunk, p.T);
            for (int t0 = 0; t0 < p.T; t0 += rows_max) {
                const int nt = min(rows_max, p.T - t0);
                __syncthreads();
                stage_shared(p, t0, nt);
                __syncthreads();
                const float *const sc = (const float *)(smem + p.o_planes + nt * p.nqs * QUAD);
                auto unit = [&](int u, const Rows &x) {
                    const int tile = u % tiles, b = u / tiles;
                    for (int tg = 0; tg < nt; tg += 4) {
                        const int slot = tg + (r >> 2), digit = r & 3, tt = tg + g;
                        const bool in = digit < 3 && slot < nt;
                        const int8_t *const a =
                            digit_base(p, in, slot, p.nqs * QUAD, (b >> 2) * QUAD + g * 192 + ((b & 3) * 3 + digit) * 16);
                        i32x4 acc = {0, 0, 0, 0};
#pragma unroll
                        for (int s = 0; s < 4; ++s) acc = mfma_i8(*(const i32x4 *)(a + s * 768), x.w[s], acc);
                        if (tt < nt) ya[(t0 + tt) * 32 + tile * 16 + r] += joined(acc) * (sc[tt * 4 * p.nqs + b] * x.scale);
                    }
                };
                if (t0) {
                    load_shared(wave, x0);
                    load_shared(wave + NW, x1);
                }
                for (int u = wave; u < tiles * p.nbs; u += 2 * NW) {
                    unit(u, x0);
                    load_shared(u + 2 * NW, x0);
                    if (u + NW < tiles * p.nbs) unit(u + NW, x1);
                    load_shared(u + 3 * NW, x1);
                }
            }
        } else {
            load_down(wave, lo, total, even);
            load_down(wave + NW, lo, total, odd);
        }
        for (int c0 = 0; c0 < n; c0 += p.chunk) {
            if (c0) {
                count = min(p.chunk, n - c0);
                lo = small().seg[c0];
                total = (small().seg[c0 + count - 1] + 1 - lo) * units;
                load_down(wave, lo, total, even);
                load_down(wave + NW, lo, total, odd);
            }
            if (first) {
                if (tid == 0) word = wait_for(p.ctl + C_ROUTED, (uint32_t)(n_list * p.nf));
                __syncthreads();
                if (!word) return false;
                first = false;
            }
            __syncthreads();
            stage_h(p, c0, count);
            __syncthreads();
            // a unit's blocks are requested two units ahead
            auto unit = [&](int v, DownBlock &x) {
                const DownBlock now = x;
                load_down(v + 2 * NW, lo, total, x);
                const int u = v % units, tile = u % tiles, quad = u / tiles, entry = small().entry[lo + v / units];
                const int begin = max(entry >> 10 & 1023, c0), end = min((entry >> 10 & 1023) + (entry >> 20), c0 + count);
                for (int j = begin; j < end; j += 2) {
                    if (end - j == 1) down_rows<1>(p, now.c, c0, j - c0, 1, quad, ya + tile * 16);
                    else down_rows<2>(p, now.c, c0, j - c0, 2, quad, ya + tile * 16);
                }
            };
            for (int v = wave; v < total; v += 2 * NW) {
                unit(v, even);
                if (v + NW < total) unit(v + NW, odd);
            }
        }
        __syncthreads();
        if (tid == 0) next = draw(p.ctl);
        for (int i = tid; i < p.T * p.rows; i += NT) {
            const int t = i / p.rows, row = i % p.rows;
            if (r0 + row >= p.H) continue;
            float v = ya_all[t * 32 + row];
            for (int w = 1; w < NW; ++w) v += ya_all[(w * p.T + t) * 32 + row];
            if (p.sh && p.down_bias) v += p.down_bias[r0 + row];
            p.y[(int64_t)t * p.ldy + r0 + row] = v;
            if (p.sum) {
                const int64_t from = (int64_t)t * p.H + r0 + row, to = (int64_t)t * p.ldsum + r0 + row;
                if (p.res_bf16) ((uint16_t *)p.sum)[to] = ((const uint16_t *)p.s)[from];
                else ((float *)p.sum)[to] = ((const float *)p.s)[from];
            }
        }
        __syncthreads();
        item = (int)next - base;
        __syncthreads();                         // and the sums are read
        if (item < 0) return false;
    }
    return true;
}

// the codewords, 16 copies (a lane reads copy lane % 16: no two of 16 lanes share a bank), and the zeros
__device__ __noinline__ void tables(Args pa)
{
    const BlockPass &p = args_of(pa);
    static_assert(NT == 512, "two threads a codeword");
    const int i = threadIdx.x >> 1;
    const uint2 c = *(const uint2 *)(p.codebook + 8 * i);
    const u32x4 two = {c.x, c.y, c.x, c.y};
#pragma unroll
    for (int j = 0; j < 4; ++j) *(u32x4 *)(smem + 128 * i + 64 * (threadIdx.x & 1) + 16 * j) = two;
    for (int i = threadIdx.x; i < QUAD / 4; i += NT) ((uint32_t *)(smem + O_ZERO))[i] = 0;
}

__device__ __noinline__ void give_up(Args pa)
{
    const BlockPass &p = args_of(pa);
    for (int i = threadIdx.x; i < p.T * p.H; i += NT) p.y[(int64_t)(i / p.H) * p.ldy + i % p.H] = __uint_as_float(0x7fc00000u);
}

// the list into LDS
__device__ __noinline__ void load_list(Args pa, int n_list)
{
    const BlockPass &p = args_of(pa);
    const int tid = threadIdx.x, n = p.T * p.k;
    Small &l = small();
    // in bounds whatever another call may have left there
    int e = 0, first = 0, count = 0;
    if (tid < n_list) {
        const int entry = peek(p.list + tid);
        e = min(entry & 1023, p.E - 1);
        first = min(entry >> 10 & 1023, n - 1);
        count = min(entry >> 20 & 31, n - first);
        l.entry[tid] = e | first << 10 | count << 20;
    }
    if (tid < n) {
        l.tok[tid] = (int16_t)min(max(peek(p.list + 256 + tid), 0), p.T - 1);
        l.weight[tid] = peek((const float *)p.list + 512 + tid);
        l.seg[tid] = 0;
    }
    __syncthreads();
    for (int i = 0; i < count; ++i) l.seg[first + i] = (int16_t)tid;
    __syncthreads();
}

__global__ __launch_bounds__(NT) void block_kernel(BlockPass p)
{
    __shared__ uint32_t next, word;
    const int tid = threadIdx.x;
    const uint64_t at = (uint64_t)__builtin_amdgcn_kernarg_segment_ptr();
    const Args pa{(uint32_t)at, (uint32_t)(at >> 32)};
    uint32_t *const ctl = p.ctl;
    if (tid == 0) next = draw(ctl);
    tables(pa);
    bool resident = false;                       // all tokens' digits are in LDS
    int item;
    for (;;) {
        __syncthreads();
        item = (int)next;
        __syncthreads();
        if (item == 0) {
            if (p.E <= 256) select<4>(pa);
            else select<8>(pa);
            if (tid == 0) next = draw(ctl);
            continue;
        }
        item -= 1;
        if (item < p.t_shared) {
            for (int t0 = 0; t0 < p.T; t0 += p.slots) {
                const int nt = min(p.slots, p.T - t0);
                if (!resident) {
                    __syncthreads();
                    stage_tokens(pa, t0, nullptr, nt);
                    resident = p.T <= p.slots;
                    __syncthreads();
                }
                shared_item(pa, item, t0, nt);
            }
            arrive(ctl, C_SHARED, next);
            continue;
        }
        break;
    }
    // the rest is inlined: it needs all registers, and would save and restore them at every call
    item -= p.t_shared;
    if (!resident && p.T <= p.slots) stage_tokens(pa, 0, nullptr, p.T);
    if (tid == 0) word = wait_for(ctl + C_LIST, 1) ? peek(ctl + C_LIST) : 0;
    __syncthreads();
    const int n_list = min((int)word, p.T * p.k), n_routed = n_list * p.nf;
    if (n_list <= 0) {
        give_up(pa);
        return;
    }
    load_list(pa, n_list);
    while (item >= 0 && item < n_routed) {       // a negative one: the counters are another call's
        routed_item(p, pa, item);
        arrive(ctl, C_ROUTED, next);
        __syncthreads();
        item = (int)next - 1 - p.t_shared;
        __syncthreads();
    }
    if (item < 0 || !down_items(p, item - n_routed, 1 + p.t_shared + n_routed, n_list, next, word)) give_up(pa);
}

}  // namespace

void block_layout(BlockPass &p)
{
    auto up = [](int v, int to) { return (v + to - 1) / to; };
    p.nb = up(p.H, 256); p.nq = up(p.nb, 4);
    p.nbi = up(p.I, 256); p.nqi = up(p.nbi, 4);
    p.nbs = up(p.sh, 256); p.nqs = up(p.nbs, 4);
    // an item's units are F / 16 * nq, for eight waves: of wide rows 64 features are enough (7168: one token 55 us and four 130, with
    // 128 features 62 and 129, eight 236 and 226), of narrow ones 128 (sixteen tokens of 2048: 101 us, with 64 features 104)
    p.F = p.nq >= 4 ? 64 : 128;
    p.nf = up(p.I, p.F);
    p.records = p.nf * p.F / 64;
    const int cus = cu_count();
    p.rows = std::min(32, std::max(16, up(p.H, cus)));
    p.experts = std::max(1, up(p.E * p.T, 256));
    p.t_shared = up(p.sh, 8);
    p.t_down = up(p.H, p.rows);
    // four tokens' digits are the 16 rows of an instruction, and at 8192 features all of the LDS that is left (with two tokens, four of
    // 7168 take 143 us, not 130, and sixteen of 2048 112, not 101)
    p.slots = std::min(p.T, 4);
    // LDS: table, zeros, planes (or rows of h), scales, sums
    const int units = p.F / 16 * p.nq;
    const int sums = std::max({units * std::min(p.slots, 2) * 128, NW * 64 * 4, NW * p.T * 128});
    const int red = sums + NW * REC;             // and the waves' records
    const int scales = p.slots * 4 * p.nq * 4;
    const int row_i = p.nqi * 4 * REC_BLOCK, row_s = p.nqs * (QUAD + 16), row = std::max(row_i, row_s);
    constexpr int LDS = 160 * 1024 - 256;        // the static shared memory is apart
    const int want = std::max({p.slots * p.nq * QUAD + scales, std::min(16, p.T * p.k) * row, p.T * p.E * 8});
    const int room = LDS - O_END - red;
    const int area = std::min(want, room) / 16 * 16;
    p.chunk = std::min(area / row, p.T * p.k);
    p.o_planes = O_END;
    p.o_scales = O_END + p.slots * p.nq * QUAD;
    p.o_red = O_END + area;
    p.o_recs = p.o_red + sums;
    p.lds = O_END + area + red;
}

// Every piece begins on cache lines of its own, so from a multiple of 256 on, wherever the caller's workspace begins: h is
// read with plain loads, and a line that holds anything a work-group has read earlier would come from its cache.  Returns the
// bytes from `base` on.
size_t block_workspace(BlockPass &p, char *base)
{
    const size_t gap = -(uintptr_t)base & 255;
    base += gap;
    size_t off = 0;
    auto take = [&](size_t bytes) {
        char *at = base + off;
        off = (off + bytes + 255) / 256 * 256;
        return (void *)at;
    };
    p.ctl = (uint32_t *)take(C_WORDS * 4);
    p.list = (int32_t *)take(768 * 4);
    p.logits = (double *)take((size_t)p.T * p.E * 8);
    p.s = take((size_t)p.T * p.H * 4);
    p.planes = (int8_t *)take((size_t)p.T * p.nq * QUAD);
    p.scales = (float *)take((size_t)p.T * 4 * p.nq * 4);
    p.h = (int8_t *)take((size_t)p.T * p.k * p.records * REC_LINES);
    p.hs = (float *)take((size_t)p.T * p.sh * 4);
    return gap + off;
}

hipError_t launch_block_norm(const BlockPass &p, hipStream_t s)
{
    block_norm<<<dim3((unsigned)p.T, (unsigned)((p.E + p.experts - 1) / p.experts)), NORM_NT, 0, s>>>(p);
    return hipGetLastError();
}

hipError_t launch_block(const BlockPass &p, hipStream_t s)
{
    const unsigned grid = (unsigned)cu_count();  // one work-group's LDS fills a CU
    static DevSlots slots{};
    const hipError_t e = lds_limit((const void *)block_kernel, slots, p.lds);
    if (e != hipSuccess) return e;
    block_kernel<<<grid, NT, p.lds, s>>>(p);
    return hipGetLastError();
}

}  // namespace moe
