// int8 linear layer on gfx950: y = (x w^T) * (xs ws^T) + bias + add, with the
// integer product on the int8 matrix instructions (exact int32 sums).
#include "common.h"
#include "devcache.h"
#include "linear.h"

#include <algorithm>

// the products with the scales, the bias and the addition each round to fp32, in
// every kernel alike: no fma of two of them
#pragma clang fp contract(off)

namespace moe {

namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ uint32_t to_bf16(float f) { return __builtin_bit_cast(uint16_t, (__bf16)f); }

// zeroes the bytes of a 16-byte piece that lie at or past column K (the piece
// starts at column k < K)
__device__ __forceinline__ i32x4 mask_tail(i32x4 v, int k, int K)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int left = K - (k + 4 * i);
        v[i] = left >= 4 ? v[i] : left <= 0 ? 0 : v[i] & (int)((1u << (8 * left)) - 1u);
    }
    return v;
}

// Scales and bias of channels n .. n + CNT (0 past N), loaded once per lane.
template <int CNT>
struct Channels {
    float scale[CNT], bias[CNT];
    bool wide;                                   // all CNT channels exist
    __device__ __forceinline__ Channels(const LinearPass &p, int n)
    {
        wide = n + CNT <= p.N;
        if (wide && (uintptr_t)(p.w_scale + n) % 16 == 0 && (uintptr_t)(p.bias + n) % 16 == 0) {
#pragma unroll
            for (int i = 0; i < CNT; i += 4) {
                const f32x4 w = *(const f32x4 *)(p.w_scale + n + i);
                const f32x4 b = p.bias ? *(const f32x4 *)(p.bias + n + i) : f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int j = 0; j < 4; ++j) { scale[i + j] = w[j]; bias[i + j] = b[j]; }
            }
        } else {
#pragma unroll
            for (int i = 0; i < CNT; ++i) {
                scale[i] = n + i < p.N ? p.w_scale[n + i] : 0.0f;
                bias[i] = p.bias && n + i < p.N ? p.bias[n + i] : 0.0f;
            }
        }
    }
};

// y[t][n .. n + CNT) from the integer sums of one lane; wide accesses where
// the lane's channels are all there and aligned
template <int CNT>
__device__ __forceinline__ void finish(const LinearPass &p, int t, int n, const Channels<CNT> &c, const int acc[CNT])
{
    if (t >= p.T || n >= p.N) return;
    const float xs = p.x_scale[t];
    float v[CNT];
#pragma unroll
    for (int i = 0; i < CNT; ++i) {
        v[i] = (float)acc[i] * (xs * c.scale[i]);
        if (p.bias) v[i] += c.bias[i];
    }
    const int size = p.y_bf16 ? 2 : 4;
    char *const y = (char *)p.y + ((int64_t)t * p.ldy + n) * size;
    const char *const add = (const char *)p.add + ((int64_t)t * p.ldadd + n) * size;
    constexpr int PIECE = CNT >= 8 ? 8 : 4;      // channels of an access
    const uintptr_t at = (uintptr_t)y | (p.add ? (uintptr_t)add : 0);
    if (c.wide && at % (p.y_bf16 ? 2 * PIECE : 16) == 0) {
#pragma unroll
        for (int i = 0; i < CNT; i += PIECE) {
            if (p.y_bf16) {
                uint32_t u[PIECE / 2];
                if (p.add) __builtin_memcpy(u, __builtin_assume_aligned(add + 2 * i, 2 * PIECE), 2 * PIECE);
#pragma unroll
                for (int j = 0; j < PIECE; j += 2) {
                    float lo = v[i + j], hi = v[i + j + 1];
                    if (p.add) {
                        lo += __uint_as_float(u[j / 2] << 16);
                        hi += __uint_as_float(u[j / 2] & 0xffff0000u);
                    }
                    u[j / 2] = to_bf16(lo) | (to_bf16(hi) << 16);
                }
                __builtin_memcpy(__builtin_assume_aligned(y + 2 * i, 2 * PIECE), u, 2 * PIECE);
            } else {
#pragma unroll
                for (int j = 0; j < PIECE; j += 4) {
                    f32x4 o = {v[i + j], v[i + j + 1], v[i + j + 2], v[i + j + 3]};
                    if (p.add) o += *(const f32x4 *)(add + 4 * (i + j));
                    *(f32x4 *)(y + 4 * (i + j)) = o;
                }
            }
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < CNT; ++i) {
        if (n + i < p.N) {
            float o = v[i];
            if (p.add) o += p.y_bf16 ? bf16_bits_to_f32(((const uint16_t *)add)[i]) : ((const float *)add)[i];
            if (p.y_bf16) ((uint16_t *)y)[i] = (uint16_t)to_bf16(o);
            else ((float *)y)[i] = o;
        }
    }
}

// The same for 16 tokens x 16 FA channels of a wave whose rows of y (or add) are
// not aligned for wide accesses: through LDS (buf: this wave's, 16 (16 FA + 1)
// floats), so that the lanes of a store hold neighbouring channels of a token.
// acc: the lane's 4 FA channels, from 4 FA fg on, of token fr.  4118 x 2211 x
// 968: 34 us, and 67 with each lane storing its own channels.
template <int FA>
__device__ __forceinline__ void finish_odd(const LinearPass &p, int t0, int n0, int fr, int fg, const Channels<4 * FA> &c,
                                           const int acc[4 * FA], float *buf)
{
    constexpr int W = 16 * FA, LD = W + 1;
    const float xs = p.x_scale[min(t0 + fr, p.T - 1)];
#pragma unroll
    for (int i = 0; i < 4 * FA; ++i) {
        float v = (float)acc[i] * (xs * c.scale[i]);
        if (p.bias) v += c.bias[i];
        buf[fr * LD + 4 * FA * fg + i] = v;
    }
    asm volatile("" ::: "memory");               // one wave: its LDS operations run in order
    const int lane = 16 * fg + fr, ch = lane % W, n = n0 + ch;
#pragma unroll 1                                 // small: the callers' loops over fragments have to unroll
    for (int i = 0; i < 16; i += 64 / W) {
        const int r = i + lane / W, t = t0 + r;
        if (t < p.T && n < p.N) {
            float v = buf[r * LD + ch];
            const int64_t at = (int64_t)t * p.ldadd + n;
            if (p.add) v += p.y_bf16 ? bf16_bits_to_f32(((const uint16_t *)p.add)[at]) : ((const float *)p.add)[at];
            const int64_t yt = (int64_t)t * p.ldy + n;
            if (p.y_bf16) ((uint16_t *)p.y)[yt] = (uint16_t)to_bf16(v);
            else ((float *)p.y)[yt] = v;
        }
    }
    asm volatile("" ::: "memory");
}

// whether rows of y and add start on 16 bytes
__device__ __forceinline__ bool wide_rows(const LinearPass &p)
{
    const int size = p.y_bf16 ? 2 : 4;
    uintptr_t a = (uintptr_t)p.y | (uintptr_t)(p.ldy * size);
    if (p.add) a |= (uintptr_t)p.add | (uintptr_t)(p.ldadd * size);
    return a % 16 == 0;
}

constexpr int BK = 128;                          // bytes of K per step: eight 16-byte chunks of a row

// Order of the work-groups over the tiles: work-group b runs on XCD b % 8 (each
// has its own L2), which gets a contiguous run of tiles, ordered in stripes of
// 4 token tiles so that what runs at once shares x and w rows.
__device__ __forceinline__ void tile_of(int b, int nt, int nn, int &tt, int &tn)
{
    const int total = nt * nn, per = total / 8, more = total % 8;
    const int xcd = b % 8;
    int i = b / 8 + xcd * per + min(xcd, more);  // XCDs 0 .. more - 1 take one tile more
    const int stripe = i / (4 * nn), rows = min(4, nt - 4 * stripe);
    i -= stripe * 4 * nn;
    tt = 4 * stripe + i % rows;
    tn = i / rows;
}

// wait until at most `vm` of this wave's loads are in flight (and, with lgkm 0,
// its LDS reads have landed), then the work-group's barrier; nothing moves across
template <int VM, int LGKM, bool STRICT = true>
__device__ __forceinline__ void sync_waves()
{
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt((VM & 15) | 0x70 | (LGKM << 8) | ((VM >> 4) << 14));
    if (STRICT) __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_barrier();
    if (STRICT) __builtin_amdgcn_sched_barrier(0);
    asm volatile("" ::: "memory");
}
constexpr int VM_ANY = 63, LGKM_ANY = 15;

// int32 sums of one part of K: ws[part][T][N]
template <int CNT>
__device__ __forceinline__ void store_part(const LinearPass &p, int part, int t, int n, const int acc[CNT])
{
    if (t >= p.T || n >= p.N) return;
    int *const o = (int *)p.ws + ((int64_t)part * p.T + t) * p.N + n;
    if (n + CNT <= p.N && p.N % 4 == 0) {
#pragma unroll
        for (int i = 0; i < CNT; i += 4) *(i32x4 *)(o + i) = i32x4{acc[i], acc[i + 1], acc[i + 2], acc[i + 3]};
    } else {
#pragma unroll
        for (int i = 0; i < CNT; ++i)
            if (n + i < p.N) o[i] = acc[i];
    }
}

// adds the parts (integers: in any order) and finishes, 4 channels a thread
__global__ __launch_bounds__(256) void linear_join(LinearPass p, int parts)
{
    const int per = (p.N + 3) / 4;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= (int64_t)p.T * per) return;
    const int t = (int)(i / per), n = (int)(i % per) * 4;
    const int *in = (const int *)p.ws + (int64_t)t * p.N + n;
    const int64_t stride = (int64_t)p.T * p.N;
    int acc[4] = {0, 0, 0, 0};
    for (int c = 0; c < parts; ++c, in += stride) {
        if (p.N % 4 == 0) {
            const i32x4 v = *(const i32x4 *)in;
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[j] += v[j];
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[j] += in[min(j, p.N - 1 - n)];
        }
    }
    finish<4>(p, t, n, Channels<4>(p, n), acc);
}

// Tile kernel: BM = 16 FB WB tokens x BN = 16 FA WA channels, WA x WB waves of
// 16 FA channels x 16 FB tokens each, K in steps of 128 through a ring of LDS
// buffers that the loads write without passing registers, RING - 1 steps ahead.
// One barrier a step: after it, every wave has read the oldest buffer, which
// the next loads then fill.  The deeper rings are for the small tiles, whose
// products are shorter than a load's latency (64 x 4096 x 7168 in one part: 42.7
// us with two buffers, 21 with four).
//
// A row's eight chunks lie in LDS at chunk ^ key(row), so that the lanes that
// read the same chunk of 8 neighbouring rows of a fragment hit 8 different
// 16-byte columns.  The loads write 64 consecutive chunks, 8 rows; the
// permutation is in which chunk of its row a lane fetches.  Row i of channel
// fragment f is channel 4 FA (i / 4) + 4 f + i % 4, so that a lane ends with 4 FA
// consecutive channels of a token.
template <int FA, int FB, int WA, int WB, int RING>
struct Tile {
    static constexpr int BN = 16 * FA * WA, BM = 16 * FB * WB, NW = WA * WB, NT = 64 * NW;
    static constexpr int XB = BM * BK, WBYTES = BN * BK, SLOT = XB + WBYTES, LDS = RING * SLOT;
    static constexpr int LX = BM / 8 / NW, LW = BN / 8 / NW;   // loads of a wave in a step
    static constexpr int SH = FA == 4 ? 4 : 3;                 // log2(4 FA)
    static_assert(4 * FA == 1 << SH, "four or two fragments");
    static_assert(LX * 8 * NW == BM && LW * 8 * NW == BN, "whole loads");
    static __device__ __forceinline__ int xkey(int r) { return r & 7; }
    static __device__ __forceinline__ int wkey(int r) { return (r & 3) | (((r >> SH) & 1) << 2); }
};

template <int FA, int FB, int WA, int WB, int RING>
__global__ __launch_bounds__(64 * WA * WB, 2) void linear_tile(LinearPass p, int parts)
{
    using C = Tile<FA, FB, WA, WB, RING>;
    extern __shared__ __align__(16) int8_t lds[];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int fr = lane & 15, fg = lane >> 4;
    int tt, tn;
    tile_of(blockIdx.x / parts, (p.T + C::BM - 1) / C::BM, (p.N + C::BN - 1) / C::BN, tt, tn);
    // this part's steps; the last part also takes the last K % 128 bytes
    const int part = blockIdx.x % parts, all = p.K / BK, kb = (int)((int64_t)all * part / parts);
    const int steps = (int)((int64_t)all * (part + 1) / parts) - kb;
    const int t0 = tt * C::BM, n0 = tn * C::BN;

    // the wave's loads: LX x 8 token rows, then LW x 8 channel rows
    const int8_t *xp[C::LX], *wp[C::LW];
    const int lr = lane >> 3, lc = lane & 7;
#pragma unroll
    for (int i = 0; i < C::LX; ++i) {
        const int r = (wave * C::LX + i) * 8 + lr;
        xp[i] = p.x + (int64_t)min(t0 + r, p.T - 1) * p.ldx + 16 * (lc ^ C::xkey(r)) + (int64_t)kb * BK;
    }
#pragma unroll
    for (int i = 0; i < C::LW; ++i) {
        const int r = (wave * C::LW + i) * 8 + lr;
        wp[i] = p.w + (int64_t)min(n0 + r, p.N - 1) * p.ldw + 16 * (lc ^ C::wkey(r)) + (int64_t)kb * BK;
    }
    auto slot = [&](int k) { return lds + (RING == 3 ? k % 3 : k & (RING - 1)) * C::SLOT; };
    auto fetch = [&](int k) {
        int8_t *const buf = slot(k);
        const int64_t at = (int64_t)min(k, steps - 1) * BK;    // past the end: the last step again, into a slot that nobody reads
#pragma unroll
        for (int i = 0; i < C::LX; ++i)
            __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)(xp[i] + at),
                                             (__attribute__((address_space(3))) void *)(buf + (wave * C::LX + i) * 1024), 16, 0, 0);
#pragma unroll
        for (int i = 0; i < C::LW; ++i)
            __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)(wp[i] + at),
                                             (__attribute__((address_space(3))) void *)(buf + C::XB + (wave * C::LW + i) * 1024), 16, 0, 0);
    };
    // the rows this lane reads as fragments
    const int wa = wave % WA, wb = wave / WA;
    int xo[FB], wo[FA];
#pragma unroll
    for (int j = 0; j < FB; ++j) xo[j] = wb * 16 * FB + 16 * j + fr;
#pragma unroll
    for (int i = 0; i < FA; ++i) wo[i] = wa * 16 * FA + 4 * FA * (fr >> 2) + 4 * i + (fr & 3);

    i32x4 acc[FA][FB];
#pragma unroll
    for (int i = 0; i < FA; ++i)
#pragma unroll
        for (int j = 0; j < FB; ++j) acc[i][j] = i32x4{0, 0, 0, 0};
    auto products = [&](const int8_t *buf) {
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
            i32x4 a[FA], b[FB];
#pragma unroll
            for (int i = 0; i < FA; ++i)
                a[i] = *(const i32x4 *)(buf + C::XB + wo[i] * BK + 16 * ((4 * kk + fg) ^ C::wkey(wo[i])));
#pragma unroll
            for (int j = 0; j < FB; ++j) b[j] = *(const i32x4 *)(buf + xo[j] * BK + 16 * ((4 * kk + fg) ^ C::xkey(xo[j])));
#pragma unroll
            for (int j = 0; j < FB; ++j)
#pragma unroll
                for (int i = 0; i < FA; ++i) acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(a[i], b[j], acc[i][j], 0, 0, 0);
        }
    };

    if (steps) {
#pragma unroll
        for (int k = 0; k < RING - 1; ++k) fetch(k);
    }
    for (int k = 0; k < steps; ++k) {
        sync_waves<(RING - 2) * (C::LX + C::LW), 0, false>();  // step k has landed for everybody, and step k - 1 is read
        fetch(k + RING - 1);
        products(slot(k));
    }
    sync_waves<0, 0, false>();                   // no load may be in flight when the LDS is reused or freed
    const int k0 = all * BK;
    if (part == parts - 1 && k0 < p.K) {                              // the last K % 128 bytes, masked, through registers
#pragma unroll
        for (int i = 0; i < C::LX; ++i) {
            const int r = (wave * C::LX + i) * 8 + lr, k = k0 + 16 * (lc ^ C::xkey(r));
            i32x4 v = {0, 0, 0, 0};
            if (k < p.K) v = mask_tail(*(const i32x4 *)(xp[i] + (int64_t)steps * BK), k, p.K);
            *(i32x4 *)(lds + r * BK + 16 * lc) = v;
        }
#pragma unroll
        for (int i = 0; i < C::LW; ++i) {
            const int r = (wave * C::LW + i) * 8 + lr, k = k0 + 16 * (lc ^ C::wkey(r));
            i32x4 v = {0, 0, 0, 0};
            if (k < p.K) v = *(const i32x4 *)(wp[i] + (int64_t)steps * BK);
            *(i32x4 *)(lds + C::XB + r * BK + 16 * lc) = v;
        }
        __syncthreads();
        products(lds);
    }
    // D: lane (fr, fg) of fragment (i, j) holds rows 4 fg .. 4 fg + 3 (channels) of column fr (token)
    const int n = n0 + wa * 16 * FA + 4 * FA * fg;
    const Channels<4 * FA> chan(p, n);
    const bool odd = parts == 1 && !wide_rows(p);
    if (odd) __syncthreads();                    // the LDS is read
#pragma unroll
    for (int j = 0; j < FB; ++j) {
        int v[4 * FA];
#pragma unroll
        for (int i = 0; i < FA; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r) v[4 * i + r] = acc[i][j][r];
        if (odd) finish_odd<FA>(p, t0 + xo[j] - fr, n0 + wa * 16 * FA, fr, fg, chan, v, (float *)lds + wave * 16 * (16 * FA + 1));
        else if (parts == 1) finish<4 * FA>(p, t0 + xo[j], n, chan, v);
        else store_part<4 * FA>(p, part, t0 + xo[j], n, v);
    }
}

// The large tile: 256 tokens x 256 channels, eight waves of 64 channels x 128
// tokens, K in steps of 128 bytes (whole cache lines: 64-byte rows doubled the
// requests to L2 and were slower on the smaller tiles).  The LDS is a ring of
// five units of 32 KB, x and w of a step one each: w of the next step is
// requested at the start of a step and x of the one after it, so that the load
// path, which takes as long as the products, never idles.
//
// The waves of a SIMD alternate: while waves 0-3 run the 32 products of half a
// step, waves 4-7 read the fragments of theirs, and a barrier swaps them.
// Interval 4 k of the loop is waves 0-3 reading the first half of step k.  x and
// w of step k - 1 are read by interval 4 k - 1, so their units are loaded again
// from interval 4 k on; step k + 1 has landed by the barrier that ends interval
// 4 k + 3 (waves 0-3 wait there for all their loads, of w; waves 4-7 for all but
// the newest eight, which are x of step k + 2).
//
// 8192 x 4096 x 7168: 198 us, 2.43 POP/s at 1.84 to 2.02 GHz (a kernel bound by
// memory runs at 2.4), where products alone take 143 us (4.2 POP/s at the clock they
// leave), loads alone 105 us.  Tiles of
// 32x32 products, one wave a SIMD with 128 x 128 outputs, and two buffers of a
// whole step each were slower (239, 368, 222 us).
namespace big {
constexpr int BM = 256, BN = 256, KS = 128, UNIT = 256 * KS, UNITS = 5, LDS = UNITS * UNIT;
constexpr int FA = 4, FB = 8;
__device__ __forceinline__ int xkey(int r) { return r & 7; }
__device__ __forceinline__ int wkey(int r) { return (r & 3) | (((r >> 4) & 1) << 2); }
}

__global__ __launch_bounds__(512) void linear_big(LinearPass p)
{
    using namespace big;
    extern __shared__ __align__(16) int8_t lds[];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int fr = lane & 15, fg = lane >> 4;
    int tt, tn;
    tile_of(blockIdx.x, (p.T + BM - 1) / BM, (p.N + BN - 1) / BN, tt, tn);
    const int t0 = tt * BM, n0 = tn * BN;
    const bool second = wave >= 4;
    const int wa = wave & 3, wb = wave >> 2;

    // waves 0-3 load w, waves 4-7 load x: 64 rows each
    const int8_t *lp[8];
    const int lr = lane >> 3, lc = lane & 7;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int r = wa * 64 + i * 8 + lr;
        lp[i] = second ? p.x + (int64_t)min(t0 + r, p.T - 1) * p.ldx + 16 * (lc ^ xkey(r))
                       : p.w + (int64_t)min(n0 + r, p.N - 1) * p.ldw + 16 * (lc ^ wkey(r));
    }
    const int steps = p.K / KS;
    auto fetch = [&](int unit) {
        int8_t *const buf = lds + unit * UNIT + wa * 8192;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)lp[i],
                                             (__attribute__((address_space(3))) void *)(buf + i * 1024), 16, 0, 0);
            lp[i] += KS;
        }
    };
    const int x0 = wb * 128 + fr, w0 = wa * 64 + 16 * (fr >> 2) + (fr & 3);
    i32x4 acc[FA][FB], fa[FA], fb[FB];
#pragma unroll
    for (int i = 0; i < FA; ++i)
#pragma unroll
        for (int j = 0; j < FB; ++j) acc[i][j] = i32x4{0, 0, 0, 0};
    auto reads = [&](const int8_t *xb, const int8_t *wbuf, int kk) {
#pragma unroll
        for (int i = 0; i < FA; ++i) fa[i] = *(const i32x4 *)(wbuf + (w0 + 4 * i) * KS + 16 * ((4 * kk + fg) ^ wkey(w0 + 4 * i)));
#pragma unroll
        for (int j = 0; j < FB; ++j) fb[j] = *(const i32x4 *)(xb + (x0 + 16 * j) * KS + 16 * ((4 * kk + fg) ^ xkey(x0)));
    };
    auto products = [&]() {
#pragma unroll
        for (int j = 0; j < FB; ++j)
#pragma unroll
            for (int i = 0; i < FA; ++i) acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fa[i], fb[j], acc[i][j], 0, 0, 0);
    };
    auto wrap = [](int u) { return u >= UNITS ? u - UNITS : u; };

    if (steps) {
        if (second) {
            fetch(0);
            if (steps > 1) fetch(2);
            if (steps > 1) sync_waves<8, LGKM_ANY>();
            else sync_waves<0, LGKM_ANY>();
            sync_waves<VM_ANY, LGKM_ANY>();
        } else {
            fetch(1);
            sync_waves<0, LGKM_ANY>();
        }
        int ux = 0;                              // unit of x of this step; w is in the next
        for (int k = 0; k < steps; ++k) {
            const int8_t *xb = lds + ux * UNIT, *wbuf = lds + wrap(ux + 1) * UNIT;
            reads(xb, wbuf, 0);
            __builtin_amdgcn_sched_barrier(0);   // the reads first: requests ahead of them cost 2%
            if (second) { if (k + 2 < steps) fetch(wrap(ux + 4)); }
            else if (k + 1 < steps) fetch(wrap(ux + 3));
            sync_waves<VM_ANY, 0>();
            __builtin_amdgcn_s_setprio(1);
            products();
            __builtin_amdgcn_s_setprio(0);
            sync_waves<VM_ANY, LGKM_ANY>();
            reads(xb, wbuf, 1);
            if (second) {
                if (k + 2 < steps) sync_waves<8, 0>();
                else sync_waves<0, 0>();
            } else sync_waves<VM_ANY, 0>();
            __builtin_amdgcn_s_setprio(1);
            products();
            __builtin_amdgcn_s_setprio(0);
            if (second) sync_waves<VM_ANY, LGKM_ANY>();
            else sync_waves<0, LGKM_ANY>();
            ux = wrap(ux + 2);
        }
        if (!second) sync_waves<VM_ANY, LGKM_ANY>();
    }
    const int k0 = steps * KS;
    if (k0 < p.K) {                              // the last K % 128 bytes, masked, through registers
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int r = wa * 64 + i * 8 + lr, k = k0 + 16 * (lc ^ (second ? xkey(r) : wkey(r)));
            i32x4 v = {0, 0, 0, 0};
            if (k < p.K) {
                v = *(const i32x4 *)lp[i];
                if (second) v = mask_tail(v, k, p.K);
            }
            *(i32x4 *)(lds + (second ? 0 : UNIT) + r * KS + 16 * lc) = v;
        }
        __syncthreads();
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
            reads(lds, lds + UNIT, kk);
            products();
        }
    }
    const int n = n0 + wa * 64 + 16 * fg;
    const Channels<16> chan(p, n);
    const bool odd = !wide_rows(p);
    if (odd) __syncthreads();                    // the LDS is read
#pragma unroll
    for (int j = 0; j < FB; ++j) {
        int v[16];
#pragma unroll
        for (int i = 0; i < FA; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r) v[4 * i + r] = acc[i][j][r];
        if (odd) finish_odd<FA>(p, t0 + x0 - fr + 16 * j, n0 + wa * 64, fr, fg, chan, v, (float *)lds + wave * 16 * 65);
        else finish<16>(p, t0 + x0 + 16 * j, n, chan, v);
    }
}

hipError_t launch_big(const LinearPass &p, hipStream_t s)
{
    static DevSlots slots{};
    const hipError_t e = lds_limit((const void *)linear_big, slots, big::LDS);
    if (e != hipSuccess) return e;
    const int64_t tiles = ((int64_t)p.T + big::BM - 1) / big::BM * (((int64_t)p.N + big::BN - 1) / big::BN);
    linear_big<<<dim3((unsigned)tiles), 512, big::LDS, s>>>(p);
    return hipGetLastError();
}

// Up to 16 tokens: bound by reading w once.  A work-group owns 16 channels; its
// waves split K in slices of 512 bytes and load a slice of w straight into
// registers as matrix operands (a lane's 16 bytes of K are the same for both
// operands, whichever they are), every load of a slice in flight before the
// first product.  The waves' integer sums meet in LDS.  1 x 4096 x 7168: 7.0 us,
// 4.2 TB/s.
constexpr int SLICE = 8;                         // products of 64 bytes of K in a slice

__global__ __launch_bounds__(1024) void linear_stream(LinearPass p)
{
    extern __shared__ __align__(16) int8_t lds[];
    i32x4 *const sums = (i32x4 *)lds;            // [waves][64]
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, nw = blockDim.x >> 6;
    const int fr = lane & 15, fg = lane >> 4;
    const int n0 = blockIdx.x * 16;
    const int8_t *wr = p.w + (int64_t)min(n0 + fr, p.N - 1) * p.ldw + 16 * fg;
    const int8_t *xr = p.x + (int64_t)min(fr, p.T - 1) * p.ldx + 16 * fg;
    i32x4 acc = {0, 0, 0, 0};
    for (int k0 = wave * 64 * SLICE; k0 < p.K; k0 += nw * 64 * SLICE) {
        i32x4 w[SLICE], x[SLICE];
        if (k0 + 64 * SLICE <= p.K) {
#pragma unroll
            for (int s = 0; s < SLICE; ++s) w[s] = *(const i32x4 *)(wr + k0 + 64 * s);
#pragma unroll
            for (int s = 0; s < SLICE; ++s) x[s] = *(const i32x4 *)(xr + k0 + 64 * s);
        } else {
#pragma unroll
            for (int s = 0; s < SLICE; ++s) {
                const int k = k0 + 64 * s + 16 * fg;
                w[s] = x[s] = i32x4{0, 0, 0, 0};
                if (k < p.K) {
                    w[s] = *(const i32x4 *)(wr + k0 + 64 * s);
                    x[s] = mask_tail(*(const i32x4 *)(xr + k0 + 64 * s), k, p.K);
                }
            }
        }
#pragma unroll
        for (int s = 0; s < SLICE; ++s) acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(w[s], x[s], acc, 0, 0, 0);
    }
    if (nw > 1) {
        sums[wave * 64 + lane] = acc;
        __syncthreads();
        if (wave > 0) return;
        for (int v = 1; v < nw; ++v) acc += sums[v * 64 + lane];
    }
    const int v[4] = {acc[0], acc[1], acc[2], acc[3]};
    finish<4>(p, fr, n0 + 4 * fg, Channels<4>(p, n0 + 4 * fg), v);
}

hipError_t launch_stream(const LinearPass &p, hipStream_t s)
{
    const int waves = std::max(1, std::min(16, (p.K + 64 * SLICE - 1) / (64 * SLICE)));
    linear_stream<<<dim3((unsigned)((p.N + 15) / 16)), 64 * waves, waves * 1024, s>>>(p);
    return hipGetLastError();
}

template <int FA, int FB, int WA, int WB, int RING>
hipError_t launch_tile(const LinearPass &p, int parts, hipStream_t s)
{
    using C = Tile<FA, FB, WA, WB, RING>;
    static DevSlots slots{};
    const hipError_t e = lds_limit((const void *)linear_tile<FA, FB, WA, WB, RING>, slots, C::LDS);
    if (e != hipSuccess) return e;
    const int64_t tiles = ((int64_t)p.T + C::BM - 1) / C::BM * (((int64_t)p.N + C::BN - 1) / C::BN);
    linear_tile<FA, FB, WA, WB, RING><<<dim3((unsigned)(tiles * parts)), C::NT, C::LDS, s>>>(p, parts);
    if (parts > 1) linear_join<<<dim3((unsigned)(((int64_t)p.T * ((p.N + 3) / 4) + 255) / 256)), 256, 0, s>>>(p, parts);
    return hipGetLastError();
}

// The kernel for a shape.  Measured costs of a step of 128 bytes of K (us, one
// tile on a CU, and two at once where two fit) and of a tile's start and end;
// the sizes are those of the tiles, the times those of N = 4096 and K = 7168.
// Larger tiles read the operands fewer times, smaller ones fill the 256 CUs and
// lose less at ragged edges: there the variants take, in this order, 91 / 52 / 30 /
// 32 / 45 us for T = 512, 91 / 68 / 86 / 111 us for 2048 and 201 / 250 / 314 / 388 /
// 518 us for 8192.
struct Plan {
    int kernel, parts;                           // kernel: index below, or STREAM
};
constexpr int STREAM = -1;
struct Cost {
    int tokens, channels;
    float one, two, tile;
};
constexpr Cost COSTS[] = {
    {256, 256, 1.50f, 3.00f, 12.0f}, {128, 128, 0.92f, 1.20f, 5.0f}, {128, 64, 0.55f, 0.81f, 4.0f},
    {64, 64, 0.38f, 0.58f, 2.0f},    {32, 64, 0.30f, 0.46f, 1.5f},
};
constexpr int CUS = 256, SPLIT_STEPS = 14;

Plan plan_of(int T, int N, int K)
{
    // up to one fragment of tokens: w streams through registers once (16 x 4096
    // x 7168: 11 us, against 17 of the smallest tile and 13 of it on 4 parts of K)
    if (T <= 16) return {STREAM, 1};
    const int steps = (K + BK - 1) / BK;
    Plan best{0, 1};
    float least = 0.0f;
    for (int i = 0; i < 5; ++i) {
        const Cost &c = COSTS[i];
        const int64_t tiles = ((int64_t)T + c.tokens - 1) / c.tokens * (((int64_t)N + c.channels - 1) / c.channels);
        const float n = (float)((tiles + CUS - 1) / CUS), pairs = (float)(((int64_t)n) / 2);
        const float t = steps * (pairs * c.two + (n - 2 * pairs) * c.one) + n * c.tile;
        if (i == 0 || t < least) {
            least = t;
            best.kernel = i;
        }
    }
    // few tiles and a long K: parts of K of at least 14 steps, joined by a
    // second launch (64 x 4096 x 7168: 14.5 us in 4 parts, 21 in one; in parts
    // of 8 steps the join costs more than it gains)
    const Cost &c = COSTS[best.kernel];
    const int64_t tiles = ((int64_t)T + c.tokens - 1) / c.tokens * (((int64_t)N + c.channels - 1) / c.channels);
    while (best.kernel > 0 && tiles * best.parts * 2 <= CUS && steps / (best.parts * 2) >= SPLIT_STEPS) best.parts *= 2;
    return best;
}

}  // namespace

// A bound of the parts' sums that grows with T, so that a workspace serves every
// smaller batch too, of whichever plan: no more parts than plan_of makes of K, and
// no more than CUS tiles in all of at most 128 x 128.  Past 128 x 128 channels
// every tile row is more than half the CUs: no parts.
size_t linear_ws_bytes(int T, int N, int K)
{
    int parts = 1;
    while ((K + BK - 1) / BK / (parts * 2) >= SPLIT_STEPS) parts *= 2;
    if (T <= 16 || parts == 1 || N > 128 * 128) return 0;
    return std::min<size_t>((size_t)parts * T * N, (size_t)CUS * 128 * 128) * sizeof(int32_t);
}

bool linear_needs_ws(int T, int N, int K) { return plan_of(T, N, K).parts > 1; }

hipError_t launch_linear(const LinearPass &p, hipStream_t s)
{
    const Plan plan = plan_of(p.T, p.N, p.K);
    switch (plan.kernel) {
    case STREAM: return launch_stream(p, s);
    case 0: return launch_big(p, s);
    case 1: return launch_tile<4, 4, 2, 2, 2>(p, plan.parts, s);
    case 2: return launch_tile<2, 4, 2, 2, 3>(p, plan.parts, s);
    case 3: return launch_tile<2, 2, 2, 2, 4>(p, plan.parts, s);
    default: return launch_tile<2, 1, 2, 2, 4>(p, plan.parts, s);
    }
}

}  // namespace moe
