// Row kernels on gfx950: the residual's addition with the root-mean-square
// norm, and rows to int8 codes with a scale each (optionally through SwiGLU).
//
//   norm:   s = round(x + res);  v = (s * r) * g,  r = 1 / sqrt(mean s^2 + eps)
//   swiglu: v = gate / (1 + exp(-gate)) * up
//   codes:  amax = max |v|;  q = rint(v * (127 / amax));  scale = amax / 127
//
// Bound by memory: every input is read once and every output written once.  A
// work-group owns one row and keeps it in registers (fp32) between the sum,
// the maximum and the outputs, so the row is never read again.  The mean of
// squares is an fp64 sum: the scale r then does not depend on the order of
// the sum (but for the rare tie of its one rounding to fp32), and no code
// next to a rounding border does.  The maximum is an integer maximum over the
// magnitudes' bits, which an infinity or a NaN wins, so a row that holds one is seen.
//
// 8192 x 7168, fp32 x + bf16 residual to sum, bf16 and codes: 114 us, 5.7 TB/s (a
// 1 GiB copy runs at 4.8 TB/s: the norm reads more than it writes).  8192 x 2048
// SwiGLU from bf16: 17 us, 4.9 TB/s.  One row: 4.3 us and 2.3 us, latency.
//
// Rows that are not aligned go element by element: 227 us and 31 us for the same
// two.  The longest rows do not fit the registers, and what is over goes through
// scratch memory: the norm past 32768 (1024 x 65536: 470 us, 1.6 TB/s; a few
// registers from 16384 on, 2048 x 32768: 164 us, 4.5 TB/s) and unaligned rows past
// 16384 (norm) or 32768 (1024 x 65536: norm 846 us, codes 124 us).
#include "common.h"
#include "rows.h"

namespace moe {

namespace {

__device__ __forceinline__ uint32_t to_bf16(float f) { return __builtin_bit_cast(uint16_t, (__bf16)f); }

// 8 consecutive elements starting at p + c (VEC), or elements c, c + step, ..
// below n (the others are zero)
template <bool VEC>
__device__ __forceinline__ void load8(const void *p, int bf16, int c, int step, int n, float v[8])
{
    if (VEC) {
        if (c >= n) {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = 0.0f;
        } else if (bf16) {
            const u32x4 u = *(const u32x4 *)((const uint16_t *)p + c);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[2 * j] = __uint_as_float(u[j] << 16);
                v[2 * j + 1] = __uint_as_float(u[j] & 0xffff0000u);
            }
        } else {
            const f32x4 a = *(const f32x4 *)((const float *)p + c), b = *(const f32x4 *)((const float *)p + c + 4);
#pragma unroll
            for (int j = 0; j < 4; ++j) { v[j] = a[j]; v[4 + j] = b[j]; }
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int e = c + j * step;
            v[j] = e >= n ? 0.0f : bf16 ? bf16_bits_to_f32(((const uint16_t *)p)[e]) : ((const float *)p)[e];
        }
    }
}

template <bool VEC>
__device__ __forceinline__ void store8(void *p, int bf16, int c, int step, int n, const float v[8])
{
    if (VEC) {
        if (c >= n) return;
        if (bf16) {
            u32x4 u;
#pragma unroll
            for (int j = 0; j < 4; ++j) u[j] = to_bf16(v[2 * j]) | (to_bf16(v[2 * j + 1]) << 16);
            *(u32x4 *)((uint16_t *)p + c) = u;
        } else {
            *(f32x4 *)((float *)p + c) = f32x4{v[0], v[1], v[2], v[3]};
            *(f32x4 *)((float *)p + c + 4) = f32x4{v[4], v[5], v[6], v[7]};
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int e = c + j * step;
            if (e >= n) break;
            if (bf16) ((uint16_t *)p)[e] = (uint16_t)to_bf16(v[j]);
            else ((float *)p)[e] = v[j];
        }
    }
}

// silu(a) * u.  exp(-a) = 2^p (1 + t ln 2) with p = -a log2 e rounded and t what
// its rounding and log2 e's lost, and the quotient is a times a reciprocal after
// one Newton step: off by at most 7 half units in the last place (3 of the
// exponential, the sum, the reciprocal and two products), in half the
// instructions of expf and a division (8192 x 2048: 22 us with those, bound by
// arithmetic).  Past p = 125 the 1 of the sum is below its last place: it is left
// out, the exponential is taken 2^120 smaller (p - 120 is exact) and u too, so that
// all stays normal; and from a = -170.5 on silu is below 2^-238, which with the
// largest u is below half a code of any row that has codes: zero there.  The
// exponential's argument stops at 170.5 either way (silu(a) is a by then).  FAR:
// whether a may be below SILU_FAR; otherwise the same without these cases (8192 x
// 2048: 17 us, and 20 with them).
constexpr float SILU_FAR = -86.6f;               // p = 124.9

template <bool FAR>
__device__ __forceinline__ float silu_mul(float a, float u)
{
#pragma clang fp contract(off)                   // t is what p's own rounding lost
    constexpr float L = 1.44269502f, L_REST = 1.92596303e-8f, LN2 = 0.693147182f;   // log2 e in two parts, ln 2
    const float b = __builtin_amdgcn_fmed3f(-a, -170.5f, 170.5f), p = b * L;
    const float t = fmaf(b, L_REST, fmaf(b, L, -p));
    const bool far = FAR && p > 125.0f;
    float e = __builtin_amdgcn_exp2f(far ? p - 120.0f : p);
    e = fmaf(e, t * LN2, e);
    const float d = far ? e : 1.0f + e;
    float r = __builtin_amdgcn_rcpf(d);
    r = fmaf(fmaf(-d, r, 1.0f), r, r);
    return a * r * (FAR && a <= -170.5f ? u * 0.0f : far ? u * 0x1p-120f : u);
}

// rint(v * inv), |v * inv| < 2^22, in the low bits: the sum's spacing is 1
__device__ __forceinline__ uint32_t code_bits(float v, float inv)
{
    float x = v * inv;
    asm("" : "+v"(x));                          // the product is rounded before the sum: no fma of the two
    return __float_as_uint(x + 12582912.0f);
}

// the low bytes of four dwords
__device__ __forceinline__ uint32_t low_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d)
{
    return __builtin_amdgcn_perm(__builtin_amdgcn_perm(d, c, 0x0c0c0400u), __builtin_amdgcn_perm(b, a, 0x0c0c0400u), 0x05040100u);
}

__device__ __forceinline__ const void *row_of(const void *p, int bf16, int64_t ld, int t)
{
    return (const char *)p + (int64_t)t * ld * (bf16 ? 2 : 4);
}

// NT threads, NV groups of 8 elements each (NT * NV * 8 >= n)
template <int MODE, int NT, int NV, bool VEC>
__global__ __launch_bounds__(NT) void rows_kernel(RowsPass p)
{
    constexpr int NW = NT / 64;
    __shared__ double part[NW];
    __shared__ uint32_t pmax[NW];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int t = blockIdx.x, n = p.n;
    const int step = VEC ? 1 : NT;
    auto col = [&](int i) { return VEC ? (i * NT + tid) * 8 : i * 8 * NT + tid; };

    float v[NV][8];
    const void *xr = row_of(p.x, p.x_bf16, p.ldx, t);
#pragma unroll
    for (int i = 0; i < NV; ++i) load8<VEC>(xr, p.x_bf16, col(i), step, n, v[i]);
    if (MODE == ROWS_SWIGLU) {
        const void *ur = (const char *)xr + (int64_t)n * (p.x_bf16 ? 2 : 4);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float u[8];
            load8<VEC>(ur, p.x_bf16, col(i), step, n, u);
            float low = v[i][0];
#pragma unroll
            for (int j = 1; j < 8; ++j) low = fminf(low, v[i][j]);
            if (__any(low < SILU_FAR)) {
#pragma unroll
                for (int j = 0; j < 8; ++j) v[i][j] = silu_mul<true>(v[i][j], u[j]);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) v[i][j] = silu_mul<false>(v[i][j], u[j]);
            }
        }
    }
    if (MODE == ROWS_NORM) {
        float g[NV][8];
#pragma unroll
        for (int i = 0; i < NV; ++i) load8<VEC>(p.weight, 0, col(i), step, n, g[i]);
        if (p.res) {
            const void *rr = row_of(p.res, p.res_bf16, p.ldres, t);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                float r[8];
                load8<VEC>(rr, p.res_bf16, col(i), step, n, r);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    v[i][j] = v[i][j] + r[j];
                    if (p.res_bf16) v[i][j] = bf16_bits_to_f32(to_bf16(v[i][j]));
                }
            }
            if (p.sum) {
                void *sr = (void *)row_of(p.sum, p.res_bf16, p.ldsum, t);
#pragma unroll
                for (int i = 0; i < NV; ++i) store8<VEC>(sr, p.res_bf16, col(i), step, n, v[i]);
            }
        }
        double ss = 0.0;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) ss = fma((double)v[i][j], (double)v[i][j], ss);
#pragma unroll
        for (int off = 32; off > 0; off >>= 1) ss += __shfl_xor(ss, off, 64);
        if (NW > 1) {
            if (lane == 0) part[wave] = ss;
            __syncthreads();
            ss = part[0];
#pragma unroll
            for (int w = 1; w < NW; ++w) ss += part[w];
        }
        const float r = (float)(1.0 / sqrt(ss / (double)n + (double)p.eps));
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] = (v[i][j] * r) * g[i][j];
        if (p.out) {
            void *orow = (void *)row_of(p.out, p.out_bf16, p.ldout, t);
#pragma unroll
            for (int i = 0; i < NV; ++i) store8<VEC>(orow, p.out_bf16, col(i), step, n, v[i]);
        }
    }
    if (!p.q) return;
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            // elements past the row: v is 0, or 0 * inf of a row that holds an
            // infinity, whose scale is NaN anyway
            m = max(m, __float_as_uint(v[i][j]) & 0x7fffffffu);
        }
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, off, 64));
    if (NW > 1) {
        if (lane == 0) pmax[wave] = m;
        __syncthreads();
        m = pmax[0];
#pragma unroll
        for (int w = 1; w < NW; ++w) m = max(m, pmax[w]);
    }
    const float amax = __uint_as_float(m);
    const bool finite = m < 0x7f800000u, some = amax >= 0x1p-100f;
    const float inv = finite && some ? 127.0f / amax : 0.0f;
    if (tid == 0) p.q_scale[t] = !finite ? __uint_as_float(0x7fc00000u) : some ? amax / 127.0f : 0.0f;
    int8_t *qr = p.q + (int64_t)t * p.ldq;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = col(i);
        uint32_t b[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) b[j] = finite ? code_bits(v[i][j], inv) : 0u;
        if (VEC) {
            if (c < n) *(uint2 *)(qr + c) = uint2{low_bytes(b[0], b[1], b[2], b[3]), low_bytes(b[4], b[5], b[6], b[7])};
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (c + j * step < n) qr[c + j * step] = (int8_t)b[j];
        }
    }
}

bool aligned(const void *p, int64_t ld, int size, int to) { return !p || ((uintptr_t)p % to == 0 && ld * size % to == 0); }

template <int MODE, bool VEC>
hipError_t launch_mode(const RowsPass &p, hipStream_t s)
{
#define MOE_ROWS(nt, nv) rows_kernel<MODE, nt, nv, VEC><<<p.T, nt, 0, s>>>(p)
    if (p.n <= 512) MOE_ROWS(64, 1);
    else if (p.n <= 1024) MOE_ROWS(128, 1);
    else if (p.n <= 2048) MOE_ROWS(256, 1);
    else if (p.n <= 4096) MOE_ROWS(256, 2);
    else if (p.n <= 8192) MOE_ROWS(512, 2);
    else if (p.n <= 16384) MOE_ROWS(1024, 2);
    else if (p.n <= 32768) MOE_ROWS(1024, 4);
    else MOE_ROWS(1024, 8);
#undef MOE_ROWS
    return hipGetLastError();
}

}  // namespace

hipError_t launch_rows(const RowsPass &p, hipStream_t s)
{
    // 16-byte pieces need aligned rows of whole groups of 8 elements (the
    // codes go in 8-byte pieces); anything else runs element by element
    const int xs = p.x_bf16 ? 2 : 4, rs = p.res_bf16 ? 2 : 4, os = p.out_bf16 ? 2 : 4;
    const bool vec = p.n % 8 == 0 && aligned(p.x, p.ldx, xs, 16) && aligned(p.res, p.ldres, rs, 16) &&
                     aligned(p.sum, p.ldsum, rs, 16) && aligned(p.out, p.ldout, os, 16) && aligned(p.q, p.ldq, 1, 8) &&
                     aligned(p.weight, 0, 4, 16);
    switch (p.mode) {
    case ROWS_NORM: return vec ? launch_mode<ROWS_NORM, true>(p, s) : launch_mode<ROWS_NORM, false>(p, s);
    case ROWS_QUANT: return vec ? launch_mode<ROWS_QUANT, true>(p, s) : launch_mode<ROWS_QUANT, false>(p, s);
    default: return vec ? launch_mode<ROWS_SWIGLU, true>(p, s) : launch_mode<ROWS_SWIGLU, false>(p, s);
    }
}

}  // namespace moe
