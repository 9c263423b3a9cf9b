// int8 linear layer on gfx950: y = (x w^T) * (xs ws^T) + bias + add, with the
// integer product on the int8 matrix instructions (exact int32 sums).
#include "common.h"
#include "linear.h"

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

// y[t][n .. n+CNT) from the integer sums of one lane
template <int CNT>
__device__ __forceinline__ void finish(const LinearPass &p, int t, int n, const int acc[CNT])
{
    if (t >= p.T) return;
    const float xs = p.x_scale[t];
    float v[CNT];
#pragma unroll
    for (int i = 0; i < CNT; ++i) {
        const int c = min(n + i, p.N - 1);
        v[i] = (float)acc[i] * (xs * p.w_scale[c]);
        if (p.bias) v[i] += p.bias[c];
    }
    const int64_t yo = (int64_t)t * p.ldy + n, ao = (int64_t)t * p.ldadd + n;
#pragma unroll
    for (int i = 0; i < CNT; ++i) {
        if (n + i >= p.N) break;
        if (p.add) v[i] += p.y_bf16 ? bf16_bits_to_f32(((const uint16_t *)p.add)[ao + i]) : ((const float *)p.add)[ao + i];
        if (p.y_bf16) ((uint16_t *)p.y)[yo + i] = (uint16_t)to_bf16(v[i]);
        else ((float *)p.y)[yo + i] = v[i];
    }
}

constexpr int BK = 128;                          // bytes of K per step

// Tile of 64 tokens x 64 channels, four waves of 32 x 32, one LDS buffer.
__global__ __launch_bounds__(256) void linear_tile(LinearPass p)
{
    __shared__ __align__(16) int8_t xl[64][BK + 16], wl[64][BK + 16];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int n0 = blockIdx.x * 64, t0 = blockIdx.y * 64;
    const int wn = (wave & 1) * 32, wt = (wave >> 1) * 32;
    const int fr = lane & 15, fg = lane >> 4;
    i32x4 acc[2][2];
#pragma unroll
    for (int a = 0; a < 2; ++a)
#pragma unroll
        for (int b = 0; b < 2; ++b) acc[a][b] = i32x4{0, 0, 0, 0};
    for (int k0 = 0; k0 < p.K; k0 += BK) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = (tid >> 3) + 32 * i, c = (tid & 7) * 16, k = k0 + c;
            i32x4 xv = {0, 0, 0, 0}, wv = {0, 0, 0, 0};
            if (k < p.K) {
                xv = *(const i32x4 *)(p.x + (int64_t)min(t0 + r, p.T - 1) * p.ldx + k);
                wv = *(const i32x4 *)(p.w + (int64_t)min(n0 + r, p.N - 1) * p.ldw + k);
                if (k + 16 > p.K) xv = mask_tail(xv, k, p.K);
            }
            *(i32x4 *)&xl[r][c] = xv;
            *(i32x4 *)&wl[r][c] = wv;
        }
        __syncthreads();
#pragma unroll
        for (int kk = 0; kk < BK; kk += 64) {
            i32x4 a[2], b[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                a[i] = *(const i32x4 *)&wl[wn + 16 * i + fr][kk + 16 * fg];
                b[i] = *(const i32x4 *)&xl[wt + 16 * i + fr][kk + 16 * fg];
            }
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(a[i], b[j], acc[i][j], 0, 0, 0);
        }
    }
    // D: lane (fr, fg) holds channels 4 fg .. 4 fg + 3 of token fr
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int v[4] = {acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]};
            finish<4>(p, t0 + wt + 16 * j + fr, n0 + wn + 16 * i + 4 * fg, v);
        }
}

}  // namespace

size_t linear_ws_bytes(int T, int N, int K)
{
    (void)T; (void)N; (void)K;
    return 0;
}

hipError_t launch_linear(const LinearPass &p, hipStream_t s)
{
    linear_tile<<<dim3((unsigned)((p.N + 63) / 64), (unsigned)((p.T + 63) / 64)), 256, 0, s>>>(p);
    return hipGetLastError();
}

}  // namespace moe
