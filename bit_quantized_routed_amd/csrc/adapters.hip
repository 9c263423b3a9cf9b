// Low-rank adapters of many requests beside a shared projection on gfx950.
//
//   low[t, q r + j] = sum_k x[t, k] A_a[q r + j, k]
//   y[t, n]        = add[t, n] + scale_a sum_j low[t, q(n) r + j] B_a[n, j]
//
// with a the adapter of token t, r the rank of one of the projection's parts and
// q(n) the part that output n belongs to.  A plan (one for all projections of a
// step) sorts the tokens by adapter and cuts them into tiles of one adapter each.
//
// Bound by memory: x, add and y are read and written once, an adapter's matrices
// once per tile and from the L2 after its first.  Products run on the bf16 matrix
// instructions without a rounding of their own: weights are bf16, codes of 8 bits
// are exact in bf16, fp32 values go as three bf16 terms that add up to them.  Sums
// are fp32.
#include "adapters.h"
#include "common.h"
#include "devcache.h"

#include <algorithm>

namespace moe {

namespace {

__device__ __forceinline__ uint32_t to_bf16(float f) { return __builtin_bit_cast(uint16_t, (__bf16)f); }

// ---------------------------------------------------------------- plan
// A stable counting sort by one work-group: a wave owns a stretch of the tokens and
// a row of counts of its own; the counts become positions (adapter first, then
// wave), and each wave walks its stretch again in order, a token's place among the
// wave's 64 from the lanes that hold the same adapter.  No sum hangs on an order
// of atomics.  8192 tokens, 100 adapters: see the entry point's figures.
constexpr int PLAN_NT = 1024, PLAN_NW = PLAN_NT / 64;
constexpr int BATCH = 8;                         // loads of a lane on their way together

__global__ __launch_bounds__(PLAN_NT) void adapter_plan(const int32_t *ids, int T, int n, int tile, int32_t *order, int32_t *offsets,
                                                        AdapterTile *tiles, int max_tiles)
{
    extern __shared__ int32_t count[];           // [waves][n + 1]; then first tiles [n + 2]
    __shared__ int32_t sums[2][PLAN_NW];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, bins = n + 1;
    int32_t *const mine = count + wave * bins, *const first_tile = count + PLAN_NW * bins;
    for (int i = tid; i < PLAN_NW * bins; i += PLAN_NT) count[i] = 0;
    const int stretch = ((T + PLAN_NW - 1) / PLAN_NW + 63) / 64 * 64, begin = min(T, wave * stretch), end = min(T, begin + stretch);
    auto bin = [&](int id) { return id >= 0 && id < n ? id : n; };
    __syncthreads();
    for (int t0 = begin + lane; t0 < end; t0 += 64 * BATCH) {
        int id[BATCH];
#pragma unroll
        for (int i = 0; i < BATCH; ++i) id[i] = t0 + 64 * i < end ? ids[t0 + 64 * i] : 0;
#pragma unroll
        for (int i = 0; i < BATCH; ++i)
            if (t0 + 64 * i < end) atomicAdd(&mine[bin(id[i])], 1);
    }
    __syncthreads();
    // thread b: bin b (bins <= 1025: thread 0 has the last one too); first the sums over the waves
    int carry[2] = {0, 0};
    for (int b0 = 0; b0 < bins; b0 += PLAN_NT) {
        const int b = b0 + tid;
        int total = 0;
        if (b < bins)
            for (int w = 0; w < PLAN_NW; ++w) total += count[w * bins + b];
        const int t = (total + tile - 1) / tile;
        int upto = total, upto_t = t;
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) {
            const int u = __shfl_up(upto, off, 64), v = __shfl_up(upto_t, off, 64);
            if (lane >= off) { upto += u; upto_t += v; }
        }
        if (lane == 63) { sums[0][wave] = upto; sums[1][wave] = upto_t; }
        __syncthreads();
        int all = 0, all_t = 0;
        for (int w = 0; w < PLAN_NW; ++w) {
            if (w < wave) { upto += sums[0][w]; upto_t += sums[1][w]; }
            all += sums[0][w];
            all_t += sums[1][w];
        }
        if (b < bins) {
            int at = carry[0] + upto - total;
            offsets[b] = at;                     // offsets[n]: where tokens without an adapter begin
            first_tile[b] = carry[1] + upto_t - t;
            for (int w = 0; w < PLAN_NW; ++w) {
                const int c = count[w * bins + b];
                count[w * bins + b] = at;
                at += c;
            }
        }
        carry[0] += all;
        carry[1] += all_t;
        __syncthreads();
    }
    if (tid == 0) first_tile[bins] = carry[1];
    __syncthreads();
    const int n_tiles = carry[1];
    for (int i = tid; i < max_tiles; i += PLAN_NT) {
        AdapterTile x{-2, 0};                    // no tile
        if (i < n_tiles) {
            int lo = 0, hi = bins;               // the last bin whose first tile is <= i
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (first_tile[mid] <= i) lo = mid;
                else hi = mid;
            }
            x.adapter = lo < n ? lo : -1;
            x.begin = count[lo] + (i - first_tile[lo]) * tile;         // wave 0's count is the bin's first position
        }
        tiles[i] = x;
    }
    __syncthreads();
    const int bits = 32 - __clz(n);
    for (int t0 = begin; t0 < end; t0 += 64 * BATCH) {
        int id[BATCH];
#pragma unroll
        for (int i = 0; i < BATCH; ++i) id[i] = t0 + 64 * i + lane < end ? bin(ids[t0 + 64 * i + lane]) : -1;
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
            if (t0 + 64 * i >= end) break;
            uint64_t same = __ballot(id[i] >= 0);
            for (int q = 0; q < bits; ++q) {
                const uint64_t set = __ballot(id[i] >> q & 1);
                same &= id[i] >> q & 1 ? set : ~set;
            }
            if (id[i] >= 0) {
                const int rank = __popcll(same & ((1ull << lane) - 1ull)), at = mine[id[i]] + rank;
                order[at] = t0 + 64 * i + lane;
                // the group's last lane moves the position on; the wave's LDS operations run in order
                asm volatile("" ::: "memory");
                __builtin_amdgcn_wave_barrier();
                if (same >> lane >> 1 == 0) mine[id[i]] = at + 1;
            }
            asm volatile("" ::: "memory");
            __builtin_amdgcn_wave_barrier();
        }
    }
}

// ---------------------------------------------------------------- values as bf16 terms
template <int KIND>
constexpr int terms() { return KIND == ADAPT_F32 ? 3 : 1; }

struct Raw { u32x4 u[2]; };                      // eight values as they are in memory

// eight values of a row from k on, zeros past K
template <int KIND, bool VEC>
__device__ __forceinline__ Raw load_x(const void *row, int k, int K)
{
    Raw v;
    if (VEC && k + 8 <= K) {
        if (KIND == ADAPT_F32) {
            v.u[0] = *(const u32x4 *)((const float *)row + k);
            v.u[1] = *(const u32x4 *)((const float *)row + k + 4);
        } else if (KIND == ADAPT_BF16) v.u[0] = *(const u32x4 *)((const uint16_t *)row + k);
        else {
            const uint2 c = *(const uint2 *)((const int8_t *)row + k);
            v.u[0][0] = c.x;
            v.u[0][1] = c.y;
        }
        return v;
    }
    v.u[0] = v.u[1] = u32x4{0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (k + i < K) {
            if (KIND == ADAPT_F32) v.u[i >> 2][i & 3] = __float_as_uint(((const float *)row)[k + i]);
            else if (KIND == ADAPT_BF16) v.u[0][i >> 1] |= (uint32_t)((const uint16_t *)row)[k + i] << (16 * (i & 1));
            else v.u[0][i >> 2] |= (uint32_t)((const uint8_t *)row)[k + i] << (8 * (i & 3));
        }
    return v;
}

// terms of fp32 values, largest first: each difference is exact, and the third holds what is left of 24 bits
__device__ __forceinline__ void split(const float v[8], bf16x8 t[3])
{
    u32x4 u[3];
    float rest[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) rest[i] = v[i];
#pragma unroll
    for (int s = 0; s < 3; ++s)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t lo = to_bf16(rest[2 * i]), hi = to_bf16(rest[2 * i + 1]);
            u[s][i] = lo | hi << 16;
            rest[2 * i] -= bf16_bits_to_f32(lo);
            rest[2 * i + 1] -= bf16_bits_to_f32(hi);
        }
#pragma unroll
    for (int s = 0; s < 3; ++s) t[s] = __builtin_bit_cast(bf16x8, u[s]);
}

template <int KIND>
__device__ __forceinline__ void as_terms(const Raw &v, bf16x8 t[3])
{
    if (KIND == ADAPT_BF16) t[0] = __builtin_bit_cast(bf16x8, v.u[0]);
    else if (KIND == ADAPT_F32) {
        float f[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(v.u[i >> 2][i & 3]);
        split(f, t);
    } else {
        u32x4 u;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t w = v.u[0][i >> 1] >> (16 * (i & 1));
            u[i] = f32_to_bf16_exact((float)(int8_t)(w & 255u)) | f32_to_bf16_exact((float)(int8_t)(w >> 8 & 255u)) << 16;
        }
        t[0] = __builtin_bit_cast(bf16x8, u);
    }
}

// ---------------------------------------------------------------- down: low = x A^T
// A work-group takes a tile (TT fragments of 16 tokens) and one part of K.  Its waves
// share out the columns of low (cw ways, up to CT fragments each) and what is left of
// the split the part's K, in stretches of whole steps of 64 (a line of 128 bytes of
// bf16, requested at once; neighbouring waves are on different L2 channels); these
// sums meet in LDS in a fixed order.
template <int TT>
constexpr int down_waves() { return TT == 1 ? 8 : 4; }
constexpr int DSTEP = 64;

template <int TT, int CT, int KIND, bool VEC>
__global__ __launch_bounds__(64 * down_waves<TT>()) void adapter_down(AdapterPass p, int k_parts, int cw)
{
    constexpr int NS = terms<KIND>(), NW = down_waves<TT>();
    const AdapterTile tile = p.tiles[blockIdx.x];
    if (tile.adapter < 0) return;
    const int end = p.offsets[tile.adapter + 1], count = min(16 * TT, end - tile.begin);
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), r = lane & 15, g = lane >> 4;
    const int R = p.parts * p.rank, frags = (R + 15) / 16, kw = NW / cw, wc = wave % cw, wk = wave / cw;
    const int r8 = (p.rank + 7) & ~7, width = p.parts * r8;
    // this wave's steps: stretch part * kw + wk of k_parts * kw
    const int steps = (p.K + DSTEP - 1) / DSTEP, part = blockIdx.y, stretch = part * kw + wk;
    const int s0 = (int)((int64_t)steps * stretch / (k_parts * kw)), s1 = (int)((int64_t)steps * (stretch + 1) / (k_parts * kw));
    const void *row[TT];
#pragma unroll
    for (int i = 0; i < TT; ++i) {
        const int t = p.order[tile.begin + min(16 * i + r, count - 1)];
        row[i] = (const char *)p.x + (int64_t)t * p.ldx * (KIND == ADAPT_F32 ? 4 : KIND == ADAPT_BF16 ? 2 : 1);
    }
    const uint16_t *col[CT];
    int n_cols = 0;
#pragma unroll
    for (int c = 0; c < CT; ++c) {
        const int f = wc + c * cw;
        if (f < frags) n_cols = c + 1;
        col[c] = p.a + ((int64_t)tile.adapter * R + min(16 * f + r, R - 1)) * p.lda;
    }
    f32x4 acc[TT][CT];
#pragma unroll
    for (int i = 0; i < TT; ++i)
#pragma unroll
        for (int c = 0; c < CT; ++c) acc[i][c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    Raw x[2][TT];
    u32x4 w[2][CT];
    // the halves of a step are interleaved so that both of its loads touch whole lines; rows of A are zero past K, where there is anything
    auto load = [&](int s) {
        if (s >= s1) return;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int k = DSTEP * s + 16 * g + 8 * h;
#pragma unroll
            for (int i = 0; i < TT; ++i) x[h][i] = load_x<KIND, VEC>(row[i], k, p.K);
#pragma unroll
            for (int c = 0; c < CT; ++c)
                if (c < n_cols) w[h][c] = k < p.K ? *(const u32x4 *)(col[c] + k) : u32x4{0, 0, 0, 0};
        }
    };
    load(s0);
    for (int s = s0; s < s1; ++s) {
        Raw xn[2][TT];
        u32x4 b[2][CT];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int i = 0; i < TT; ++i) xn[h][i] = x[h][i];
#pragma unroll
            for (int c = 0; c < CT; ++c) b[h][c] = w[h][c];
        }
        load(s + 1);
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < TT; ++i) {
                bf16x8 a[3];
                as_terms<KIND>(xn[h][i], a);
#pragma unroll
                for (int c = 0; c < CT; ++c)
                    if (c < n_cols) {
#pragma unroll
                        for (int q = NS - 1; q >= 0; --q)              // smallest term first
                            acc[i][c] = mfma16x16x32(a[q], __builtin_bit_cast(bf16x8, b[h][c]), acc[i][c]);
                    }
            }
    }
    // sums over the waves that share these columns, by halves
    extern __shared__ f32x4 sums[];              // [kw / 2][TT][column fragments][64]
    for (int half = kw / 2; half > 0; half /= 2) {
        f32x4 *const at = sums + ((wk & (half - 1)) * TT * frags + wc) * 64 + lane;
        if (wk >= half && wk < 2 * half) {
#pragma unroll
            for (int c = 0; c < CT; ++c)
                if (c < n_cols) {
#pragma unroll
                    for (int i = 0; i < TT; ++i) at[(i * frags + c * cw) * 64] = acc[i][c];
                }
        }
        __syncthreads();
        if (wk < half) {
#pragma unroll
            for (int c = 0; c < CT; ++c)
                if (c < n_cols) {
#pragma unroll
                    for (int i = 0; i < TT; ++i) acc[i][c] += at[(i * frags + c * cw) * 64];
                }
        }
        __syncthreads();
    }
    if (wk > 0) return;
#pragma unroll
    for (int c = 0; c < CT; ++c) {
        const int f = 16 * (wc + c * cw) + r;    // D: lane (r, g) holds tokens 4 g .. 4 g + 3 of column r
        if (c >= n_cols || f >= R) continue;
        float *const o = p.low + ((int64_t)part * p.T + tile.begin) * width + f / p.rank * r8 + f % p.rank;
#pragma unroll
        for (int i = 0; i < TT; ++i)
#pragma unroll
            for (int q = 0; q < 4; ++q)
                if (16 * i + 4 * g + q < count) o[(int64_t)(16 * i + 4 * g + q) * width] = acc[i][c][q];
    }
}

// ---------------------------------------------------------------- up: y = add + scale B low
// A work-group takes a tile (TT fragments of 16 tokens) and a stretch of one part's
// outputs.  low, with its scale and as bf16 terms, is made once in LDS; each of the
// four waves then takes 64 outputs at a time: four fragments whose rows are dealt so
// that a lane ends up with 16 consecutive outputs of one token.
constexpr int WIDE = 64;

template <bool BF16>
struct Piece { u32x4 u[BF16 ? 2 : 4]; };         // 16 values

template <int TT, bool BF16, bool VEC, int KS>   // KS: steps of 32 of the rank
__global__ __launch_bounds__(256) void adapter_up(AdapterPass p, int k_parts, int chunks)
{
    __shared__ bf16x8 low[3][TT][KS][64];
    const AdapterTile tile = p.tiles[blockIdx.x];
    if (tile.adapter < -1 || (tile.adapter < 0 && p.add == p.y)) return;
    const int end = tile.adapter < 0 ? p.T : p.offsets[tile.adapter + 1], count = min(16 * TT, end - tile.begin);
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), r = lane & 15, g = lane >> 4;
    const int Np = p.N / p.parts, groups = (Np + WIDE - 1) / WIDE, r8 = (p.rank + 7) & ~7, width = p.parts * r8;
    const int q = blockIdx.y / chunks, chunk = blockIdx.y % chunks, u1 = groups * (chunk + 1) / chunks;
    constexpr int ES = BF16 ? 2 : 4, PW = BF16 ? 2 : 4;
    int t[TT];
#pragma unroll
    for (int i = 0; i < TT; ++i) t[i] = p.order[tile.begin + min(16 * i + r, count - 1)];
    if (tile.adapter >= 0) {
        const float scale = p.scale[tile.adapter];
#pragma unroll
        for (int i = 0; i < TT; ++i) {
            if (i % 4 != wave) continue;
            const int pos = tile.begin + min(16 * i + r, count - 1);
            const float factor = scale * (p.x_scale ? p.x_scale[t[i]] : 1.0f);
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                // the parts of K in order, eight parts' loads on their way together
                constexpr int B = 8;
                f32x4 v[2] = {f32x4{0.0f, 0.0f, 0.0f, 0.0f}, f32x4{0.0f, 0.0f, 0.0f, 0.0f}};
                const int j = 32 * s + 8 * g;
                if (j < p.rank)
                    for (int k0 = 0; k0 < k_parts; k0 += B) {
                        f32x4 x[B][2];
#pragma unroll
                        for (int k = 0; k < B; ++k)
#pragma unroll
                            for (int h = 0; h < 2; ++h)
                                x[k][h] = *(const f32x4 *)(p.low + ((int64_t)min(k0 + k, k_parts - 1) * p.T + pos) * width + q * r8 + j + 4 * h);
#pragma unroll
                        for (int k = 0; k < B; ++k)
                            if (k0 + k < k_parts) {
                                v[0] += x[k][0];
                                v[1] += x[k][1];
                            }
                    }
                float f[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) f[e] = j + e < p.rank ? v[e >> 2][e & 3] * factor : 0.0f;
                bf16x8 terms[3];
                split(f, terms);
#pragma unroll
                for (int m = 0; m < 3; ++m) low[m][i][s][lane] = terms[m];
            }
        }
        __syncthreads();
    }
    for (int u = groups * chunk / chunks + wave; u < u1; u += 4) {
        const int n0 = u * WIDE, outs = min(16, Np - n0 - 16 * g);     // of this lane (none if negative)
        const int64_t at = (int64_t)q * Np + n0 + 16 * g;
        u32x4 w[4][KS];
        if (tile.adapter >= 0) {
            // b's rows of this lane: output n0 + 16 (r / 4) + 4 f + r % 4 of fragment f; zero past the rank
#pragma unroll
            for (int f = 0; f < 4; ++f) {
                const int n = min(n0 + 16 * (r >> 2) + 4 * f + (r & 3), Np - 1);
                const uint16_t *const row = p.b + ((int64_t)tile.adapter * p.N + (int64_t)q * Np + n) * p.ldb;
#pragma unroll
                for (int s = 0; s < KS; ++s) w[f][s] = 32 * s + 8 * g < p.rank ? *(const u32x4 *)(row + 32 * s + 8 * g) : u32x4{0, 0, 0, 0};
            }
        }
        Piece<BF16> old[TT];
#pragma unroll
        for (int i = 0; i < TT; ++i)
            if (VEC && outs == 16 && 16 * i + r < count) {
#pragma unroll
                for (int h = 0; h < PW; ++h) old[i].u[h] = ((const u32x4 *)((const char *)p.add + ((int64_t)t[i] * p.ldadd + at) * ES))[h];
            }
#pragma unroll
        for (int i = 0; i < TT; ++i) {
            if (16 * i >= count) break;
            const bool whole = VEC && outs == 16 && 16 * i + r < count;
            const int mine = 16 * i + r < count ? outs : 0;
            const char *const add = (const char *)p.add + ((int64_t)t[i] * p.ldadd + at) * ES;
            char *const y = (char *)p.y + ((int64_t)t[i] * p.ldy + at) * ES;
            if (tile.adapter < 0) {              // no adapter: add as it is
                if (whole) {
#pragma unroll
                    for (int h = 0; h < PW; ++h) ((u32x4 *)y)[h] = old[i].u[h];
                } else
                    for (int e = 0; e < mine; ++e) {
                        if (BF16) ((uint16_t *)y)[e] = ((const uint16_t *)add)[e];
                        else ((float *)y)[e] = ((const float *)add)[e];
                    }
                continue;
            }
            f32x4 acc[4];
#pragma unroll
            for (int f = 0; f < 4; ++f) acc[f] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int m = 2; m >= 0; --m)         // smallest term first
#pragma unroll
                for (int s = 0; s < KS; ++s) {
                    const bf16x8 x = low[m][i][s][lane];
#pragma unroll
                    for (int f = 0; f < 4; ++f) acc[f] = mfma16x16x32(__builtin_bit_cast(bf16x8, w[f][s]), x, acc[f]);
                }
            // D: lane (r, g) holds rows 4 g + i of token r: acc[f][i] is output 4 f + i of its 16
            if (whole) {
#pragma unroll
                for (int h = 0; h < PW; ++h) {
                    u32x4 o;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        if (BF16) {
                            const int f = 2 * h + (e >> 1), j = 2 * (e & 1);
                            o[e] = to_bf16(__uint_as_float(old[i].u[h][e] << 16) + acc[f][j]) |
                                   to_bf16(__uint_as_float(old[i].u[h][e] & 0xffff0000u) + acc[f][j + 1]) << 16;
                        } else o[e] = __float_as_uint(__uint_as_float(old[i].u[h][e]) + acc[h][e]);
                    }
                    ((u32x4 *)y)[h] = o;
                }
            } else {
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    if (e < mine) {
                        const float v = acc[e >> 2][e & 3];
                        if (BF16) ((uint16_t *)y)[e] = (uint16_t)to_bf16(bf16_bits_to_f32(((const uint16_t *)add)[e]) + v);
                        else ((float *)y)[e] = ((const float *)add)[e] + v;
                    }
            }
        }
    }
}

bool aligned(const void *p, int64_t ld, int size, int to) { return (uintptr_t)p % to == 0 && ld * size % to == 0; }

}  // namespace

// Work-groups of up to two a CU at once: tiles of a large batch fill them, a few tokens are cut along K, into parts of at least
// 256.
int adapter_k_parts(int T, int K, int n)
{
    const int tiles = std::min(T, (T + adapter_tile(T) - 1) / adapter_tile(T) + n), steps = (K + 31) / 32;
    return std::max(1, std::min(512 / tiles, steps / 8));
}

size_t adapter_low_bytes(int T, int K, int width, int n)
{
    int64_t rows = 0;
    for (int t = 1; t <= std::min(T, 512); ++t) rows = std::max(rows, (int64_t)t * adapter_k_parts(t, K, n));
    // past 512 tokens a tile is 64: t * (512 / (t / 64)) rows at most, and t of one part
    if (T > 512) rows = std::max(rows, std::min(std::max((int64_t)T, (int64_t)512 * 64), (int64_t)T * std::max(1, (K + 31) / 32 / 8)));
    return (size_t)rows * width * sizeof(float);
}

hipError_t launch_adapter_plan(const int32_t *ids, int T, int n, int32_t *order, int32_t *offsets, AdapterTile *tiles, hipStream_t s)
{
    static DevSlots slots{};
    const size_t lds = ((size_t)PLAN_NW * (n + 1) + n + 2) * 4;
    const hipError_t e = lds_limit((const void *)adapter_plan, slots, lds);
    if (e != hipSuccess) return e;
    adapter_plan<<<1, PLAN_NT, lds, s>>>(ids, T, n, adapter_tile(T), order, offsets, tiles, adapter_tiles(T, n));
    return hipGetLastError();
}

hipError_t launch_adapter_down(const AdapterPass &p, hipStream_t s)
{
    const int parts = adapter_k_parts(p.T, p.K, p.n), frags = (p.parts * p.rank + 15) / 16, tt = adapter_tile(p.T) / 16;
    // up to four column fragments a wave; the other waves divide K
    const int cw = frags <= 4 ? 1 : frags <= 8 ? 2 : 4, ct = (frags + cw - 1) / cw, waves = tt == 1 ? down_waves<1>() : down_waves<4>();
    const int es = p.kind == ADAPT_F32 ? 4 : p.kind == ADAPT_BF16 ? 2 : 1;
    const bool vec = aligned(p.x, p.ldx, es, std::min(16, 8 * es));
    const dim3 grid((unsigned)adapter_tiles(p.T, p.n), (unsigned)parts);
    const size_t lds = (size_t)(waves / cw / 2) * tt * frags * 64 * 16;
#define MOE_DOWN3(t, c, kind, v)                                                                  \
    do {                                                                                          \
        static DevSlots slots{};                                                                  \
        const hipError_t e = lds_limit((const void *)adapter_down<t, c, kind, v>, slots, lds);    \
        if (e != hipSuccess) return e;                                                            \
        adapter_down<t, c, kind, v><<<grid, 64 * waves, lds, s>>>(p, parts, cw);                  \
    } while (0)
#define MOE_DOWN2(t, c, kind)                                                                     \
    do {                                                                                          \
        if (vec) MOE_DOWN3(t, c, kind, true);                                                     \
        else MOE_DOWN3(t, c, kind, false);                                                        \
    } while (0)
#define MOE_DOWN1(t, kind)                                                                        \
    do {                                                                                          \
        if (ct <= 2) MOE_DOWN2(t, 2, kind);                                                       \
        else MOE_DOWN2(t, 4, kind);                                                               \
    } while (0)
#define MOE_DOWN(t)                                                                               \
    do {                                                                                          \
        if (p.kind == ADAPT_F32) MOE_DOWN1(t, ADAPT_F32);                                         \
        else if (p.kind == ADAPT_BF16) MOE_DOWN1(t, ADAPT_BF16);                                  \
        else MOE_DOWN1(t, ADAPT_I8);                                                              \
    } while (0)
    if (tt == 1) MOE_DOWN(1);
    else MOE_DOWN(4);
#undef MOE_DOWN1
#undef MOE_DOWN3
#undef MOE_DOWN
#undef MOE_DOWN2
    return hipGetLastError();
}

hipError_t launch_adapter_up(const AdapterPass &p, hipStream_t s)
{
    const int parts = adapter_k_parts(p.T, p.K, p.n), es = p.y_bf16 ? 2 : 4;
    const int tiles = adapter_tiles(p.T, p.n), groups = (p.N / p.parts + WIDE - 1) / WIDE;
    // about 16 waves a CU, stretches of at least a group a wave
    const int chunks = std::max(1, std::min((groups + 3) / 4, (1024 + tiles * p.parts - 1) / (tiles * p.parts)));
    const bool vec = aligned(p.y, p.ldy, es, 16) && aligned(p.add, p.ldadd, es, 16) && p.N / p.parts % (16 / es) == 0;
    const dim3 grid((unsigned)tiles, (unsigned)(p.parts * chunks));
#define MOE_UP3(t, bf, v)                                                                         \
    do {                                                                                          \
        if (p.rank <= 32) adapter_up<t, bf, v, 1><<<grid, 256, 0, s>>>(p, parts, chunks);         \
        else adapter_up<t, bf, v, 2><<<grid, 256, 0, s>>>(p, parts, chunks);                      \
    } while (0)
#define MOE_UP2(t, bf)                                                                            \
    do {                                                                                          \
        if (vec) MOE_UP3(t, bf, true);                                                            \
        else MOE_UP3(t, bf, false);                                                               \
    } while (0)
#define MOE_UP(t)                                                                                 \
    do {                                                                                          \
        if (p.y_bf16) MOE_UP2(t, true);                                                           \
        else MOE_UP2(t, false);                                                                   \
    } while (0)
    if (adapter_tile(p.T) == 16) MOE_UP(1);
    else MOE_UP(4);
#undef MOE_UP3
#undef MOE_UP
#undef MOE_UP2
    return hipGetLastError();
}

}  // namespace moe
