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
// of atomics.  Bound by latency: 8192 tokens, 100 adapters 14 us, 64 tokens 4.5 us.
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
    // walks the wave's stretch in order: step(token, bin, lanes of the same bin), bin -1 past the end
    const int bits = 32 - __clz(n);
    auto walk = [&](auto step) {
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
                // the wave's LDS operations run in order
                asm volatile("" ::: "memory");
                __builtin_amdgcn_wave_barrier();
                if (id[i] >= 0) step(t0 + 64 * i + lane, id[i], same);
                asm volatile("" ::: "memory");
                __builtin_amdgcn_wave_barrier();
            }
        }
    };
    __syncthreads();
    // one lane counts for all of a bin (with 64 lanes' atomics on one word 8192 tokens took 15.9 us, not 14.3)
    walk([&](int, int b, uint64_t same) {
        if (same >> lane >> 1 == 0) mine[b] += __popcll(same);
    });
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
    walk([&](int t, int b, uint64_t same) {
        const int at = mine[b] + __popcll(same & ((1ull << lane) - 1ull));
        if (at < T) order[at] = t;               // ids that another stream changes between the walks
        asm volatile("" ::: "memory");
        __builtin_amdgcn_wave_barrier();
        if (same >> lane >> 1 == 0) mine[b] = at + 1;                  // the last lane moves the position on
    });
}

// ---------------------------------------------------------------- what the kernels take from a plan
// In bounds whatever the plan's memory holds: it is the caller's, and one that is read before it is filled, or while another
// stream fills it, may cost the results of the call but no access past its tensors.
struct Taken { int adapter, begin, count; };     // count 0: nothing to do

template <int SIZE>
__device__ __forceinline__ Taken take_tile(const AdapterPass &p)
{
    const AdapterTile tile = p.tiles[blockIdx.x];
    const int adapter = max(-1, min(tile.adapter, p.n - 1)), begin = max(0, min(tile.begin, p.T));
    const int end = adapter < 0 ? p.T : max(0, min(p.offsets[adapter + 1], p.T));
    return Taken{adapter, begin, adapter == tile.adapter ? max(0, min(SIZE, end - begin)) : 0};
}

__device__ __forceinline__ int token_at(const AdapterPass &p, int pos) { return (int)min((uint32_t)p.order[pos], (uint32_t)(p.T - 1)); }

// ---------------------------------------------------------------- values as bf16 terms
template <int KIND>
constexpr int terms() { return KIND == ADAPT_F32 ? 3 : 1; }

struct Raw { u32x4 u[2]; };                      // eight values as they are in memory

// Eight values of a row from k on.  VEC: aligned rows of K % 8 == 0 values, and past K the row's last eight, without a
// branch (A is zero there, and what an infinity times that zero is comes to its own token alone); else element by element,
// zeros past K.
template <int KIND, bool VEC>
__device__ __forceinline__ Raw load_x(const void *row, int k, int K)
{
    Raw v;
    if (VEC) {
        k = min(k, K - 8);
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
// sums meet in LDS in a fixed order.  64 tokens of 32 adapters, 7168 in, rank 2 x 16: 6 us.
template <int TT>
constexpr int down_waves() { return TT == 1 ? 8 : 4; }
constexpr int DSTEP = 64;

template <int TT, int CT, int KIND, bool VEC>
__global__ __launch_bounds__(64 * down_waves<TT>()) void adapter_down(AdapterPass p, int k_parts, int cw)
{
    constexpr int NS = terms<KIND>(), NW = down_waves<TT>();
    const Taken tile = take_tile<16 * TT>(p);
    if (tile.adapter < 0 || tile.count == 0) return;
    const int count = tile.count;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), r = lane & 15, g = lane >> 4;
    const int R = p.parts * p.rank, frags = (R + 15) / 16, kw = NW / cw, wc = wave % cw, wk = wave / cw;
    const int r8 = (p.rank + 7) & ~7, width = p.parts * r8;
    // this wave's steps: stretch part * kw + wk of k_parts * kw
    const int steps = (p.K + DSTEP - 1) / DSTEP, part = blockIdx.y, stretch = part * kw + wk;
    const int s0 = (int)((int64_t)steps * stretch / (k_parts * kw)), s1 = (int)((int64_t)steps * (stretch + 1) / (k_parts * kw));
    const void *row[TT];
#pragma unroll
    for (int i = 0; i < TT; ++i) {
        const int t = token_at(p, tile.begin + min(16 * i + r, count - 1));
        row[i] = (const char *)p.x + (int64_t)t * p.ldx * (KIND == ADAPT_F32 ? 4 : KIND == ADAPT_BF16 ? 2 : 1);
    }
    const uint16_t *col[CT];
    // fragments past the last one compute it again and are not stored
#pragma unroll
    for (int c = 0; c < CT; ++c) {
        const int f = wc + c * cw;
        col[c] = p.a + ((int64_t)tile.adapter * R + min(16 * f + r, R - 1)) * p.lda;
    }
    f32x4 acc[TT][CT];
#pragma unroll
    for (int i = 0; i < TT; ++i)
#pragma unroll
        for (int c = 0; c < CT; ++c) acc[i][c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    struct Step { Raw x[2][TT]; u32x4 w[2][CT]; };
    const int last = ((p.K + 7) & ~7) - 8;       // rows of A have zeros up to a multiple of 8
    auto load = [&](int s, Step &v) {
        s = min(s, s1 - 1);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int k = DSTEP * s + 32 * h + 8 * g;
#pragma unroll
            for (int i = 0; i < TT; ++i) v.x[h][i] = load_x<KIND, VEC>(row[i], k, p.K);
#pragma unroll
            for (int c = 0; c < CT; ++c) v.w[h][c] = *(const u32x4 *)(col[c] + min(k, last));
        }
    };
    auto multiply = [&](int s, Step &v) {
        if (DSTEP * (s + 1) > last + 8) {        // the row's last step: nothing past its end
#pragma unroll
            for (int h = 0; h < 2; ++h)
                if (DSTEP * s + 32 * h + 8 * g > last) {
#pragma unroll
                    for (int c = 0; c < CT; ++c) v.w[h][c] = u32x4{0, 0, 0, 0};
                }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < TT; ++i) {
                bf16x8 a[3];
                as_terms<KIND>(v.x[h][i], a);
#pragma unroll
                for (int c = 0; c < CT; ++c)
#pragma unroll
                    for (int q = NS - 1; q >= 0; --q)                  // smallest term first
                        acc[i][c] = mfma16x16x32(a[q], __builtin_bit_cast(bf16x8, v.w[h][c]), acc[i][c]);
            }
    };
    // two steps by name: a copy of the one would wait for its loads
    if (s0 < s1) {
        Step even, odd;
        load(s0, even);
        for (int s = s0; s < s1; s += 2) {
            if (s + 1 < s1) load(s + 1, odd);
            multiply(s, even);
            if (s + 2 < s1) load(s + 2, even);
            if (s + 1 < s1) multiply(s + 1, odd);
        }
    }
    // sums over the waves that share these columns, by halves
    extern __shared__ f32x4 sums[];              // [kw / 2][TT][column fragments][64]
    for (int half = kw / 2; half > 0; half /= 2) {
        f32x4 *const at = sums + ((wk & (half - 1)) * TT * frags + wc) * 64 + lane;
        if (wk >= half && wk < 2 * half) {
#pragma unroll
            for (int c = 0; c < CT; ++c)
                if (wc + c * cw < frags) {
#pragma unroll
                    for (int i = 0; i < TT; ++i) at[(i * frags + c * cw) * 64] = acc[i][c];
                }
        }
        __syncthreads();
        if (wk < half) {
#pragma unroll
            for (int c = 0; c < CT; ++c)
                if (wc + c * cw < frags) {
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
        if (f >= R) continue;
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
// four waves then takes 64 outputs at a time: fragment f has outputs f, f + 4, .. of
// them, so that a lane ends up with four outputs in a row and 16 neighbouring lanes
// with the 64 of one token.  Bound by memory: 8192 tokens, two parts of 2048 outputs,
// add and y bf16, 134 MB: 56 us (2.4 TB/s).  512 x 7168 of fp32 12 us.
constexpr int WIDE = 64;

template <bool BF16>
struct Four { uint32_t u[BF16 ? 2 : 4]; };       // four outputs

template <bool BF16>
__device__ __forceinline__ Four<BF16> load_four(const void *p)
{
    Four<BF16> v;
    if (BF16) {
        const uint2 u = *(const uint2 *)p;
        v.u[0] = u.x;
        v.u[1] = u.y;
    } else {
        const u32x4 u = *(const u32x4 *)p;
#pragma unroll
        for (int i = 0; i < 4; ++i) v.u[BF16 ? 0 : i] = u[i];
    }
    return v;
}

template <int TT, bool BF16, bool VEC, int KS>   // KS: steps of 32 of the rank
__global__ __launch_bounds__(256) void adapter_up(AdapterPass p, int k_parts, int chunks)
{
    __shared__ bf16x8 low[3][TT][KS][64];
    const Taken tile = take_tile<16 * TT>(p);
    if (tile.count == 0 || (tile.adapter < 0 && p.add == p.y)) return;
    const int count = tile.count;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), r = lane & 15, g = lane >> 4;
    const int Np = p.N / p.parts, groups = (Np + WIDE - 1) / WIDE, r8 = (p.rank + 7) & ~7, width = p.parts * r8;
    const int q = blockIdx.y / chunks, chunk = blockIdx.y % chunks, u1 = groups * (chunk + 1) / chunks;
    constexpr int ES = BF16 ? 2 : 4;
    int t[TT][4];                                // tokens 4 g .. 4 g + 3 of each fragment
#pragma unroll
    for (int i = 0; i < TT; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) t[i][e] = token_at(p, tile.begin + min(16 * i + 4 * g + e, count - 1));
    // what a group of 64 outputs reads: b's rows of this lane and add; the first group's are on their way while low is made.  No
    // branches: what lies past the end is clamped, and not stored; past the rank low is zero
    struct Group { u32x4 w[4][KS]; Four<BF16> old[TT][4]; };
    auto load = [&](int u, Group &v) {
        const int n0 = min(u, groups - 1) * WIDE;
#pragma unroll
        for (int f = 0; f < 4; ++f) {
            const uint16_t *const row = p.b + ((int64_t)max(tile.adapter, 0) * p.N + (int64_t)q * Np + min(n0 + 4 * r + f, Np - 1)) * p.ldb;
#pragma unroll
            for (int s = 0; s < KS; ++s) v.w[f][s] = *(const u32x4 *)(row + min(32 * s + 8 * g, r8 - 8));
        }
        if (VEC) {
#pragma unroll
            for (int i = 0; i < TT; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    v.old[i][e] = load_four<BF16>((const char *)p.add + ((int64_t)t[i][e] * p.ldadd + (int64_t)q * Np + min(n0 + 4 * r, Np - 4)) * ES);
        }
    };
    const int u0 = groups * chunk / chunks + wave;
    Group even, odd;
    load(u0, even);
    if (tile.adapter >= 0) {
        const float scale = p.scale[tile.adapter];
#pragma unroll
        for (int i = 0; i < TT; ++i) {
            if (i % 4 != wave) continue;
            const int pos = tile.begin + min(16 * i + r, count - 1);
            const float factor = scale * (p.x_scale ? p.x_scale[token_at(p, pos)] : 1.0f);
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
    auto finish = [&](int u, const Group &v) {
        const int n0 = u * WIDE, mine = min(4, Np - n0 - 4 * r);       // outputs of this lane (none if negative)
        const int64_t from = (int64_t)q * Np + n0 + 4 * r;
#pragma unroll
        for (int i = 0; i < TT; ++i) {
            f32x4 acc[4];
#pragma unroll
            for (int f = 0; f < 4; ++f) acc[f] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            if (tile.adapter >= 0) {
#pragma unroll
                for (int m = 2; m >= 0; --m)     // smallest term first
#pragma unroll
                    for (int s = 0; s < KS; ++s) {
                        const bf16x8 x = low[m][i][s][lane];
#pragma unroll
                        for (int f = 0; f < 4; ++f) acc[f] = mfma16x16x32(x, __builtin_bit_cast(bf16x8, v.w[f][s]), acc[f]);
                    }
            }
            // D: lane (r, g) holds tokens 4 g + e of output 4 r + f
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (16 * i + 4 * g + e >= count) continue;
                const char *const add = (const char *)p.add + ((int64_t)t[i][e] * p.ldadd + from) * ES;
                char *const y = (char *)p.y + ((int64_t)t[i][e] * p.ldy + from) * ES;
                if (VEC && mine == 4) {
                    Four<BF16> o = v.old[i][e];
                    if (tile.adapter >= 0) {     // else add as it is
                        if (BF16) {
#pragma unroll
                            for (int j = 0; j < 2; ++j)
                                o.u[j] = to_bf16(__uint_as_float(o.u[j] << 16) + acc[2 * j][e]) |
                                         to_bf16(__uint_as_float(o.u[j] & 0xffff0000u) + acc[2 * j + 1][e]) << 16;
                        } else {
#pragma unroll
                            for (int j = 0; j < 4; ++j) o.u[BF16 ? 0 : j] = __float_as_uint(__uint_as_float(o.u[BF16 ? 0 : j]) + acc[j][e]);
                        }
                    }
                    if (BF16) *(uint2 *)y = uint2{o.u[0], o.u[1]};
                    else *(u32x4 *)y = u32x4{o.u[0], o.u[1], o.u[BF16 ? 0 : 2], o.u[BF16 ? 0 : 3]};
                } else {
#pragma unroll
                    for (int f = 0; f < 4; ++f)
                        if (f < mine) {
                            if (BF16) {
                                const uint16_t a = ((const uint16_t *)add)[f];
                                ((uint16_t *)y)[f] = tile.adapter < 0 ? a : (uint16_t)to_bf16(bf16_bits_to_f32(a) + acc[f][e]);
                            } else {
                                const uint32_t a = ((const uint32_t *)add)[f];
                                ((uint32_t *)y)[f] = tile.adapter < 0 ? a : __float_as_uint(__uint_as_float(a) + acc[f][e]);
                            }
                        }
                }
            }
        }
    };
    // two groups by name: a copy of the one would wait for its loads
    for (int u = u0; u < u1; u += 8) {
        if (u + 4 < u1) load(u + 4, odd);
        finish(u, even);
        if (u + 8 < u1) load(u + 8, even);
        if (u + 4 < u1) finish(u + 4, odd);
    }
}

// ---------------------------------------------------------------- down for large batches
// Tiles of 64 tokens with aligned rows: x and A go to LDS without passing registers,
// in steps of 128 bytes of K's x (64 bf16 or 64 codes and 32 fp32 values a row), three
// steps deep.  Eight neighbouring lanes load a row's 128 bytes: in the layout of the
// matrix instructions neighbouring lanes are different rows, and the cache then
// serves one lane a cycle (8192 x 7168 of bf16, rank 2 x 64: 89 us; this way 41, 2.9
// TB/s).  16-byte pieces are stored at piece ^ key(row), for the banks.
constexpr int RING = 3;

template <int KIND>
constexpr int step_k() { return KIND == ADAPT_F32 ? 32 : 64; }

// FR: fragments of 16 columns, a power of two
template <int FR, int KIND>
__global__ __launch_bounds__(256) void adapter_down_wide(AdapterPass p, int k_parts)
{
    constexpr int NS = terms<KIND>(), SK = step_k<KIND>(), XROW = KIND == ADAPT_I8 ? 64 : 128, AROW = SK * 2;
    constexpr int XB = 64 * XROW, AB = FR * 16 * AROW, LX = XB / 4096, LA = AB < 4096 ? 1 : AB / 4096;   // loads of a wave and step
    constexpr int CW = FR >= 4 ? 4 : FR, TW = 4 / CW, CT = FR / CW, TT = 4 / TW;       // waves along columns and tokens, fragments of a wave
    extern __shared__ __align__(16) int8_t ring[];                     // [RING][x, A]
    const Taken tile = take_tile<64>(p);
    if (tile.adapter < 0 || tile.count == 0) return;
    const int count = tile.count;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), r = lane & 15, g = lane >> 4;
    const int R = p.parts * p.rank, r8 = (p.rank + 7) & ~7, width = p.parts * r8;
    const int steps = (p.K + SK - 1) / SK, part = blockIdx.y;
    const int s0 = (int)((int64_t)steps * part / k_parts), s1 = (int)((int64_t)steps * (part + 1) / k_parts);
    constexpr int ES = KIND == ADAPT_F32 ? 4 : KIND == ADAPT_BF16 ? 2 : 1, STAGE = XB + AB;
    constexpr int XP = XROW / 16, AP = AROW / 16;                      // pieces of a row
    auto key = [](int row, int pieces) { return (row >> (pieces == 4 ? 1 : 0)) & (pieces - 1); };
    // what this lane loads: piece (lane % pieces) ^ key of row (wave, load, lane / pieces)
    const char *xp[LX];
    int xk[LX];
#pragma unroll
    for (int i = 0; i < LX; ++i) {
        const int row = ((wave * LX + i) * 64 + lane) / XP, piece = (lane % XP) ^ key(row, XP);
        xp[i] = (const char *)p.x + (int64_t)token_at(p, tile.begin + min(row, count - 1)) * p.ldx * ES;
        xk[i] = piece * (16 / ES);
    }
    const uint16_t *ap[LA];
    int ak[LA];
#pragma unroll
    for (int i = 0; i < LA; ++i) {
        const int row = (((wave * LA + i) * 64 + lane) / AP) % (FR * 16), piece = (lane % AP) ^ key(row, AP);
        ap[i] = p.a + ((int64_t)tile.adapter * R + min(row, R - 1)) * p.lda;
        ak[i] = piece * 8;
    }
    const int last_x = p.K - 16 / ES, last_a = ((p.K + 7) & ~7) - 8;
    auto fetch = [&](int s) {                    // past the end: the last step again, into a slot that nobody reads
        int8_t *const at = ring + s % RING * STAGE;
        const int k = SK * min(s, s1 - 1);
#pragma unroll
        for (int i = 0; i < LX; ++i)
            __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)(xp[i] + (int64_t)min(k + xk[i], last_x) * ES),
                                             (__attribute__((address_space(3))) void *)(at + (wave * LX + i) * 1024), 16, 0, 0);
#pragma unroll
        for (int i = 0; i < LA; ++i)
            __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)(ap[i] + min(k + ak[i], last_a)),
                                             (__attribute__((address_space(3))) void *)(at + XB + (wave * LA + i) * 1024 % AB), 16, 0, 0);
    };
    const int wc = wave % CW, wt = wave / CW;
    f32x4 acc[TT][CT];
#pragma unroll
    for (int i = 0; i < TT; ++i)
#pragma unroll
        for (int c = 0; c < CT; ++c) acc[i][c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    fetch(s0);
    fetch(s0 + 1);
    for (int s = s0; s < s1; ++s) {
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_waitcnt((LX + LA) | 0x70);                  // vmcnt: the next step may be on its way; lgkmcnt(0)
        __builtin_amdgcn_s_barrier();            // step s has landed for everybody, and step s - 1 is read
        asm volatile("" ::: "memory");
        fetch(s + 2);
        const int8_t *const xb = ring + s % RING * STAGE, *const ab = xb + XB;
#pragma unroll
        for (int h = 0; h < SK / 32; ++h) {
            const int k = 32 * h + 8 * g;        // of the step
            u32x4 w[CT];
#pragma unroll
            for (int c = 0; c < CT; ++c) {
                const int row = 16 * (wc + CW * c) + r;
                w[c] = *(const u32x4 *)(ab + row * AROW + 16 * ((k / 8) ^ key(row, AP)));
                if (SK * s + k > last_a) w[c] = u32x4{0, 0, 0, 0};     // past K
            }
#pragma unroll
            for (int i = 0; i < TT; ++i) {
                const int row = 16 * (wt + TW * i) + r;
                Raw v;
                if (KIND == ADAPT_F32) {
#pragma unroll
                    for (int q = 0; q < 2; ++q) v.u[q] = *(const u32x4 *)(xb + row * XROW + 16 * ((k / 4 + q) ^ key(row, XP)));
                } else if (KIND == ADAPT_BF16) v.u[0] = *(const u32x4 *)(xb + row * XROW + 16 * ((k / 8) ^ key(row, XP)));
                else {
                    const uint2 c = *(const uint2 *)(xb + row * XROW + 16 * ((k / 16) ^ key(row, XP)) + (k & 8));
                    v.u[0][0] = c.x;
                    v.u[0][1] = c.y;
                }
                bf16x8 a[3];
                as_terms<KIND>(v, a);
#pragma unroll
                for (int c = 0; c < CT; ++c)
#pragma unroll
                    for (int q = NS - 1; q >= 0; --q)                  // smallest term first
                        acc[i][c] = mfma16x16x32(a[q], __builtin_bit_cast(bf16x8, w[c]), acc[i][c]);
            }
        }
    }
    __builtin_amdgcn_s_waitcnt(0x0f70);          // no load may be in flight when the LDS is freed
#pragma unroll
    for (int c = 0; c < CT; ++c) {
        const int f = 16 * (wc + CW * c) + r;    // D: lane (r, g) holds tokens 4 g .. 4 g + 3 of column r
        if (f >= R) continue;
        float *const o = p.low + ((int64_t)part * p.T + tile.begin) * width + f / p.rank * r8 + f % p.rank;
#pragma unroll
        for (int i = 0; i < TT; ++i)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int t = 16 * (wt + TW * i) + 4 * g + q;
                if (t < count) o[(int64_t)t * width] = acc[i][c][q];
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
    const bool vec = aligned(p.x, p.ldx, es, std::min(16, 8 * es)) && p.K % 8 == 0;
    const dim3 grid((unsigned)adapter_tiles(p.T, p.n), (unsigned)parts);
    // rows whose 16-byte pieces are aligned
    if (tt == 4 && aligned(p.x, p.ldx, es, 16) && p.K % (16 / es) == 0) {
#define MOE_WIDE2(fr, kind)                                                                       \
    do {                                                                                          \
        static DevSlots slots{};                                                                  \
        const size_t ring = (size_t)RING * (64 * (kind == ADAPT_I8 ? 64 : 128) + fr * 16 * step_k<kind>() * 2); \
        const hipError_t e = lds_limit((const void *)adapter_down_wide<fr, kind>, slots, ring);   \
        if (e != hipSuccess) return e;                                                            \
        adapter_down_wide<fr, kind><<<grid, 256, ring, s>>>(p, parts);                            \
        return hipGetLastError();                                                                 \
    } while (0)
#define MOE_WIDE(fr)                                                                              \
    do {                                                                                          \
        if (p.kind == ADAPT_F32) MOE_WIDE2(fr, ADAPT_F32);                                        \
        else if (p.kind == ADAPT_BF16) MOE_WIDE2(fr, ADAPT_BF16);                                 \
        else MOE_WIDE2(fr, ADAPT_I8);                                                             \
    } while (0)
        if (frags <= 2) MOE_WIDE(2);
        else if (frags <= 4) MOE_WIDE(4);
        else if (frags <= 8) MOE_WIDE(8);
        else MOE_WIDE(16);
#undef MOE_WIDE
#undef MOE_WIDE2
    }
    const size_t lds = (size_t)(waves / cw / 2) * tt * frags * 64 * 16;
#define MOE_DOWN4(t, c, kind, v)                                                                  \
    do {                                                                                          \
        static DevSlots slots{};                                                                  \
        const hipError_t e = lds_limit((const void *)adapter_down<t, c, kind, v>, slots, lds);    \
        if (e != hipSuccess) return e;                                                            \
        adapter_down<t, c, kind, v><<<grid, 64 * waves, lds, s>>>(p, parts, cw);                  \
    } while (0)
// large tiles of aligned rows are the kernel's above, but for codes at multiples of 8 bytes
#define MOE_DOWN3(t, c, kind)                                                                     \
    do {                                                                                          \
        if constexpr (t == 1 || kind == ADAPT_I8) {                                               \
            if (vec) MOE_DOWN4(t, c, kind, true);                                                 \
            else MOE_DOWN4(t, c, kind, false);                                                    \
        } else MOE_DOWN4(t, c, kind, false);                                                      \
    } while (0)
#define MOE_DOWN2(t, kind)                                                                        \
    do {                                                                                          \
        if (ct == 1) MOE_DOWN3(t, 1, kind);                                                       \
        else if (ct == 2) MOE_DOWN3(t, 2, kind);                                                  \
        else MOE_DOWN3(t, 4, kind);                                                               \
    } while (0)
#define MOE_DOWN(t)                                                                               \
    do {                                                                                          \
        if (p.kind == ADAPT_F32) MOE_DOWN2(t, ADAPT_F32);                                         \
        else if (p.kind == ADAPT_BF16) MOE_DOWN2(t, ADAPT_BF16);                                  \
        else MOE_DOWN2(t, ADAPT_I8);                                                              \
    } while (0)
    if (tt == 1) MOE_DOWN(1);
    else MOE_DOWN(4);
#undef MOE_DOWN
#undef MOE_DOWN2
#undef MOE_DOWN3
#undef MOE_DOWN4
    return hipGetLastError();
}

hipError_t launch_adapter_up(const AdapterPass &p, hipStream_t s)
{
    const int parts = adapter_k_parts(p.T, p.K, p.n), es = p.y_bf16 ? 2 : 4;
    const int tiles = adapter_tiles(p.T, p.n), groups = (p.N / p.parts + WIDE - 1) / WIDE;
    // about two work-groups a CU, stretches of at least a group a wave (8192 x 4096, rank 64, with the down kernel 97 us; one a CU
    // 103, four 98, eight 110)
    const int chunks = std::max(1, std::min((groups + 3) / 4, (512 + tiles * p.parts - 1) / (tiles * p.parts)));
    const bool vec = aligned(p.y, p.ldy, es, 4 * es) && aligned(p.add, p.ldadd, es, 4 * es) && p.N / p.parts % 4 == 0;
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
