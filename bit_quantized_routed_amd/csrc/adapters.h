// Launchers of the low-rank adapters (csrc/adapters.hip).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moe {

enum { ADAPT_F32 = 0, ADAPT_BF16 = 1, ADAPT_I8 = 2 };
constexpr int ADAPT_MAX = 1024, ADAPT_MAX_T = 1 << 20, ADAPT_MAX_RANK = 64, ADAPT_MAX_WIDTH = 256;

// A tile: up to adapter_tile(T) tokens of one adapter, consecutive in the plan's order.
struct AdapterTile { int32_t adapter, begin; };  // adapter -1: tokens that have none

struct AdapterPass {
    int T, K, N, n, rank, parts;                 // tokens, features in and out, adapters, rank of a part
    int kind;                                    // of x
    const void *x;
    const float *x_scale;                        // of codes
    const uint16_t *a, *b;                       // [n][parts * rank] rows lda apart, [n][N] rows ldb apart
    const float *scale;                          // [n]
    const void *add;                             // may be y
    void *y;
    int64_t ldx, lda, ldb, ldadd, ldy;
    int y_bf16;
    const int32_t *order, *offsets;
    const AdapterTile *tiles;
    float *low;                                  // workspace: [parts of K][T, in the plan's order][parts][rank up to a multiple of 8]
};

// Small tiles waste fewer rows where an adapter has few tokens, large ones read its matrices less often.  512 tokens take 17 to 19 us in
// tiles of 16 and 20 to 26 in tiles of 64 (7168 -> 4096 with rank 2 x 16 and codes of 2048 -> 7168 with rank 32), with rank 2 x 64 33
// and 34 to 49; 2048 tokens 33 to 38 and 32 to 41, with rank 2 x 64 68 to 74 and 43 to 47.  Between them it hangs on the adapters:
// 1024 tokens 22 to 26 and 28 to 31, with rank 2 x 64 39 and 46 (8 adapters in runs) or 50 and 40 (32, mixed).
inline int adapter_tile(int T) { return T <= 512 ? 16 : 64; }
// at most so many tiles, with those of tokens without an adapter
inline int adapter_tiles(int T, int n) { return T / adapter_tile(T) + (T < n + 1 ? T : n + 1); }
int adapter_k_parts(int T, int K, int n);
size_t adapter_low_bytes(int T, int K, int width, int n);              // of `low` for any batch of up to T tokens

hipError_t launch_adapter_plan(const int32_t *ids, int T, int n, int32_t *order, int32_t *offsets, AdapterTile *tiles, hipStream_t s);
hipError_t launch_adapter_down(const AdapterPass &p, hipStream_t s);
hipError_t launch_adapter_up(const AdapterPass &p, hipStream_t s);

}  // namespace moe
