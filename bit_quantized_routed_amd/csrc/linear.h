// Launcher of the int8 linear layer (csrc/linear.hip).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moe {

struct LinearPass {
    int T, N, K;
    const int8_t *x, *w;
    int64_t ldx, ldw;
    const float *x_scale, *w_scale, *bias;       // bias may be null
    const void *add;                             // may be null
    void *y;
    int64_t ldadd, ldy;
    int y_bf16;
    void *ws;
};

size_t linear_ws_bytes(int T, int N, int K);     // enough for up to T tokens
bool linear_needs_ws(int T, int N, int K);       // whether T tokens use it
hipError_t launch_linear(const LinearPass &p, hipStream_t s);

}  // namespace moe
