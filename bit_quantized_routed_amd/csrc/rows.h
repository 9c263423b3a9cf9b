// Launchers of the row kernels (csrc/rows.hip): residual + norm, and rows to int8.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moe {

enum { ROWS_NORM = 0, ROWS_QUANT = 1, ROWS_SWIGLU = 2 };
constexpr int ROWS_MAX = 65536;                  // elements of a row

struct RowsPass {
    int mode, T, n;                              // rows, elements of an output row
    const void *x, *res;                         // res may be null
    int x_bf16, res_bf16, out_bf16;
    int64_t ldx, ldres, ldsum, ldout, ldq;
    void *sum, *out;                             // may be null
    int8_t *q;                                   // may be null
    float *q_scale;
    const float *weight;
    float eps;
};

hipError_t launch_rows(const RowsPass &p, hipStream_t s);

}  // namespace moe
