// Arguments of the layer norm launchers (checked by the C entry points).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace fc {

struct LnForward {
    const void *x;
    int64_t rows, cols, ldx;
    const void *weight, *bias;
    int ptype;  // type of weight and bias
    float eps;
    void *y;
    int64_t ldy;
    float *mean, *rstd;
};

struct LnBackward {
    const void *dy;
    int64_t lddy;
    const void *x;
    int64_t ldx;
    const void *weight;
    int ptype;
    const float *mean, *rstd;
    int64_t rows, cols;
    void *dx;
    int64_t lddx;
    void *dweight, *dbias;
    int gtype;        // type of dweight and dbias
    float *partials;  // [2][parts][cols]; NULL if no sum is wanted
};

// Sets of column sums that the backward pass leaves at most.
int64_t ln_max_parts(int64_t rows, int64_t cols);

cudaError_t launch_ln_forward(const LnForward &a, int type, cudaStream_t s);
cudaError_t launch_ln_backward(const LnBackward &a, int type, cudaStream_t s);

}  // namespace fc
