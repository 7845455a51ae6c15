// rms_add_bwd.h -- parameter block and launch functions of the backward of
// the RMSNorm with a residual's addition (rms_add_bwd_kernels.cuh).
// Internal to libgbnorm.so.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace gbn {

struct AddBwdParams {
    const void *dy;
    const void *dh;     // the gradient that reaches h beside the norm
    const void *h;
    const void *gamma;
    const float *rstd;
    void *dx;
    float *part;        // [G][ldp] dgamma partial rows
    int64_t M;
    int N;
    int ldp;            // row stride of the partial rows, in floats (multiple of 4)
    int G;
    int64_t ld_dy, ld_dh, ld_h, ld_dx;  // row strides, in elements
};

cudaError_t launch_rms_add_bwd_plain(int dtype, const AddBwdParams &p, cudaStream_t s);

}  // namespace gbn
