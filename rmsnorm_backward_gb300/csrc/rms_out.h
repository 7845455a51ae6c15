// rms_out.h -- parameter block and launch functions of the RMSNorm forward
// with a residual's addition and / or an 8-bit output (rms_out_kernels.cuh).
// Internal to libgbnorm.so.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace gbn {

// what the rows are written as
enum OutKind : int { kOutSame = 0, kOutE4M3 = 1, kOutInt8 = 2 };

// columns that share a scale where the scales are by group
constexpr int kQuantGroup = 128;

struct OutParams {
    const void *x;
    const void *res;    // the residual, or nullptr: h is x itself and is not written
    const void *gamma;
    void *h;            // x + residual in the storage type (with a residual)
    void *out;          // y in the storage type, or the 8-bit codes
    float *rstd;
    float *scale;       // 8-bit outputs: [M], or [M][ceil(N / kQuantGroup)]
    float eps;
    int64_t M;
    int N;
    int64_t ld_x, ld_res, ld_h, ld_out;  // row strides, in elements
};

cudaError_t launch_rms_out_plain(int dtype, int kind, bool group, const OutParams &p, int sms, cudaStream_t s);

}  // namespace gbn
