// rms_add_bwd_kernels.cuh -- backward of the RMSNorm with a residual's
// addition, for sm_103a; instantiated once per storage dtype in
// rms_add_bwd_f32.cu, rms_add_bwd_f16.cu and rms_add_bwd_bf16.cu.
//
// Per row, with xhat = h*rstd (recomputed from the saved rstd) and dyhat =
// dy*gamma:
//   dx = rstd*(dyhat - xhat*mean(dyhat*xhat)) + dh,
//   dgamma[j] = sum over rows of dy*xhat.
// The sum with dh is float32, before the one rounding to the storage type.
// dgamma takes the partial rows and the fixed-order column reduce of the
// other backward kernels: no atomics, the same bits from run to run.
#pragma once

#include "gbn_device.cuh"
#include "rms_add_bwd.h"

namespace gbn {

// ---------------------------------------------------------------------------
// any N, stride and alignment: CTA b takes a contiguous block of rows, with
// scalar accesses; its partial row in global memory is the accumulator
// (column j always by thread j mod 256: a fixed order per column)
// ---------------------------------------------------------------------------
template <typename T>
__global__ void __launch_bounds__(kGenericThreads) rms_add_bwd_plain_kernel(const AddBwdParams p) {
    using Tr = Traits<T>;
    __shared__ float sm[kGenericThreads / 32];
    const int N = p.N;
    const float inv_n = 1.0f / static_cast<float>(N);
    int64_t row0;
    int nrows;
    block_rows(p.M, p.G, blockIdx.x, row0, nrows);
    float *pg = p.part + (size_t)blockIdx.x * p.ldp;
    for (int j = threadIdx.x; j < N; j += blockDim.x) pg[j] = 0.f;
    const T *g = static_cast<const T *>(p.gamma);
    for (int i = 0; i < nrows; ++i) {
        const int64_t row = row0 + i;
        const T *h = static_cast<const T *>(p.h) + row * p.ld_h;
        const T *dy = static_cast<const T *>(p.dy) + row * p.ld_dy;
        const T *dh = static_cast<const T *>(p.dh) + row * p.ld_dh;
        T *dx = static_cast<T *>(p.dx) + row * p.ld_dx;
        const float rs = p.rstd[row];
        float s = 0.f;
        for (int j = threadIdx.x; j < N; j += blockDim.x)
            s = fmaf(Tr::load1(dy + j) * Tr::load1(g + j), Tr::load1(h + j) * rs, s);
        const float a = -rs * (block_sum(s, sm) * inv_n);
        for (int j = threadIdx.x; j < N; j += blockDim.x) {
            const float xhat = Tr::load1(h + j) * rs, d = Tr::load1(dy + j);
            const float o = fmaf(d * Tr::load1(g + j), rs, xhat * a) + Tr::load1(dh + j);
            pg[j] = fmaf(d, xhat, pg[j]);
            Tr::store1(dx + j, o);
        }
    }
}

template <typename T>
cudaError_t rms_add_bwd_plain_dispatch(const AddBwdParams &p, cudaStream_t s) {
    rms_add_bwd_plain_kernel<T><<<p.G, kGenericThreads, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace gbn
