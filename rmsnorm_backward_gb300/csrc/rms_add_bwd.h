// rms_add_bwd.h -- parameter block and launch functions of the backward of
// the RMSNorm with a residual's addition (rms_add_bwd_kernels.cuh).
// Internal to libgbnorm.so.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "row_phase.h"

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
    // the ring kernel only
    int tpr;            // threads per row slot (multiple of 32)
    int slots;          // rows at once (16 warps hold slots * tpr threads at least)
    int stages;         // ring stages per slot
    int stat_rows;      // most rows of a CTA
    int nvec;           // 16-byte vectors that a row touches, at most
    int shift0, shift_step;
    int *err;
    uint64_t wait_ns;
};

// shared memory of the ring kernel: ring [slots][stages][3 rows of nvec
// vectors], reused for the combine of the slots' partial sums | gamma's
// vectors, where they are kept there | mbarriers [slots][stages] | rstd
// [stat_rows] | reduction scratch [slots][2][16] | abort flags [slots]
struct AddBwdLayout {
    size_t gam, bar, stat, red, flag, total;
};
__host__ __device__ inline AddBwdLayout add_bwd_layout(int slots, int stages, int nvec, int stat_rows, bool gamma) {
    AddBwdLayout L;
    L.gam = (size_t)slots * stages * 3 * nvec * 16;
    L.bar = L.gam + (gamma ? (size_t)nvec * 16 : 0);
    L.stat = L.bar + (size_t)slots * stages * 8;
    L.red = (L.stat + (size_t)stat_rows * 4 + 15) / 16 * 16;
    L.flag = L.red + (size_t)slots * 2 * 16 * 4;
    L.total = L.flag + (size_t)slots * 4;
    return L;
}
__host__ __device__ constexpr bool add_bwd_gamma_smem(size_t es, int nv) { return es == 2 && nv == 4; }

constexpr int kAddBwdThreads = 512;

// the longest rows of the short-row kernel, in 16-byte vectors and in
// elements, and the rows that a CTA of it takes at once
constexpr int kBwdShortVectors = 64, kBwdShortElements = 256;
inline int add_bwd_short_rows(bool vec, int N, int V) {
    if (!vec) return N <= 128 ? 32 : 16;
    const int nvec = N / V;
    return nvec <= 8 ? 128 : nvec <= 16 ? 64 : nvec <= 32 ? 32 : 16;
}
// vec: rows of whole 16-byte vectors, else element by element
cudaError_t launch_rms_add_bwd_short(int dtype, bool vec, const AddBwdParams &p, cudaStream_t s);
cudaError_t launch_rms_add_bwd_plain(int dtype, const AddBwdParams &p, cudaStream_t s);
// nv: vectors a thread owns (1 to 4; float32 also 6 and 8); shift: some row does
// not start or end on 16 bytes
cudaError_t launch_rms_add_bwd_ring(int dtype, int nv, bool shift, const AddBwdParams &p, size_t smem, cudaStream_t s);

}  // namespace gbn
