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
    // the ring kernel only
    int kind;            // OutKind
    int group;           // scales by groups of kQuantGroup columns
    int G;               // CTAs
    int cta_step, slot_step;  // slot q of CTA b takes rows b*cta_step + q*slot_step + k*G*slots
    int tpr;             // threads per row slot (multiple of 32)
    int slots;           // rows at once
    int stages;          // ring stages per slot
    int nvec;            // 16-byte vectors that a row touches, at most
    int shift0, shift_step;  // row_shift's (row_phase.h)
    int late;            // a stage is refilled once the next one has landed, not before
    int codes_aligned;   // a vector's codes can be stored at once
    int *err;
};

// shared memory of the ring kernel: ring [slots][stages][1 or 2 rows of nvec
// vectors] | mbarriers [slots][stages] | sums and maxima [slots][2][2][16] |
// group maxima [slots][3][groups] (kLieAcross) | abort flags [slots]
struct OutLayout {
    size_t bar, red, gmax, flag, total;
};
__host__ __device__ inline OutLayout out_layout(int slots, int stages, int streams, int nvec, int groups) {
    OutLayout L;
    L.bar = (size_t)slots * stages * streams * nvec * 16;
    L.red = (L.bar + (size_t)slots * stages * 8 + 15) / 16 * 16;
    L.gmax = L.red + (size_t)slots * 4 * 16 * 4;
    L.flag = L.gmax + (size_t)slots * 3 * groups * 4;
    L.total = L.flag + (size_t)slots * 4;
    return L;
}

constexpr int kOutThreads = 512;

// the longest rows of the short-row kernel, in 16-byte vectors and in elements
constexpr int kShortVectors = 64, kShortElements = 512;

// how rows lie to 16-byte boundaries (rms_out_kernels.cuh)
enum RowLie : int { kLieFull = 0, kLieWhole = 1, kLieAcross = 2, kLieShift = 3 };

// nv: vectors a thread owns (1 to 4; float32 also 6 and 8)
cudaError_t launch_rms_out_ring(int dtype, int nv, int lie, const OutParams &p, size_t smem, cudaStream_t s);
// vec: rows of whole 16-byte vectors (their codes on V), else element by element
cudaError_t launch_rms_out_short(int dtype, bool vec, const OutParams &p, int sms, cudaStream_t s);
cudaError_t launch_rms_out_plain(int dtype, int kind, bool group, const OutParams &p, int sms, cudaStream_t s);

}  // namespace gbn
