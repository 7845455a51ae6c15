// grad_clip.h -- tables and launch functions of the global gradient norm and
// the clip (grad_clip.cu).  Internal to libgbnorm.so.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "gbnorm.h"

namespace gbn {

constexpr int kGradThreads = 256;
constexpr int kGradVecs = 8;                                 // 16-byte vectors a thread takes of a chunk
constexpr int kGradChunkVecs = kGradThreads * kGradVecs;     // 32 KiB
constexpr int kGradCtasPerSm = 4;

// a CTA's sums of squares, float32 pairs each: ordinary ones, and those scaled
// by 2^-160 (big) and 2^160 (small)
struct alignas(16) GradSums {
    float hi, lo, big, small, big_lo, small_lo;
};

// CTAs for `chunks` chunks in all; the workspace has a GradSums for each
inline int grad_grid(int64_t chunks, int sms) {
    const int64_t most = static_cast<int64_t>(sms) * kGradCtasPerSm;
    return static_cast<int>(chunks < 1 ? 1 : chunks < most ? chunks : most);
}

cudaError_t launch_grad_norm(const gbn_tensor *g, int64_t count, float *norm, GradSums *partial, int sms,
                             cudaStream_t s);
cudaError_t launch_grad_clip(const gbn_tensor *g, const gbn_tensor *out, int64_t count, float max_norm, float eps,
                             float *norm, GradSums *partial, int sms, cudaStream_t s);

}  // namespace gbn
