// rms_add_bwd.cu -- dtype dispatch of the backward with the residual's gradient.
#include "rms_add_bwd.h"

namespace gbn {

cudaError_t launch_rms_add_bwd_plain_f32(const AddBwdParams &, cudaStream_t);
cudaError_t launch_rms_add_bwd_plain_f16(const AddBwdParams &, cudaStream_t);
cudaError_t launch_rms_add_bwd_plain_bf16(const AddBwdParams &, cudaStream_t);

cudaError_t launch_rms_add_bwd_plain(int dtype, const AddBwdParams &p, cudaStream_t s) {
    switch (dtype) {
        case 0: return launch_rms_add_bwd_plain_f32(p, s);
        case 1: return launch_rms_add_bwd_plain_f16(p, s);
        case 2: return launch_rms_add_bwd_plain_bf16(p, s);
    }
    return cudaErrorInvalidValue;
}

cudaError_t launch_rms_add_bwd_ring_f32(int, bool, const AddBwdParams &, size_t, cudaStream_t);
cudaError_t launch_rms_add_bwd_ring_f16(int, bool, const AddBwdParams &, size_t, cudaStream_t);
cudaError_t launch_rms_add_bwd_ring_bf16(int, bool, const AddBwdParams &, size_t, cudaStream_t);

cudaError_t launch_rms_add_bwd_ring(int dtype, int nv, bool shift, const AddBwdParams &p, size_t smem,
                                    cudaStream_t s) {
    switch (dtype) {
        case 0: return launch_rms_add_bwd_ring_f32(nv, shift, p, smem, s);
        case 1: return launch_rms_add_bwd_ring_f16(nv, shift, p, smem, s);
        case 2: return launch_rms_add_bwd_ring_bf16(nv, shift, p, smem, s);
    }
    return cudaErrorInvalidValue;
}

cudaError_t launch_rms_add_bwd_short_f32(bool, const AddBwdParams &, cudaStream_t);
cudaError_t launch_rms_add_bwd_short_f16(bool, const AddBwdParams &, cudaStream_t);
cudaError_t launch_rms_add_bwd_short_bf16(bool, const AddBwdParams &, cudaStream_t);

cudaError_t launch_rms_add_bwd_short(int dtype, bool vec, const AddBwdParams &p, cudaStream_t s) {
    switch (dtype) {
        case 0: return launch_rms_add_bwd_short_f32(vec, p, s);
        case 1: return launch_rms_add_bwd_short_f16(vec, p, s);
        case 2: return launch_rms_add_bwd_short_bf16(vec, p, s);
    }
    return cudaErrorInvalidValue;
}

}  // namespace gbn
