// rms_add_bwd_f32.cu -- the backward kernels with the residual's gradient for float storage
// (templates in rms_add_bwd_kernels.cuh).
#include "rms_add_bwd_kernels.cuh"

namespace gbn {

cudaError_t launch_rms_add_bwd_plain_f32(const AddBwdParams &p, cudaStream_t s) {
    return rms_add_bwd_plain_dispatch<float>(p, s);
}

cudaError_t launch_rms_add_bwd_ring_f32(int nv, bool shift, const AddBwdParams &p, size_t smem, cudaStream_t s) {
    return rms_add_bwd_ring_dispatch<float>(nv, shift, p, smem, s);
}

cudaError_t launch_rms_add_bwd_short_f32(bool vec, const AddBwdParams &p, cudaStream_t s) {
    return rms_add_bwd_short_dispatch<float>(vec, p, s);
}

}  // namespace gbn
