// rms_add_bwd_f16.cu -- the backward kernels with the residual's gradient for __half storage
// (templates in rms_add_bwd_kernels.cuh).
#include "rms_add_bwd_kernels.cuh"

namespace gbn {

cudaError_t launch_rms_add_bwd_plain_f16(const AddBwdParams &p, cudaStream_t s) {
    return rms_add_bwd_plain_dispatch<__half>(p, s);
}

cudaError_t launch_rms_add_bwd_ring_f16(int nv, bool shift, const AddBwdParams &p, size_t smem, cudaStream_t s) {
    return rms_add_bwd_ring_dispatch<__half>(nv, shift, p, smem, s);
}

cudaError_t launch_rms_add_bwd_short_f16(bool vec, const AddBwdParams &p, cudaStream_t s) {
    return rms_add_bwd_short_dispatch<__half>(vec, p, s);
}

}  // namespace gbn
