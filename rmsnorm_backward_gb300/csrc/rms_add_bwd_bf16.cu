// rms_add_bwd_bf16.cu -- the backward kernels with the residual's gradient for __nv_bfloat16 storage
// (templates in rms_add_bwd_kernels.cuh).
#include "rms_add_bwd_kernels.cuh"

namespace gbn {

cudaError_t launch_rms_add_bwd_plain_bf16(const AddBwdParams &p, cudaStream_t s) {
    return rms_add_bwd_plain_dispatch<__nv_bfloat16>(p, s);
}

cudaError_t launch_rms_add_bwd_ring_bf16(int nv, bool shift, const AddBwdParams &p, size_t smem, cudaStream_t s) {
    return rms_add_bwd_ring_dispatch<__nv_bfloat16>(nv, shift, p, smem, s);
}

cudaError_t launch_rms_add_bwd_short_bf16(bool vec, const AddBwdParams &p, cudaStream_t s) {
    return rms_add_bwd_short_dispatch<__nv_bfloat16>(vec, p, s);
}

}  // namespace gbn
