// rms_out_bf16.cu -- the residual / 8-bit forward kernels for __nv_bfloat16 storage (templates in rms_out_kernels.cuh).
#include "rms_out_kernels.cuh"

namespace gbn {

cudaError_t launch_rms_out_plain_bf16(int kind, bool group, const OutParams &p, int sms, cudaStream_t s) {
    return rms_out_plain_dispatch<__nv_bfloat16>(kind, group, p, sms, s);
}

cudaError_t launch_rms_out_ring_bf16(int nv, int lie, const OutParams &p, size_t smem, cudaStream_t s) {
    return rms_out_ring_dispatch<__nv_bfloat16>(nv, lie, p, smem, s);
}

cudaError_t launch_rms_out_short_bf16(bool vec, const OutParams &p, int sms, cudaStream_t s) {
    return rms_out_short_dispatch<__nv_bfloat16>(vec, p, sms, s);
}

}  // namespace gbn
