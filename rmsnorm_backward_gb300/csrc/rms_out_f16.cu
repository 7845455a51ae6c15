// rms_out_f16.cu -- the residual / 8-bit forward kernels for __half storage (templates in rms_out_kernels.cuh).
#include "rms_out_kernels.cuh"

namespace gbn {

cudaError_t launch_rms_out_plain_f16(int kind, bool group, const OutParams &p, int sms, cudaStream_t s) {
    return rms_out_plain_dispatch<__half>(kind, group, p, sms, s);
}

cudaError_t launch_rms_out_ring_f16(int nv, int lie, const OutParams &p, size_t smem, cudaStream_t s) {
    return rms_out_ring_dispatch<__half>(nv, lie, p, smem, s);
}

cudaError_t launch_rms_out_short_f16(bool vec, const OutParams &p, int sms, cudaStream_t s) {
    return rms_out_short_dispatch<__half>(vec, p, sms, s);
}

}  // namespace gbn
