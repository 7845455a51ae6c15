// rms_out_f32.cu -- the residual / 8-bit forward kernels for float storage (templates in rms_out_kernels.cuh).
#include "rms_out_kernels.cuh"

namespace gbn {

cudaError_t launch_rms_out_plain_f32(int kind, bool group, const OutParams &p, int sms, cudaStream_t s) {
    return rms_out_plain_dispatch<float>(kind, group, p, sms, s);
}

cudaError_t launch_rms_out_ring_f32(int nv, int lie, const OutParams &p, size_t smem, cudaStream_t s) {
    return rms_out_ring_dispatch<float>(nv, lie, p, smem, s);
}

cudaError_t launch_rms_out_short_f32(bool vec, const OutParams &p, int sms, cudaStream_t s) {
    return rms_out_short_dispatch<float>(vec, p, sms, s);
}

}  // namespace gbn
