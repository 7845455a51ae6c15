// rms_out.cu -- dtype dispatch of the residual / 8-bit RMSNorm forward.
#include "rms_out.h"

namespace gbn {

cudaError_t launch_rms_out_plain_f32(int, bool, const OutParams &, int, cudaStream_t);
cudaError_t launch_rms_out_plain_f16(int, bool, const OutParams &, int, cudaStream_t);
cudaError_t launch_rms_out_plain_bf16(int, bool, const OutParams &, int, cudaStream_t);

cudaError_t launch_rms_out_plain(int dtype, int kind, bool group, const OutParams &p, int sms, cudaStream_t s) {
    switch (dtype) {
        case 0: return launch_rms_out_plain_f32(kind, group, p, sms, s);
        case 1: return launch_rms_out_plain_f16(kind, group, p, sms, s);
        case 2: return launch_rms_out_plain_bf16(kind, group, p, sms, s);
    }
    return cudaErrorInvalidValue;
}

cudaError_t launch_rms_out_ring_f32(int, int, const OutParams &, size_t, cudaStream_t);
cudaError_t launch_rms_out_ring_f16(int, int, const OutParams &, size_t, cudaStream_t);
cudaError_t launch_rms_out_ring_bf16(int, int, const OutParams &, size_t, cudaStream_t);

cudaError_t launch_rms_out_ring(int dtype, int nv, int lie, const OutParams &p, size_t smem, cudaStream_t s) {
    switch (dtype) {
        case 0: return launch_rms_out_ring_f32(nv, lie, p, smem, s);
        case 1: return launch_rms_out_ring_f16(nv, lie, p, smem, s);
        case 2: return launch_rms_out_ring_bf16(nv, lie, p, smem, s);
    }
    return cudaErrorInvalidValue;
}

cudaError_t launch_rms_out_short_f32(bool, const OutParams &, int, cudaStream_t);
cudaError_t launch_rms_out_short_f16(bool, const OutParams &, int, cudaStream_t);
cudaError_t launch_rms_out_short_bf16(bool, const OutParams &, int, cudaStream_t);

cudaError_t launch_rms_out_short(int dtype, bool vec, const OutParams &p, int sms, cudaStream_t s) {
    switch (dtype) {
        case 0: return launch_rms_out_short_f32(vec, p, sms, s);
        case 1: return launch_rms_out_short_f16(vec, p, sms, s);
        case 2: return launch_rms_out_short_bf16(vec, p, sms, s);
    }
    return cudaErrorInvalidValue;
}

}  // namespace gbn
