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

}  // namespace gbn
