// norm_bf16.cu -- the norms in bf16 (norm_launch.cuh).
#include "norm_launch.cuh"

namespace ccv3d {

void norm_forward_bf16(const NormFwd& p, cudaStream_t st) { norm_fwd_type<bf16_t>(p, st); }
void norm_backward_bf16(const NormBwd& p, const BwdShape& s, int form, const NormFin* f,
                        cudaStream_t st) {
    norm_backward_type<bf16_t>(p, s, form, f, st);
}
cudaError_t norm_status_bf16(int* v, cudaStream_t st) { return take_status(v, st); }

}  // namespace ccv3d
