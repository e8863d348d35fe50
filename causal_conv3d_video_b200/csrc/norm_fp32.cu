// norm_fp32.cu -- the norms in fp32 (norm_launch.cuh).
#include "norm_launch.cuh"

namespace ccv3d {

void norm_forward_fp32(const NormFwd& p, cudaStream_t st) { norm_fwd_type<float>(p, st); }
void norm_backward_fp32(const NormBwd& p, const BwdShape& s, int form, const NormFin* f,
                        cudaStream_t st) {
    norm_backward_type<float>(p, s, form, f, st);
}
cudaError_t norm_status_fp32(int* v, cudaStream_t st) { return take_status(v, st); }

}  // namespace ccv3d
