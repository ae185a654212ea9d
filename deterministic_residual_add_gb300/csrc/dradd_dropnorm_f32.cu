// dradd_dropnorm_f32.cu -- the kernels of dradd_dropnorm.cuh for f32 tensors.
#include "dradd_dropnorm.cuh"

namespace dradd {

cudaError_t launch_drop_norm_f32(const DropNormArgs& a, const DropNormPlan& p, bool backward, cudaStream_t stream)
{
    return launch_drop_norm_of<kElemF32>(a, p, backward, stream);
}

}  // namespace dradd
