// dradd_dropnorm_f16.cu -- the kernels of dradd_dropnorm.cuh for f16 tensors.
#include "dradd_dropnorm.cuh"

namespace dradd {

cudaError_t launch_drop_norm_f16(const DropNormArgs& a, const DropNormPlan& p, bool backward, cudaStream_t stream)
{
    return launch_drop_norm_of<kElemF16>(a, p, backward, stream);
}

}  // namespace dradd
