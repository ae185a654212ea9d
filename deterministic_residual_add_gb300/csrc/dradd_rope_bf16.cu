// dradd_rope_bf16.cu -- the kernels of dradd_rope.cuh for bf16 tensors.
#include "dradd_rope.cuh"

namespace dradd {

cudaError_t launch_rope_bf16(const RopeArgs& a, int mode, bool interleaved, bool blocks, int grid, cudaStream_t stream)
{
    return launch_rope_of<kElemBf16>(a, mode, interleaved, blocks, grid, stream);
}

}  // namespace dradd
