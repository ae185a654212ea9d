// dradd_rope.cu -- how the tokens of a rotary call are spread over CTAs
// (dradd_rope.cuh).
#include "dradd_train_internal.h"

#include "dradd_elem.cuh"

namespace dradd {

namespace {

constexpr int kSms = 152;  // a constant, not the device's count: partial sums follow the grid
constexpr int kFwdCtasPerSm = 12;
constexpr int kBwdCtasPerSm = 2;
// A token is split among warps until there are this many work items per SM
// (4096 tokens of 32 + 8 heads: unsplit 13.6 us, in two 14.4).
constexpr int kWorkPerSm = 16;

int lanes_for(int units)
{
    int g = 4;
    while (g < units)
        g *= 2;
    return g;
}

}  // namespace

void rope_plan(RopeArgs* a, bool backward, int* grid)
{
    a->rot_units = (a->rot + 15) / 16;
    a->units = a->rot_units + (a->dim - a->rot + 15) / 16;
    a->group = lanes_for(a->units);
    a->heads_per_step = 32 / a->group;
    a->q_steps = (a->q.heads + a->heads_per_step - 1) / a->heads_per_step;
    a->k_steps = (a->k.heads + a->heads_per_step - 1) / a->heads_per_step;
    const int64_t steps = a->q_steps + a->k_steps;
    int64_t split = (kWorkPerSm * kSms + a->tokens - 1) / a->tokens;
    if (split > steps)
        split = steps;
    a->steps_per_warp = static_cast<int>((steps + split - 1) / split);
    a->warps_per_token = static_cast<int>((steps + a->steps_per_warp - 1) / a->steps_per_warp);
    const int64_t work = a->tokens * a->warps_per_token;
    a->n_work = static_cast<uint32_t>(work);
    const int64_t ctas = (work + kRopeThreads / 32 - 1) / (kRopeThreads / 32);
    const int64_t most = static_cast<int64_t>(backward ? kBwdCtasPerSm : kFwdCtasPerSm) * kSms;
    *grid = static_cast<int>(ctas < most ? ctas : most);
}

cudaError_t launch_rope(const RopeArgs& a, int mode, int elem, bool interleaved, bool blocks, int grid,
                        cudaStream_t stream)
{
    return elem == kElemBf16  ? launch_rope_bf16(a, mode, interleaved, blocks, grid, stream)
           : elem == kElemF16 ? launch_rope_f16(a, mode, interleaved, blocks, grid, stream)
                              : launch_rope_f32(a, mode, interleaved, blocks, grid, stream);
}

}  // namespace dradd
