// dradd_rope.cu -- how the tokens of a rotary call are spread over CTAs
// (dradd_rope.cuh).
#include "dradd_train_internal.h"

#include "dradd_elem.cuh"

namespace dradd {

namespace {

constexpr int kSms = 152;  // a constant, not the device's count: partial sums follow the grid
constexpr int kAngleBytes = 16 * 1024;
constexpr int kBwdCtasPerSm = 2;

int lanes_for(int units)
{
    int g = 1;
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
    // Enough tokens for about four heads a group, so that the angles' cost
    // is shared, but no fewer CTAs than about six per SM.
    const int heads = a->q.heads + a->k.heads;
    const int groups = kRopeThreads / a->group;
    int64_t step = (4 * groups + heads - 1) / heads;
    const int64_t room = kAngleBytes / (a->rot_units * 64);
    const int64_t spread = a->tokens / (6 * kSms);
    if (step > room)
        step = room;
    if (step > spread)
        step = spread;
    if (step < 1)
        step = 1;
    a->tokens_per_step = static_cast<int>(step);
    int64_t ctas = (a->tokens + step - 1) / step;
    if (backward && ctas > kBwdCtasPerSm * kSms)
        ctas = kBwdCtasPerSm * kSms;
    *grid = static_cast<int>(ctas);
}

cudaError_t launch_rope(const RopeArgs& a, int mode, int elem, bool interleaved, bool blocks, int grid,
                        cudaStream_t stream)
{
    return elem == kElemBf16  ? launch_rope_bf16(a, mode, interleaved, blocks, grid, stream)
           : elem == kElemF16 ? launch_rope_f16(a, mode, interleaved, blocks, grid, stream)
                              : launch_rope_f32(a, mode, interleaved, blocks, grid, stream);
}

}  // namespace dradd
