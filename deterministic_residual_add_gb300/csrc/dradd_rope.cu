// dradd_rope.cu -- how the tokens of a rotary call are spread over CTAs
// (dradd_rope.cuh).
#include "dradd_elem.cuh"
#include "dradd_train_internal.h"

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

// Whether the lane groups of a warp take one head each of as many tokens,
// instead of several heads of one token (`whole` steps a token): where more
// than a fifth of the lanes would idle, and tokens are enough.  bf16 13036
// tokens of 2 + 2 heads of 128 9.7 us against 12.6, 32768 of 7 + 1 of 32 13.3
// against 25.2; 16384 of 8 + 2 of 64 at 13.5 items per SM 12.5 against 15.1;
// fp32 8192 of 4 + 1 of 128, also 13.5, 16.3 against 15.5.
bool by_token(int64_t tokens, int heads, int whole, int lane_groups, int elem)
{
    const int64_t least = (elem == kElemF32 ? 16 : 8) * kSms;
    return 4 * whole * lane_groups > 5 * heads && tokens >= lane_groups * least;
}

}  // namespace

void rope_plan(RopeArgs* a, int elem, bool backward, int* grid)
{
    a->rot_units = (a->rot + 15) / 16;
    a->units = a->rot_units + (a->dim - a->rot + 15) / 16;
    a->group = lanes_for(a->units);
    const int lane_groups = 32 / a->group;
    const int heads = a->q.heads + a->k.heads;
    const int whole = (a->q.heads + lane_groups - 1) / lane_groups + (a->k.heads + lane_groups - 1) / lane_groups;
    a->by_token = by_token(a->tokens, heads, whole, lane_groups, elem);
    a->heads_per_step = a->by_token ? 1 : lane_groups;
    a->q_steps = a->by_token ? a->q.heads : (a->q.heads + lane_groups - 1) / lane_groups;
    a->k_steps = a->by_token ? a->k.heads : (a->k.heads + lane_groups - 1) / lane_groups;
    const int64_t items = a->by_token ? (a->tokens + lane_groups - 1) / lane_groups : a->tokens;
    const int64_t steps = a->q_steps + a->k_steps;
    int64_t split = (kWorkPerSm * kSms + items - 1) / items;
    if (split > steps)
        split = steps;
    a->steps_per_warp = static_cast<int>((steps + split - 1) / split);
    a->warps_per_item = static_cast<int>((steps + a->steps_per_warp - 1) / a->steps_per_warp);
    const int64_t work = items * a->warps_per_item;
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
