// dradd_rope.cu -- how the tokens of a rotary call are spread over CTAs
// (dradd_rope.cuh).
#include "dradd_elem.cuh"
#include "dradd_train_internal.h"

namespace dradd {

namespace {

constexpr int kSms = 152;  // a constant, not the device's count: partial sums follow the grid
// CTAs an SM holds at once.
constexpr int kFwdCtasPerSm = 4;
constexpr int kFwdCtasPerSmF32 = 3;
constexpr int kBwdCtasPerSm = 2;

int lanes_for(int units)
{
    int g = 4;
    while (g < units)
        g *= 2;
    return g;
}

// Steps a warp takes so that the warps that are resident at once take all.
int64_t share_of(int64_t n_steps, int64_t resident) { return (n_steps + resident - 1) / resident; }

}  // namespace

void rope_plan(RopeArgs* a, int elem, bool backward, int* grid)
{
    a->rot_units = (a->rot + 15) / 16;
    a->units = a->rot_units + (a->dim - a->rot + 15) / 16;
    a->group = lanes_for(a->units);
    const int lane_groups = 32 / a->group;
    const int ctas = backward ? kBwdCtasPerSm : elem == kElemF32 ? kFwdCtasPerSmF32 : kFwdCtasPerSm;
    const int64_t resident = static_cast<int64_t>(kSms) * ctas * (kRopeThreads / 32);
    // A warp's lane groups take heads of one token, or, where that leaves
    // lanes idle and costs two steps or more of a share, a token each: bf16
    // 13036 tokens of 2 + 2 heads of 128 8.4 us against 12.6, 8192 of 7 + 1 of
    // 32 (2 steps a warp against 4) 6.3 against 8.1, its gradients 10.7
    // against 14.3; 4096 of 4 + 1 of 128 (2 against 2) 8.7 against 5.8.
    const int64_t q_whole = (a->q.heads + lane_groups - 1) / lane_groups;
    const int64_t k_whole = (a->k.heads + lane_groups - 1) / lane_groups;
    const int64_t groups = (a->tokens + lane_groups - 1) / lane_groups;
    const int64_t share_whole = share_of(a->tokens * (q_whole + k_whole), resident);
    const int64_t share_groups = share_of(groups * (a->q.heads + a->k.heads), resident);
    a->by_token = lane_groups > 1 && share_groups + 1 < share_whole;
    a->heads_per_step = a->by_token ? 1 : lane_groups;
    a->q_steps = a->by_token ? a->q.heads : static_cast<int>(q_whole);
    a->k_steps = a->by_token ? a->k.heads : static_cast<int>(k_whole);
    const int64_t steps = a->q_steps + a->k_steps;
    a->n_steps = (a->by_token ? groups : a->tokens) * steps;
    int64_t share = a->by_token ? share_groups : share_whole;
    // A share that saves no more than a step of a token's is not worth the
    // angles of two tokens: bf16 2048 tokens of 8 + 1 heads 4.4 us against
    // 6.3, 4096 of 32 + 8 13.0 against 13.1.  Over several tokens a lane
    // group it is: 13036 of 2 + 2 8.4 against 9.9.
    if (share < steps && share + 1 >= steps && !a->by_token)
        share = steps;
    // Forward, a long share has its warps at tokens far apart; shorter ones of
    // whole tokens, more than are resident at once, keep them together:
    // 20000 tokens of 32 + 8 heads bf16 64.4 us against 74.9, 8192 28.4
    // against 29.0.
    constexpr int64_t kLongShare = 16;
    if (!backward && share > kLongShare)
        share = steps < kLongShare ? kLongShare / steps * steps : steps;
    a->steps_per_warp = static_cast<int>(share);
    const int64_t warps = share_of(a->n_steps, share);
    *grid = static_cast<int>((warps + kRopeThreads / 32 - 1) / (kRopeThreads / 32));
}

cudaError_t launch_rope(const RopeArgs& a, int mode, int elem, bool interleaved, bool blocks, int grid,
                        cudaStream_t stream)
{
    return elem == kElemBf16  ? launch_rope_bf16(a, mode, interleaved, blocks, grid, stream)
           : elem == kElemF16 ? launch_rope_f16(a, mode, interleaved, blocks, grid, stream)
                              : launch_rope_f32(a, mode, interleaved, blocks, grid, stream);
}

}  // namespace dradd
