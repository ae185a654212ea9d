// dradd_train_internal.h -- argument blocks and launchers of the dropout, RMSNorm
// gradient and rotary kernels, shared by the C-ABI layer and the kernels.
// Not part of the public interface.
#pragma once

#include <atomic>
#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "dradd_philox.cuh"

namespace dradd {

// Lets kernel FN use all the dynamic shared memory a CTA may have on the
// current device, once per kernel and device.  The limit belongs to the
// kernel, which serves calls of many sizes from many threads: set to what
// one call needs, it would refuse a larger call made at the same time.
template <auto FN>
cudaError_t allow_all_shared()
{
    static std::atomic<uint64_t> done{0};  // a bit per device
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    const uint64_t bit = dev >= 0 && dev < 64 ? 1ull << dev : 0;
    if (done.load(std::memory_order_acquire) & bit)
        return cudaSuccess;
    int optin = 0;
    e = cudaDeviceGetAttribute(&optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev);
    if (e != cudaSuccess)
        return e;
    const void* const fn = reinterpret_cast<const void*>(FN);
    cudaFuncAttributes attr;
    e = cudaFuncGetAttributes(&attr, fn);
    if (e != cudaSuccess)
        return e;
    e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             optin - static_cast<int>(attr.sharedSizeBytes));
    if (e != cudaSuccess)
        return e;
    done.fetch_or(bit, std::memory_order_acq_rel);
    return cudaSuccess;
}

// ------------------------------------------------------------------ dropout
// Row strides in elements.  residual NULL: plain dropout.
struct DropoutArgs {
    void* out;
    const void* x;
    const void* residual;
    int64_t out_stride, x_stride, residual_stride;
    int64_t n_rows, hidden;
    DropParams drop;
};

// Threads per CTA, and CTAs launched per SM at most: two waves of the sixteen
// that fit at once.  8192 x 4096 bf16 with 256 threads: 16 CTAs per SM 21.5
// us, 64 22.2, 128 24.3; with 128: 32 21.5.  The flat kernel, 8192 x 4097: 256
// threads 29.6, 128 28.5.
constexpr int kDropoutThreads = 128;
constexpr int kDropoutCtasPerSm = 32;

// Blocks: hidden, strides and addresses let every row move as aligned blocks
// of 8 elements.  Flat: contiguous 16-byte aligned tensors, at least
// kFlatHidden wide.  Ragged: anything.
enum DropoutLayout : int { kDropoutBlocks = 0, kDropoutFlat = 1, kDropoutRagged = 2 };
constexpr int64_t kFlatHidden = 8;
cudaError_t launch_dropout(const DropoutArgs& a, int elem, DropoutLayout layout, int sm_count, cudaStream_t stream);

// ------------------------------------- dropout + residual add + RMSNorm
struct DropNormArgs {
    void* out;           // forward: the normalised rows
    void* residual_out;  // forward: acc rounded
    const void* x;
    const void* residual;
    const void* weight;
    // backward
    void* dx;               // or NULL
    void* dresidual;
    float* partials;        // parts x hidden sums of dweight, or NULL
    const void* dout;
    const void* dresidual_out;  // or NULL (zero)
    const void* h;              // the forward's residual_out
    int64_t n_rows;
    int hidden;
    float inv_hidden;  // 1 / hidden if a power of two, else 0
    float eps;
    DropParams drop;  // threshold 0: no generator call
    int stages;       // staged kernels: rows in flight per CTA
    unsigned* status;
    uint64_t wait_limit_ns;
};

// The rings of the narrow-row kernels: N tensors (forward 2, backward 3), K
// blocks of 8 a lane, 256 threads.  CTAs an SM, and slots: as many as those
// CTAs have room for, two to four.
constexpr uint32_t narrow_slot_bytes(int elem, int n, int K)
{
    return static_cast<uint32_t>(n * K * (elem == 2 ? 2 : 1)) * 256u * 16u;
}
constexpr int narrow_ctas(int elem, int n, int K)
{
    const uint32_t two = 2 * narrow_slot_bytes(elem, n, K);
    const int most = n == 2 ? 4 : 2;  // what the registers allow
    const int fit = static_cast<int>(220u * 1024u / two);
    return fit < most ? fit : most;
}
constexpr int narrow_slots(int elem, int n, int K)
{
    const int fit =
        static_cast<int>(220u * 1024u / (narrow_ctas(elem, n, K) * narrow_slot_bytes(elem, n, K)));
    return fit > 4 ? 4 : fit;
}
constexpr uint32_t narrow_ring_bytes(int elem, int n, int K)
{
    return narrow_slots(elem, n, K) * narrow_slot_bytes(elem, n, K);
}

// Backward, two blocks a thread: CTAs of up to this many threads run two to
// an SM.
constexpr int bwd_pair_threads(int elem) { return elem == 2 ? 256 : 320; }

// How a call's rows are spread: a function of (n_rows, hidden, element type,
// direction, memory) alone.
struct DropNormPlan {
    bool warp;     // several rows a warp, or a warp a row
    bool staged;   // rows staged through shared memory by bulk copies
    int lanes;     // warp: lanes per row
    int threads;   // threads per CTA
    int K;         // blocks of 8 per thread
    int stages;
    int grid;      // CTAs; backward: also the number of dweight partial sums
    size_t smem;
};

DropNormPlan drop_norm_plan(int64_t n_rows, int hidden, int elem, bool backward, bool device_memory);
cudaError_t launch_drop_norm_fwd(const DropNormArgs& a, const DropNormPlan& p, int elem, cudaStream_t stream);
cudaError_t launch_drop_norm_bwd(const DropNormArgs& a, const DropNormPlan& p, int elem, cudaStream_t stream);
// One pair per element type, each in its own translation unit.
cudaError_t launch_drop_norm_bf16(const DropNormArgs& a, const DropNormPlan& p, bool backward, cudaStream_t stream);
cudaError_t launch_drop_norm_f16(const DropNormArgs& a, const DropNormPlan& p, bool backward, cudaStream_t stream);
cudaError_t launch_drop_norm_f32(const DropNormArgs& a, const DropNormPlan& p, bool backward, cudaStream_t stream);

// Column sums of parts x cols partial sums in a fixed order: columns
// [0, first) to out0, the others to out1 (either may be NULL: not wanted).
cudaError_t launch_column_sums(const float* partials, int parts, int cols, float* out0, int first, float* out1,
                               cudaStream_t stream);

// ------------------------------------------------------------------- rotary
// Tensors of heads: element (b, s, head, 0) at data + b * batch + s * seq +
// head * head_stride, in bytes; step: from a lane's head to its next one.
struct HeadsView {
    char* data;
    int64_t batch, seq, head, step;
};

enum RopeTensor : int { kRopeIn = 0, kRopeGrad = 1, kRopeOut = 2 };

// One of q and k: x, the gradient's dy, and what is written.
struct RopeSide {
    HeadsView t[3];
    const void* weight;  // behind the norm
    int heads;
    float eps;
    int skip_rest;  // in place without a norm: the units that do not turn stay
};

struct RopeArgs {
    RopeSide q, k;
    const double* inv_freq;
    const int64_t* positions;  // [batch, seq], or NULL: position0 + s
    int64_t position0;
    int64_t tokens;  // batch * seq, below 2^31
    int64_t seq;
    int dim, rot;
    int rot_units, units, group;  // 16-element units that rotate, in all; lanes per head (4, 8, 16 or 32)
    float inv_dim;                // 1 / dim
    float scale;
    float sign;                   // +1, or -1 for the inverse rotation
    // A warp has 32 / group lane groups.  They take as many heads of one
    // token a step (by_token 0), or one head each of as many tokens (1).  An
    // item is that token or those tokens, q_steps + k_steps steps; a warp
    // takes steps_per_warp of all n_steps, in order.
    int by_token;
    int heads_per_step, q_steps, k_steps, steps_per_warp;
    int64_t n_steps;
    float* partials;  // gradient: grid x 2 dim sums
};

enum RopeMode : int { kRopePlain = 0, kRopeNorm = 1, kRopeNormBwd = 2 };
constexpr int kRopeThreads = 256;
constexpr int kRopeMaxDim = 512;

// Steps and CTAs; backward: the grid is also the number of partial
// sums.  A function of the shape and the element type alone.
void rope_plan(RopeArgs* a, int elem, bool backward, int* grid);

cudaError_t launch_rope(const RopeArgs& a, int mode, int elem, bool interleaved, bool blocks, int grid,
                        cudaStream_t stream);
cudaError_t launch_rope_bf16(const RopeArgs& a, int mode, bool interleaved, bool blocks, int grid, cudaStream_t stream);
cudaError_t launch_rope_f16(const RopeArgs& a, int mode, bool interleaved, bool blocks, int grid, cudaStream_t stream);
cudaError_t launch_rope_f32(const RopeArgs& a, int mode, bool interleaved, bool blocks, int grid, cudaStream_t stream);

}  // namespace dradd
