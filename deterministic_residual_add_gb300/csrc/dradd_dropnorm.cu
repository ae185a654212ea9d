// dradd_dropnorm.cu -- how the rows of dropout + residual add + RMSNorm and
// of its gradients are spread (dradd_dropnorm.cuh), and the sums of dweight's
// parts.
#include "dradd_elem.cuh"
#include "dradd_internal.h"
#include "dradd_train_internal.h"

namespace dradd {

namespace {

constexpr int kSms = 152;  // a constant, not the device's count: the parts of dweight follow the grid
constexpr int kSmemPerSm = 227 * 1024;
// Rows the busiest CTA takes with `ctas` per SM.
int64_t rounds(int64_t n_rows, int ctas)
{
    const int64_t grid = static_cast<int64_t>(kSms) * ctas;
    return (n_rows + grid - 1) / grid;
}

}  // namespace

DropNormPlan drop_norm_plan(int64_t n_rows, int hidden, int elem, bool backward, bool device_memory)
{
    DropNormPlan p = {};
    int P = 64;
    while (P < hidden)
        P *= 2;
    int per_sm;
    int64_t units;
    // Narrow kernels: backward wins up to 1024 for 2-byte types (16384 x 1024
    // 29.3 us, one CTA a row 32.3 to 43.3), not for fp32 (4096 x 1024 25.3, 19.5).
    if (P <= (backward && elem != kElemF32 ? 1024 : 256)) {
        p.warp = true;
        p.lanes = P / 8 < 32 ? P / 8 : 32;
        p.K = P / 8 / p.lanes;
        p.threads = 256;
        const int rows = p.threads / p.lanes;
        units = (n_rows + rows - 1) / rows;
        per_sm = narrow_ctas(elem, backward ? 3 : 2, p.K);
        p.smem = narrow_ring_bytes(elem, backward ? 3 : 2, p.K);
        const size_t sums = static_cast<size_t>(P) * 4 * (p.threads / 32);
        if (backward && p.smem < sums)
            p.smem = sums;
    } else {
        if (backward) {
            p.K = P <= 2048 ? 1 : P <= 8192 ? 2 : P / 4096;
            p.threads = (hidden / 8 + 32 * p.K - 1) / (32 * p.K) * 32;
        } else {
            // Many small CTAs: with one warp a row of 512 or 1024 and four
            // warps one of 2048 and 4096, the rows' barriers and sums hide
            // behind each other (8192 x 2048 bf16: 256 threads of one block
            // 23.8 us, 128 of two 16.3; 16384 x 1024: 128 of one 24.4, 64 of
            // two 17.5, 32 of four 16.4).  fp32 blocks are twice the bytes:
            // below 2048 one a thread (4096 x 1024: 10.6 us, two 12.0, four 13.3).
            p.K = P <= 1024 && elem == kElemF32 ? 1 : P == 512 || P == 2048 ? 2 : P <= 8192 ? 4 : P / 4096;
            p.threads = P / 8 / p.K;
        }
        units = n_rows;
        // CTAs per SM: as many as the registers allow (dradd_dropnorm.cuh) and
        // as leave each of them enough slots: two, or three where a slot is
        // refilled a row later.
        const int64_t slot = static_cast<int64_t>(hidden) * (elem == kElemF32 ? 4 : 2) * (backward ? 3 : 2);
        const int least = backward && p.K > 2 ? 3 : 2;
        const int resident =
            backward ? (p.K == 1 ? 1024 : p.K == 2 ? 2 * bwd_pair_threads(elem) : 512)
                     : p.K <= 2 && p.threads > 32 ? 1024 : 512;
        const auto slots_of = [&](int ctas) {
            return static_cast<int>((kSmemPerSm / ctas - 4096) / slot);  // less the system's share and the kernel's own
        };
        per_sm = resident / p.threads;
        if (backward && per_sm > 4)
            per_sm = 4;  // more would only make more partial sums
        while (per_sm > 1 && slots_of(per_sm) < least)
            --per_sm;
        // Several forward CTAs an SM do best with two slots each (16384 x 4096
        // bf16 88.7 us, with three 90.0; 16384 x 512 9.6, with four 13.8).
        int stages = slots_of(per_sm);
        const int most_stages = backward || per_sm == 1 ? 4 : 2;
        if (stages > most_stages)
            stages = most_stages;
        // One CTA with more slots keeps an SM busy too where a row is long
        // enough, and deals rows out evenly where two would leave the last
        // round half empty: 4096 x 8192 bf16 40.8 us against 43.9.
        if (!backward && per_sm == 2 && slot >= 32 * 1024 && rounds(n_rows, 1) < 2 * rounds(n_rows, 2)) {
            per_sm = 1;
            stages = slots_of(1) < 4 ? slots_of(1) : 4;
        }
        if (device_memory && stages >= 2) {
            p.staged = true;
            p.stages = stages;
            p.smem = static_cast<size_t>(stages * slot) + 8 * stages;
        }
    }
    const int64_t most = static_cast<int64_t>(kSms) * per_sm;
    p.grid = static_cast<int>(units < most ? units : most);
    return p;
}

cudaError_t launch_drop_norm_fwd(const DropNormArgs& a, const DropNormPlan& p, int elem, cudaStream_t stream)
{
    return elem == kElemBf16  ? launch_drop_norm_bf16(a, p, false, stream)
           : elem == kElemF16 ? launch_drop_norm_f16(a, p, false, stream)
                              : launch_drop_norm_f32(a, p, false, stream);
}

cudaError_t launch_drop_norm_bwd(const DropNormArgs& a, const DropNormPlan& p, int elem, cudaStream_t stream)
{
    return elem == kElemBf16  ? launch_drop_norm_bf16(a, p, true, stream)
           : elem == kElemF16 ? launch_drop_norm_f16(a, p, true, stream)
                              : launch_drop_norm_f32(a, p, true, stream);
}

constexpr int kColumnLoads = 10;

// Warp w of a CTA adds parts w, w + 32, ... of its 32 columns in order; the
// 32 warps' sums are then added in warp order.
__global__ void __launch_bounds__(1024) column_sums_kernel(const float* partials, int parts, int cols, float* out0,
                                                           int first, float* out1)
{
    __shared__ float sums[32][33];
    wait_prior_grids();
    allow_next_grid();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int col = blockIdx.x * 32 + lane;
    float s = 0.0f;
    if (col < cols) {
        const float* p = partials + col;
        for (int i = warp; i < parts; i += 32 * kColumnLoads) {
            float v[kColumnLoads];  // on their way together
#pragma unroll
            for (int k = 0; k < kColumnLoads; ++k)
                v[k] = i + 32 * k < parts ? __ldcs(p + static_cast<int64_t>(i + 32 * k) * cols) : 0.0f;
#pragma unroll
            for (int k = 0; k < kColumnLoads; ++k)
                s = __fadd_rn(s, v[k]);
        }
    }
    sums[warp][lane] = s;
    __syncthreads();
    // warp w now holds column w of the CTA, one warp's sum a lane
    s = butterfly_sum(sums[lane][warp], 32);
    const int c = blockIdx.x * 32 + warp;
    if (lane == 0 && c < cols) {
        if (c < first && out0)
            out0[c] = s;
        if (c >= first && out1)
            out1[c - first] = s;
    }
}

cudaError_t launch_column_sums(const float* partials, int parts, int cols, float* out0, int first, float* out1,
                               cudaStream_t stream)
{
    return launch(column_sums_kernel, (cols + 31) / 32, 1024, 0, false, stream, partials, parts, cols, out0, first,
                  out1);
}

}  // namespace dradd
