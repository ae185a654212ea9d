// dradd_linear_few.cu -- the product of linear_act_add_fwd for up to 16 rows.
//
// The weights are read once and everything else is small, so what counts is
// how many of their bytes are on their way.  A CTA takes 16 columns of the
// output (rows of W), its 8 warps a stripe of the inner dimension each, and
// every lane holds eight 16-byte loads of W in flight.  The products are
// warp-wide m16n8k16: the sum does not mind the order of its terms, so a lane
// feeds the 8 neighbouring elements that it loaded as if they were the four
// pairs that two products ask of it.  The warps' sums are added in order.
#include "dradd_act.cuh"
#include "dradd_elem.cuh"
#include "dradd_internal.h"
#include "dradd_linear_internal.h"

namespace dradd {

namespace {

constexpr int kFewWarps = 8;
constexpr int kFewCols = 16;
constexpr int kFewUnroll = 4;  // steps of 32 of the inner dimension in flight
// Bytes of each row of W asked into L2 while the grid before may still run:
// with the up to 600 CTAs that the device holds, 80 MB at most.
constexpr int kFewPrefetch = 8192;

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1, bool bf16)
{
    if (bf16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, "
                     "%9}, {%0, %1, %2, %3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, "
                     "%9}, {%0, %1, %2, %3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// T tiles of 8 rows of x.
template <int T>
__global__ void __launch_bounds__(kFewWarps * 32) few_kernel(const FewParams p)
{
    __shared__ float sums[kFewWarps][T * 8][kFewCols + 1];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, t = lane & 3;
    const int col0 = blockIdx.x * kFewCols;
    if (threadIdx.x < kFewCols && col0 + static_cast<int>(threadIdx.x) < p.act.cols)
        prefetch_l2(static_cast<const uint16_t*>(p.weight) + (col0 + threadIdx.x) * p.weight_stride,
                    min(p.inner * 2, kFewPrefetch));
    allow_next_grid();
    wait_prior_grids();
    const bool bf16 = p.bf16;
    const uint4 none = make_uint4(0, 0, 0, 0);
    const uint16_t* w = static_cast<const uint16_t*>(p.weight);
    const uint16_t* x = static_cast<const uint16_t*>(p.x);
    // rows g and g + 8 of W's sixteen, and of each tile of x
    const bool in0 = col0 + g < p.act.cols, in1 = col0 + g + 8 < p.act.cols;
    const uint16_t* w0 = w + (in0 ? col0 + g : 0) * p.weight_stride;
    const uint16_t* w1 = w + (in1 ? col0 + g + 8 : 0) * p.weight_stride;
    float d[T][4] = {};
    const int steps = (p.inner + 31) / 32;  // of 32
    for (int s0 = warp; s0 < steps; s0 += kFewWarps * kFewUnroll) {
        uint4 a[kFewUnroll][2], b[kFewUnroll][T];
#pragma unroll
        for (int u = 0; u < kFewUnroll; ++u) {
            const int k = (s0 + u * kFewWarps) * 32 + t * 8;
            const bool in = k < p.inner;  // whole blocks of 8
            a[u][0] = in && in0 ? __ldcs(reinterpret_cast<const uint4*>(w0 + k)) : none;
            a[u][1] = in && in1 ? __ldcs(reinterpret_cast<const uint4*>(w1 + k)) : none;
        }
#pragma unroll
        for (int u = 0; u < kFewUnroll; ++u) {
            const int k = (s0 + u * kFewWarps) * 32 + t * 8;
#pragma unroll
            for (int i = 0; i < T; ++i) {
                const int row = i * 8 + g;
                b[u][i] = k < p.inner && row < p.act.rows
                              ? __ldg(reinterpret_cast<const uint4*>(x + row * p.x_stride + k))
                              : none;
            }
        }
#pragma unroll
        for (int u = 0; u < kFewUnroll; ++u)
#pragma unroll
            for (int i = 0; i < T; ++i) {
                mma16816(d[i], a[u][0].x, a[u][1].x, a[u][0].y, a[u][1].y, b[u][i].x, b[u][i].y, bf16);
                mma16816(d[i], a[u][0].z, a[u][1].z, a[u][0].w, a[u][1].w, b[u][i].z, b[u][i].w, bf16);
            }
    }
#pragma unroll
    for (int i = 0; i < T; ++i) {
        sums[warp][i * 8 + 2 * t][g] = d[i][0];
        sums[warp][i * 8 + 2 * t + 1][g] = d[i][1];
        sums[warp][i * 8 + 2 * t][g + 8] = d[i][2];
        sums[warp][i * 8 + 2 * t + 1][g + 8] = d[i][3];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < p.act.rows * kFewCols; i += kFewWarps * 32) {
        const int row = i / kFewCols, c = i % kFewCols, col = col0 + c;
        if (col >= p.act.cols)
            continue;
        float z[1] = {0.0f};
#pragma unroll
        for (int v = 0; v < kFewWarps; ++v)
            z[0] += sums[v][row][c];
        const auto widen = [&](uint16_t v) {
            return bf16 ? Elem<kElemBf16>::widen(v) : Elem<kElemF16>::widen(v);
        };
        if (p.act.bias)
            z[0] += widen(static_cast<const uint16_t*>(p.act.bias)[col]);
        act_values(z, p.act.act);
        if (p.act.other)
            z[0] += widen(static_cast<const uint16_t*>(p.act.other)[row * p.act.other_stride + col]);
        static_cast<uint16_t*>(p.act.out)[row * p.act.out_stride + col] =
            bf16 ? Elem<kElemBf16>::narrow(z[0]) : Elem<kElemF16>::narrow(z[0]);
    }
}

}  // namespace

cudaError_t launch_few(const FewParams& p, cudaStream_t stream)
{
    const int grid = (p.act.cols + kFewCols - 1) / kFewCols;
    return p.act.rows <= 8 ? launch(few_kernel<1>, grid, kFewWarps * 32, 0, false, stream, p)
                           : launch(few_kernel<2>, grid, kFewWarps * 32, 0, false, stream, p);
}

}  // namespace dradd
