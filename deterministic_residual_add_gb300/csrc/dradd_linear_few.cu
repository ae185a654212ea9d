// dradd_linear_few.cu -- the product of linear_act_add_fwd for up to 16 rows.
//
// The weights are read once and everything else is small, so what counts is
// how many of their bytes are on their way.  A CTA takes R columns of the
// output (rows of W) and brings them through a ring of four stages of 16 KB
// by bulk copies: 64 KB a CTA in flight whatever the warps do, three CTAs an
// SM (two from 9 rows on, whose sums take 8 KB more).  Its 8 warps take an eighth of each stage's inner dimension each.  The
// products are warp-wide m16n8k16: the sum does not mind the order of its
// terms, so a lane feeds the 8 neighbouring elements that it loaded as if
// they were the four pairs that two products ask of it.  The warps' sums are
// added in order.
#include "dradd_act.cuh"
#include "dradd_elem.cuh"
#include "dradd_internal.h"
#include "dradd_linear_internal.h"
#include "dradd_mma.cuh"
#include "dradd_train_internal.h"

namespace dradd {

namespace {

constexpr int kFewWarps = 8;
constexpr int kFewStages = 4;
constexpr int kFewStageElems = 8192;

// Rows of a stage lie 64 bytes further than they are long: two neighbouring
// rows' 64-byte pieces, which a quarter warp reads together, are in other banks.
__host__ __device__ constexpr int few_depth(int R) { return kFewStageElems / R; }
__host__ __device__ constexpr int few_row_bytes(int R) { return few_depth(R) * 2 + 64; }
__host__ __device__ constexpr int few_stage_bytes(int R) { return R * few_row_bytes(R); }

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

// T tiles of 8 rows of x, R (8 or 16) rows of W.
template <int T, int R>
__global__ void __launch_bounds__(kFewWarps * 32, 3) few_kernel(const FewParams p)
{
    constexpr int kDepth = few_depth(R), kSteps = kDepth / kFewWarps / 32;  // a warp's steps of 32 in a stage
    extern __shared__ __align__(128) unsigned char ring[];
    __shared__ float sums[kFewWarps][T * 8][R + 1];
    __shared__ uint64_t full[kFewStages], empty[kFewStages];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, t = lane & 3;
    const int col0 = blockIdx.x * R;
    const int cols = min(R, p.act.cols - col0);
    const int stages = (p.inner + kDepth - 1) / kDepth;
    const bool bf16 = p.bf16;
    const uint4 none = make_uint4(0, 0, 0, 0);
    const uint16_t* w = static_cast<const uint16_t*>(p.weight) + col0 * p.weight_stride;
    // The first stages are asked into L2 while the grid before ends.
    if (static_cast<int>(threadIdx.x) < cols)
        prefetch_l2(w + threadIdx.x * p.weight_stride, static_cast<uint32_t>(min(kDepth * kFewStages, p.inner)) * 2);
    if (threadIdx.x == 0) {
        for (int i = 0; i < kFewStages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], kFewWarps);
        }
        fence_mbar_init();
    }
    __syncthreads();
    allow_next_grid();
    wait_prior_grids();
    // Ordinary loads: x may be what the grid in front writes, and so is not
    // read-only as long as this one lives.
    const uint16_t* x = static_cast<const uint16_t*>(p.x);
    // Lane i < cols of warp 0 copies row i of stage s; lane 0 has said how
    // many bytes come before any of them starts.
    const auto copy = [&](int s) {
        const int at = s % kFewStages;
        const uint32_t bytes = static_cast<uint32_t>(min(kDepth, p.inner - s * kDepth)) * 2;
        if (lane == 0)
            mbar_arrive_expect_tx(&full[at], bytes * cols);
        __syncwarp();
        if (lane < cols)
            bulk_copy_g2s(ring + at * few_stage_bytes(R) + lane * few_row_bytes(R),
                          w + lane * p.weight_stride + static_cast<int64_t>(s) * kDepth, bytes, &full[at],
                          l2_policy_evict_first());
    };
    if (warp == 0)
        for (int s = 0; s < kFewStages && s < stages; ++s)
            copy(s);
    bool ok = true;
    float d[T][4] = {};
    int s = 0;
    for (; ok && s < stages; ++s) {
        const int at = s % kFewStages;
        const uint32_t parity = (s / kFewStages) & 1;
        const int k0 = s * kDepth + warp * (kDepth / kFewWarps) + t * 8;
        uint4 b[kSteps][T];
#pragma unroll
        for (int u = 0; u < kSteps; ++u)
#pragma unroll
            for (int i = 0; i < T; ++i) {
                const int row = i * 8 + g;
                b[u][i] = k0 + u * 32 < p.inner && row < p.act.rows  // whole blocks of 8
                              ? *reinterpret_cast<const uint4*>(x + row * p.x_stride + k0 + u * 32)
                              : none;
            }
        ok = __all_sync(0xffffffffu, mbar_wait_bounded(&full[at], parity, p.wait_limit_ns));
        if (!ok)
            break;
        const unsigned char* from = ring + at * few_stage_bytes(R) + (warp * (kDepth / kFewWarps) + t * 8) * 2;
        uint4 a[kSteps][2];
#pragma unroll
        for (int u = 0; u < kSteps; ++u) {
            const bool in = k0 + u * 32 < p.inner;
            a[u][0] = in && g < cols ? *reinterpret_cast<const uint4*>(from + g * few_row_bytes(R) + u * 64) : none;
            a[u][1] = R == 16 && in && g + 8 < cols
                          ? *reinterpret_cast<const uint4*>(from + (g + 8) * few_row_bytes(R) + u * 64)
                          : none;
        }
#pragma unroll
        for (int u = 0; u < kSteps; ++u)
#pragma unroll
            for (int i = 0; i < T; ++i) {
                mma16816(d[i], a[u][0].x, a[u][1].x, a[u][0].y, a[u][1].y, b[u][i].x, b[u][i].y, bf16);
                mma16816(d[i], a[u][0].z, a[u][1].z, a[u][0].w, a[u][1].w, b[u][i].z, b[u][i].w, bf16);
            }
        if (s + kFewStages < stages) {
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&empty[at]);
            if (warp == 0) {
                ok = __all_sync(0xffffffffu, mbar_wait_bounded(&empty[at], parity, p.wait_limit_ns));
                if (!ok)
                    break;
                copy(s + kFewStages);
            }
        }
    }
    if (!ok) {
        if (lane == 0)
            atomicOr(p.status, kDeviceStatusTimeout);
        if (warp == 0) {  // it started the copies: those of stages s to s + kFewStages - 1, as far as there are so many
            for (int i = s; i < s + kFewStages && i < stages; ++i)
                if (!mbar_wait_bounded(&full[i % kFewStages], (i / kFewStages) & 1, p.wait_limit_ns) && lane == 0)
                    atomicOr(p.status, kDeviceStatusUndrained);
        }
    }
#pragma unroll
    for (int i = 0; i < T; ++i) {
        sums[warp][i * 8 + 2 * t][g] = d[i][0];
        sums[warp][i * 8 + 2 * t + 1][g] = d[i][1];
        if constexpr (R == 16) {
            sums[warp][i * 8 + 2 * t][g + 8] = d[i][2];
            sums[warp][i * 8 + 2 * t + 1][g + 8] = d[i][3];
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < p.act.rows * R; i += kFewWarps * 32) {
        const int row = i / R, c = i % R, col = col0 + c;
        if (c >= cols)
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

template <int T, int R>
cudaError_t launch_few_of(const FewParams& p, cudaStream_t stream)
{
    const cudaError_t e = allow_all_shared<few_kernel<T, R>>();
    if (e != cudaSuccess)
        return e;
    return launch(few_kernel<T, R>, (p.act.cols + R - 1) / R, kFewWarps * 32, kFewStages * few_stage_bytes(R), false,
                  stream, p);
}

}  // namespace

cudaError_t launch_few(const FewParams& p, cudaStream_t stream)
{
    return p.act.rows <= 8 ? launch_few_of<1, 8>(p, stream) : launch_few_of<2, 16>(p, stream);
}

}  // namespace dradd
