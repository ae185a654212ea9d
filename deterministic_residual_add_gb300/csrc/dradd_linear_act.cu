// dradd_linear_act.cu -- products with bias, activation and residual behind
// them, and with the activation's derivative.
#include "dradd_act.cuh"
#include "dradd_linear.cuh"

namespace dradd {

// out = residual + act(z + bias).  The residual of a warp's part of the tile
// comes into the space that the results leave from, while the products run.
//
// Bound by the products where the inner dimension is long; below some 2000
// by these steps, up to 60 instructions an element, for which the kernel has
// 16 warps: four a scheduler.
struct EpiAct {
    using Kind = ActProduct;
    using Params = ActProductParams;
    static constexpr int kWarps = 16;
    static constexpr bool kStaged = true;
    static constexpr int kCols = kTileCols * 4 / kWarps;
    const Params& q;
    const ActParams& p;
    const bool bf16;
    const int row, col;
    Staging& staging;
    const bool inside;  // some of the warp's rows and columns are

    __device__ __forceinline__ EpiAct(const Params& q_, int bf16_, int row_, int col_, int, Staging& staging_)
        : q(q_), p(q_.act), bf16(bf16_), row(row_), col(col_), staging(staging_),
          inside((row_ & ~31) < q_.act.rows && col_ < q_.act.cols)
    {
        if (p.bias && col < p.cols)
            prefetch_l1(static_cast<const uint16_t*>(p.bias) + col);
        if (!p.other)
            return;
        staging.acquire();
        if (inside)
            staging.load(&q.other_map, col, row & ~31, kCols / 64);
    }
    __device__ __forceinline__ bool ready(uint64_t limit_ns)
    {
        return !(p.other && inside) || staging.loaded(limit_ns);
    }
    __device__ __forceinline__ void add_bias(const uint32_t (&bits)[16], int c, int n, float (&z)[16])
    {
#pragma unroll
        for (int j = 0; j < 16; ++j)
            z[j] = __uint_as_float(bits[j]);
        if (p.bias) {
            uint32_t w[8];
            float b[16];
            load16(static_cast<const uint16_t*>(p.bias) + col + c, n, w);
            unpack16(w, bf16, b);
#pragma unroll
            for (int j = 0; j < 16; ++j)
                z[j] += b[j];
        }
    }
    __device__ __forceinline__ void store(const float (&z)[16], int c)
    {
        uint32_t w[8];
        pack16(z, bf16, w);
        if (!p.other)
            staging.acquire_box<kCols / 64>(c);
        staging.write(c, w);
        staging.store_full(&q.out_map, c, col, row & ~31, col + c - 48 < p.cols);
    }
    __device__ __forceinline__ void columns(const uint32_t (&bits)[16], int c)
    {
        if (!inside)
            return;
        float z[16];
        add_bias(bits, c, p.cols - col - c, z);
        act_values(z, p.act);
        if (p.other) {
            uint32_t w[8];
            float other[16];
            staging.read(c, w);
            unpack16(w, bf16, other);
#pragma unroll
            for (int j = 0; j < 16; ++j)
                z[j] += other[j];
        }
        store(z, c);
    }
    __device__ __forceinline__ void end() {}
};

// dz = dout * act'(z + bias), and its sums over 32 rows for the bias.
struct EpiActGrad : EpiAct {
    using Kind = ActGradProduct;
    using EpiAct::EpiAct;
    // The warp's 32 rows of each of 16 columns: at every level a lane keeps
    // one half of its columns and hands the other one over, until it has one;
    // two lanes then have half of the rows each.
    __device__ __forceinline__ void add_up(const float (&z)[16], int c, int n)
    {
        float v[16];
#pragma unroll
        for (int j = 0; j < 16; ++j)
            v[j] = row < p.rows ? z[j] : 0.0f;
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int d = 8; d > 0; d >>= 1)
#pragma unroll
            for (int j = 0; j < d; ++j) {
                const bool upper = lane & d;
                const float give = upper ? v[j] : v[j + d];
                v[j] = (upper ? v[j + d] : v[j]) + __shfl_xor_sync(0xffffffffu, give, d);
            }
        const float sum = v[0] + __shfl_xor_sync(0xffffffffu, v[0], 16);
        if (lane < 16 && lane < n)
            p.col_sums[static_cast<int64_t>(row >> 5) * p.cols + col + c + lane] = sum;
    }
    __device__ __forceinline__ void columns(const uint32_t (&bits)[16], int c)
    {
        if (!inside)
            return;
        const int n = p.cols - col - c;
        float z[16], other[16];
        uint32_t w[8];
        add_bias(bits, c, n, z);
        act_slopes(z, p.act);
        staging.read(c, w);
        unpack16(w, bf16, other);
#pragma unroll
        for (int j = 0; j < 16; ++j)
            z[j] *= other[j];
        if (p.col_sums && n > 0)
            add_up(z, c, n);
        store(z, c);
    }
};

template <>
cudaError_t launch_product<ActProduct>(const ProductArgs<ActProduct>& a, int cta_group, int sm_count,
                                       cudaStream_t stream)
{
    return launch_with<EpiAct>(a, cta_group, sm_count, stream);
}

template <>
cudaError_t launch_product<ActGradProduct>(const ProductArgs<ActGradProduct>& a, int cta_group, int sm_count,
                                           cudaStream_t stream)
{
    return launch_with<EpiActGrad>(a, cta_group, sm_count, stream);
}

}  // namespace dradd
