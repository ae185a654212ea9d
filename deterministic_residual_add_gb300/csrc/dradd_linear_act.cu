// dradd_linear_act.cu -- products with bias, activation and residual behind
// them, and with the activation's derivative.
#include "dradd_act.cuh"
#include "dradd_linear.cuh"

namespace dradd {

// out = residual + act(z + bias).  The residual comes into the box that the
// results leave from, its first one while the products run.
//
// Bound by the products where the inner dimension is long (8192 x 16384 by
// 4096 656 to 680 us, 1620 to 1680 TFLOP/s under the power limit); below some
// 1000 by these steps (8192 x 512 by 8192 51 us plain, 59 with a bias, 66
// with silu, 86 with gelu; what has to move takes 23).
template <bool DEEP>
struct EpiAct {
    using Kind = ActProduct;
    using Params = ActProductParams;
    static constexpr int kWarps = DEEP ? 8 : 16;
    static constexpr bool kStaged = true;
    static constexpr int kRun = 0;
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
        if (p.other && inside)
            staging.load(&q.other_map, col, row & ~31);
    }
    // At the first of a box's columns: the box may be used, and what comes in is there.
    __device__ __forceinline__ void enter_box(int c)
    {
        if ((c & 63) != 0)
            return;
        if (!p.other) {
            staging.acquire(c);
            return;
        }
        if (c > 0)
            staging.load(&q.other_map, col + c, row & ~31);
        staging.loaded();
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
        staging.write(c, w);
        staging.store_full(&q.out_map, c, col, row & ~31, col + c - 48 < p.cols);
    }
    __device__ __forceinline__ void columns(const uint32_t (&bits)[16], int c)
    {
        if (!inside)
            return;
        float z[16];
        add_bias(bits, c, p.cols - col - c, z);
        enter_box(c);
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

// dz = dout * act'(z + bias), and its sums over 32 rows for the bias, from
// the values before they are rounded.  (A pass of its own over dz for the
// bias took 45 us for 8192 x 16384.)
template <bool DEEP>
struct EpiActGrad : EpiAct<DEEP> {
    using Kind = ActGradProduct;
    using Base = EpiAct<DEEP>;
    using Base::Base;
    using Base::p, Base::q, Base::row, Base::col, Base::inside, Base::bf16, Base::staging;
    // The warp's 32 rows of each of 16 columns: at every level a lane keeps
    // one half of its columns and hands the other one over, until it has one;
    // two lanes then have half of the rows each.
    __device__ __forceinline__ void add_up(const float (&z)[16], int c, int n)
    {
        float v[16];
#pragma unroll
        for (int j = 0; j < 16; ++j)
            v[j] = z[j];  // rows outside have a dout of zeros, and so no dz but where the column's is NaN anyway
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
        Base::add_bias(bits, c, n, z);
        Base::enter_box(c);
        act_slopes(z, p.act);
        staging.read(c, w);
        unpack16(w, bf16, other);
#pragma unroll
        for (int j = 0; j < 16; ++j)
            z[j] *= other[j];
        if (p.col_sums && n > 0)
            add_up(z, c, n);
        Base::store(z, c);
    }
};

template <>
cudaError_t launch_product<ActProduct>(const ProductArgs<ActProduct>& a, int cta_group, int sm_count,
                                       cudaStream_t stream)
{
    return long_sums(a) ? launch_with<EpiAct<true>>(a, cta_group, sm_count, stream)
                        : launch_with<EpiAct<false>>(a, cta_group, sm_count, stream);
}

template <>
cudaError_t launch_product<ActGradProduct>(const ProductArgs<ActGradProduct>& a, int cta_group, int sm_count,
                                           cudaStream_t stream)
{
    return long_sums(a) ? launch_with<EpiActGrad<true>>(a, cta_group, sm_count, stream)
                        : launch_with<EpiActGrad<false>>(a, cta_group, sm_count, stream);
}

}  // namespace dradd
