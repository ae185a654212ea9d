// dradd_linear_act.cu -- products with bias, activation and residual behind
// them, and with the activation's derivative.
#include "dradd_act.cuh"
#include "dradd_linear.cuh"

namespace dradd {

// out = residual + act(z + bias).  The residual's values of the two next
// steps of 16 columns are on their way while the present ones are worked on.
//
// Bound by the products where the inner dimension is long; below some 2000
// by these steps, up to 60 instructions an element, for which the kernel has
// 16 warps: four a scheduler.
struct EpiAct {
    using Kind = ActProduct;
    using Params = ActParams;
    static constexpr int kWarps = 16;
    static constexpr int kCols = kTileCols * 4 / kWarps;
    const Params& p;
    const bool bf16;
    const int row, col;
    uint32_t other[2][8];

    __device__ __forceinline__ EpiAct(const Params& p_, int bf16_, int row_, int col_, int)
        : p(p_), bf16(bf16_), row(row_), col(col_)
    {
        fetch<0>(0);
        fetch<1>(16);
    }
    template <int B>
    __device__ __forceinline__ void fetch(int c)
    {
        if (p.other && row < p.rows)
            load16(static_cast<const uint16_t*>(p.other) + row * p.other_stride + col + c, p.cols - col - c, other[B]);
    }
    __device__ __forceinline__ void add_bias(const uint32_t (&bits)[16], int c, int n, float (&z)[16])
    {
#pragma unroll
        for (int j = 0; j < 16; ++j)
            z[j] = __uint_as_float(bits[j]);
        if (p.bias) {
            uint32_t b[8];
            load16(static_cast<const uint16_t*>(p.bias) + col + c, n, b);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                float lo, hi;
                unpack2(b[j], bf16, lo, hi);
                z[2 * j] += lo;
                z[2 * j + 1] += hi;
            }
        }
    }
    __device__ __forceinline__ void store(const float (&z)[16], int c, int n)
    {
        if (row < p.rows) {
            uint32_t w[8];
            pack16(z, bf16, w);
            store16(static_cast<uint16_t*>(p.out) + row * p.out_stride + col + c, w, n);
        }
    }
    template <int B>
    __device__ __forceinline__ void columns(const uint32_t (&bits)[16], int c)
    {
        const int n = p.cols - col - c;
        if (n <= 0)
            return;
        float z[16];
        add_bias(bits, c, n, z);
        act_values(z, p.act);
        if (p.other) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                float lo, hi;
                unpack2(other[B][j], bf16, lo, hi);
                z[2 * j] += lo;
                z[2 * j + 1] += hi;
            }
            if (c + 32 < kCols)
                fetch<B>(c + 32);
        }
        store(z, c, n);
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
    template <int B>
    __device__ __forceinline__ void columns(const uint32_t (&bits)[16], int c)
    {
        const int n = p.cols - col - c;
        if (n <= 0)
            return;
        float z[16];
        add_bias(bits, c, n, z);
        act_slopes(z, p.act);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float lo, hi;
            unpack2(other[B][j], bf16, lo, hi);
            z[2 * j] *= lo;
            z[2 * j + 1] *= hi;
        }
        if (c + 32 < kCols)
            fetch<B>(c + 32);
        if (p.col_sums)
            add_up(z, c, n);
        store(z, c, n);
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
