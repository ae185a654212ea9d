// dradd_linear_grad.cu -- products whose results are gradients (two of them
// in one launch), and the partial sums of split products.
#include "dradd_linear.cuh"

namespace dradd {

// Columns come in eights.
__device__ __forceinline__ void add_partials(const float* p, float (&v)[16], int n)
{
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (4 * i < n) {
            const float4 f = *reinterpret_cast<const float4*>(p + 4 * i);
            v[4 * i] += f.x;
            v[4 * i + 1] += f.y;
            v[4 * i + 2] += f.z;
            v[4 * i + 3] += f.w;
        }
}

// A sector in one store where the workspace, which need lie on 16 bytes alone,
// allows it: partials come in rows of whole eights, so their start decides for
// all of them.
__device__ __forceinline__ void store_partials(float* p, const uint32_t (&w)[16], int n)
{
    const bool sectors = reinterpret_cast<uintptr_t>(p) % 32 == 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        if (8 * i >= n)
            continue;
        const uint32_t half[8] = {w[8 * i],     w[8 * i + 1], w[8 * i + 2], w[8 * i + 3],
                                  w[8 * i + 4], w[8 * i + 5], w[8 * i + 6], w[8 * i + 7]};
        if (sectors) {
            store_sector(p + 8 * i, half);
        } else {
            uint4* to = reinterpret_cast<uint4*>(p + 8 * i);
            to[0] = make_uint4(half[0], half[1], half[2], half[3]);
            to[1] = make_uint4(half[4], half[5], half[6], half[7]);
        }
    }
}

// A gradient's tile: rounded, or added to the fp32 sums of earlier pieces of
// the vocabulary, or a split's partial sum.  dx = dz W and dweight = dz^T x
// run in one launch, the longer tiles first, so that the shorter ones fill
// what the last round of the longer leaves idle (4096 tokens, a piece of 32768
// words: 3522 steps of the busiest pair for 3449 on average).  The operands
// whose rows lie along the summed dimension are read as they are: the
// products take either order from shared memory.
//
// Bound by the products, under the power limit 1630 to 1690 TFLOP/s (90 % of
// the cycles with the tensor pipe active at 16384 words); by the stores of
// dweight where there are few rows.
struct EpiGrad {
    using Kind = GradProducts;
    using Params = GradParams;
    static constexpr int kWarps = 8;
    static constexpr bool kStaged = true;
    static constexpr int kRun = 0;
    const Params& p;
    const bool bf16;
    const int row, col;
    Staging& staging;
    float* sums;
    float factor;

    __device__ __forceinline__ EpiGrad(const Params& p_, int bf16_, int row_, int col_, int split, Staging& staging_)
        : p(p_), bf16(bf16_), row(row_), col(col_), staging(staging_)
    {
        sums = p.partials + (static_cast<int64_t>(split) * p.rows + row) * p.cols + col;
        factor = p.factor ? *p.factor : 1.0f;
    }
    __device__ __forceinline__ void columns(const uint32_t (&bits)[16], int c)
    {
        const int n = p.cols - col - c;
        float v[16];
#pragma unroll
        for (int j = 0; j < 16; ++j)
            v[j] = __uint_as_float(bits[j]);
        if (p.add && row < p.rows)
            add_partials(sums + c, v, n);
        if (!p.to_out) {
            if (n > 0 && row < p.rows) {
                uint32_t w[16];
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    w[j] = __float_as_uint(v[j]);
                store_partials(sums + c, w, n);
            }
            return;
        }
#pragma unroll
        for (int j = 0; j < 16; ++j)
            v[j] *= factor;
        uint32_t w[8];
        pack16(v, bf16, w);
        staging.acquire(c);
        staging.write(c, w);
        staging.store_full(&p.out_map, c, col, row & ~31, (row & ~31) < p.rows && col + c - 48 < p.cols);
    }
    __device__ __forceinline__ void end() {}
};

template <class K, int RUN>
struct EpiSplit {
    using Kind = K;
    using Params = SplitParams;
    static constexpr int kWarps = 8;
    static constexpr bool kStaged = false;
    static constexpr int kRun = RUN;
    const Params& p;
    const int row, col;
    float* sums;

    __device__ __forceinline__ EpiSplit(const Params& p_, int, int row_, int col_, int split, Staging&)
        : p(p_), row(row_), col(col_)
    {
        sums = p.partials + (static_cast<int64_t>(split) * p.rows + row) * p.cols + col;
    }
    __device__ __forceinline__ void columns(const uint32_t (&bits)[16], int c)
    {
        const int n = p.cols - col - c;
        if (n > 0 && row < p.rows)
            store_partials(sums + c, bits, n);
    }
    template <int N>
    __device__ __forceinline__ void whole(const uint32_t (&bits)[N][16])
    {
#pragma unroll
        for (int i = 0; i < N; ++i)
            columns(bits[i], i * 16);
    }
    __device__ __forceinline__ void end() {}
};

template <>
cudaError_t launch_product<GradProducts>(const ProductArgs<GradProducts>& a, int cta_group, int sm_count,
                                         cudaStream_t stream)
{
    return launch_with<EpiGrad>(a, cta_group, sm_count, stream);
}

template <>
cudaError_t launch_product<SplitProduct>(const ProductArgs<SplitProduct>& a, int cta_group, int sm_count,
                                         cudaStream_t stream)
{
    return launch_with<EpiSplit<SplitProduct, 0>>(a, cta_group, sm_count, stream);
}

template <>
cudaError_t launch_product<LogitSplitProduct>(const ProductArgs<LogitSplitProduct>& a, int cta_group, int sm_count,
                                              cudaStream_t stream)
{
    return launch_with<EpiSplit<LogitSplitProduct, kLogitRun>>(a, cta_group, sm_count, stream);
}

}  // namespace dradd
