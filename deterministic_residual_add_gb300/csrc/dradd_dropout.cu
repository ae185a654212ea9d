// dradd_dropout.cu -- dropout, and dropout + residual add, of row-strided
// tensors: out = kept ? RN(x scale) : 0, plus residual where there is one
// (one fp32 addition), rounded once to the element type.
//
// Bound by the memory: 2 (3) elements of traffic an element, and one
// generator call for 8 of them (dradd_philox.cuh).
#include "dradd_elem.cuh"
#include "dradd_internal.h"
#include "dradd_philox.cuh"
#include "dradd_train_internal.h"

namespace dradd {

// Rows of whole, 16-byte aligned blocks of 8: a thread takes a block at a
// time, blocks in row-major order with a stride of the whole grid, walked as
// (row, block) with a carry so that nothing is divided inside the loop.
template <int E, bool ADD>
__global__ void __launch_bounds__(kDropoutThreads) dropout_blocks_kernel(const DropoutArgs a, uint32_t blocks,
                                                                         uint32_t step_rows, uint32_t step_blocks)
{
    using V = typename Elem<E>::Block;
    using T = typename Elem<E>::T;
    wait_prior_grids();
    allow_next_grid();
    const uint2 offset = drop_offset(a.drop);
    const uint32_t n_rows = static_cast<uint32_t>(a.n_rows);
    const uint32_t first = blockIdx.x * kDropoutThreads + threadIdx.x;
    uint32_t row = first / blocks;
    uint32_t b = first - row * blocks;
    while (row < n_rows) {
        V xv, rv;
        ld_block_stream(static_cast<const T*>(a.x) + row * a.x_stride, b, xv);
        if constexpr (ADD)
            ld_block_stream(static_cast<const T*>(a.residual) + row * a.residual_stride, b, rv);
        float v[8];
        Elem<E>::unpack(xv, v);
        if (a.drop.drops)
            drop8(v, a.drop, offset, b, row);
        if constexpr (ADD) {
            float r[8];
            Elem<E>::unpack(rv, r);
#pragma unroll
            for (int e = 0; e < 8; e += 2)
                add2_rn(r[e], r[e + 1], v[e], v[e + 1], v[e], v[e + 1]);
        }
        st_block_stream(static_cast<T*>(a.out) + row * a.out_stride, b, Elem<E>::pack(v));
        row += step_rows;
        b += step_blocks;
        if (b >= blocks) {
            b -= blocks;
            ++row;
        }
    }
}

// Any width and alignment: a warp takes 256 columns of a row.  Lane l draws
// the bits of columns 8 l .. 8 l + 7; one ballot for each of the 8 numbers
// of a block turns them into masks, in which column 32 v + l finds its bit
// at 4 v + l / 8 of ballot l % 8, so every load and store of a warp covers
// 32 neighbouring columns and each generator call is made once.
template <int E, bool ADD>
__global__ void __launch_bounds__(kDropoutThreads) dropout_ragged_kernel(const DropoutArgs a, uint32_t strips,
                                                                         uint32_t step_rows, uint32_t step_strips)
{
    using T = typename Elem<E>::T;
    wait_prior_grids();
    allow_next_grid();
    const uint2 offset = drop_offset(a.drop);
    const int lane = threadIdx.x & 31;
    const uint32_t first = blockIdx.x * (kDropoutThreads / 32) + (threadIdx.x >> 5);
    uint32_t row = first / strips;
    uint32_t strip = first - row * strips;
    while (row < a.n_rows) {
        const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
        const T* r = ADD ? static_cast<const T*>(a.residual) + row * a.residual_stride : nullptr;
        T* out = static_cast<T*>(a.out) + row * a.out_stride;
        const int64_t col = static_cast<int64_t>(strip) * 256 + lane;
        T xv[8], rv[8];
#pragma unroll
        for (int v = 0; v < 8; ++v) {
            if (col + 32 * v < a.hidden) {
                xv[v] = __ldcs(x + col + 32 * v);
                if constexpr (ADD)
                    rv[v] = __ldcs(r + col + 32 * v);
            }
        }
        uint32_t mine = 0xFFFFFFFFu;
        if (a.drop.drops) {
            const uint4 bits = drop_bits(a.drop, offset, strip * 32 + lane, row);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const uint32_t m = __ballot_sync(0xFFFFFFFFu, kept(bits, e, a.drop.limit));
                if ((lane & 7) == e)
                    mine = m >> (lane >> 3);
            }
        }
#pragma unroll
        for (int v = 0; v < 8; ++v) {
            if (col + 32 * v < a.hidden) {
                float f = (mine >> (4 * v)) & 1u ? __fmul_rn(Elem<E>::widen(xv[v]), a.drop.scale) : 0.0f;
                if constexpr (ADD)
                    f = __fadd_rn(Elem<E>::widen(rv[v]), f);
                __stcs(out + col + 32 * v, Elem<E>::narrow(f));
            }
        }
        row += step_rows;
        strip += step_strips;
        if (strip >= strips) {
            strip -= strips;
            ++row;
        }
    }
}

namespace {

template <int E, bool ADD>
cudaError_t launch_dropout_of(const DropoutArgs& a, bool blocks, int sm_count, cudaStream_t stream)
{
    const int64_t per_row = blocks ? a.hidden >> 3 : (a.hidden + 255) / 256;
    const int64_t per_cta = blocks ? kDropoutThreads : kDropoutThreads / 32;
    const int64_t wanted = (a.n_rows * per_row + per_cta - 1) / per_cta;
    const int64_t most = static_cast<int64_t>(sm_count) * kDropoutCtasPerSm;
    const int grid = static_cast<int>(wanted < most ? wanted : most);
    // rows and blocks are 32-bit in the kernels: both, and one step more, fit
    const int64_t step = grid * per_cta;
    const uint32_t span = static_cast<uint32_t>(per_row);
    const uint32_t step_rows = static_cast<uint32_t>(step / per_row), rest = static_cast<uint32_t>(step % per_row);
    if (blocks)
        return launch(dropout_blocks_kernel<E, ADD>, grid, kDropoutThreads, 0, false, stream, a, span, step_rows, rest);
    return launch(dropout_ragged_kernel<E, ADD>, grid, kDropoutThreads, 0, false, stream, a, span, step_rows, rest);
}

}  // namespace

cudaError_t launch_dropout(const DropoutArgs& a, int elem, bool blocks, int sm_count, cudaStream_t stream)
{
    const bool add = a.residual != nullptr;
    switch (elem) {
    case kElemBf16:
        return add ? launch_dropout_of<kElemBf16, true>(a, blocks, sm_count, stream)
                   : launch_dropout_of<kElemBf16, false>(a, blocks, sm_count, stream);
    case kElemF16:
        return add ? launch_dropout_of<kElemF16, true>(a, blocks, sm_count, stream)
                   : launch_dropout_of<kElemF16, false>(a, blocks, sm_count, stream);
    case kElemF32:
        return add ? launch_dropout_of<kElemF32, true>(a, blocks, sm_count, stream)
                   : launch_dropout_of<kElemF32, false>(a, blocks, sm_count, stream);
    default:
        return cudaErrorInvalidValue;
    }
}

}  // namespace dradd
