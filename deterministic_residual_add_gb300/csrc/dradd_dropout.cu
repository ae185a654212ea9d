// dradd_dropout.cu -- dropout, and dropout + residual add, of row-strided
// tensors: out = kept ? RN(x scale) : 0, plus residual where there is one
// (one fp32 addition), rounded once to the element type.
//
// Bound by the memory: 2 (3) elements of traffic an element, and one
// generator call for 8 of them (dradd_philox.cuh).  Measured on GB300 (device
// time, inputs and outputs of every pass its own; share of the 6.79 TB/s a
// copy reaches): 8192 x 4096 bf16 22.6 us (87 %), with the residual 31.0 (95
// %); 15322 x 2315 fp16 31.6 us (66 %, the flat kernel: 1.25 generator calls
// and about 25 instructions of shifting a vector), with the residual 36.4 (86
// %); 8192 x 4096 bf16 in unaligned rows 4099 apart 42.4 us (47 %, the ragged
// kernel), with the residual 46.9 (63 %).  The sweeps noted in the code shared
// their outputs between passes, which reads about a microsecond lower.
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

// ---------------------------------------------------- contiguous, any width
// Rows that no vector width divides, back to back: the tensor is read as one
// run of aligned vectors of 8, and a vector that starts at column c of its
// row takes its numbers from blocks c / 8 and c / 8 + 1, shifted by c % 8.
// The second of these is the next lane's first, so it comes by a shuffle; a
// warp goes through kFlatVectors x 32 vectors in a row, in which only the last
// lane of the last one has to draw an extra block.  A vector that reaches the
// end of a row draws the blocks it lacks itself.
constexpr int kFlatVectors = 4;

// halves >> s: the 16-bit numbers s, s + 1, ... s + 7 of the 16 in (a, b).
__device__ __forceinline__ uint4 halves_from(const uint4& a, const uint4& b, uint32_t s)
{
    uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 6; ++i)
        w[i] = (s & 4) ? w[i + 2] : w[i];
#pragma unroll
    for (int i = 0; i < 5; ++i)
        w[i] = (s & 2) ? w[i + 1] : w[i];
    const uint32_t bits = (s & 1) * 16;
    return make_uint4(__funnelshift_r(w[0], w[1], bits), __funnelshift_r(w[1], w[2], bits),
                      __funnelshift_r(w[2], w[3], bits), __funnelshift_r(w[3], w[4], bits));
}

template <int E, bool ADD>
__global__ void __launch_bounds__(kDropoutThreads) dropout_flat_kernel(const DropoutArgs a, int64_t step_rows,
                                                                       uint32_t step_cols, uint32_t vec_rows,
                                                                       uint32_t vec_cols)
{
    using V = typename Elem<E>::Block;
    using T = typename Elem<E>::T;
    wait_prior_grids();
    allow_next_grid();
    const uint2 offset = drop_offset(a.drop);
    const int lane = threadIdx.x & 31;
    const uint32_t hidden = static_cast<uint32_t>(a.hidden);
    const int64_t n = a.n_rows * a.hidden;
    const T* const x = static_cast<const T*>(a.x);
    const T* const r = static_cast<const T*>(a.residual);
    T* const out = static_cast<T*>(a.out);
    const int64_t warps = static_cast<int64_t>(gridDim.x) * (kDropoutThreads / 32);
    int64_t chunk = static_cast<int64_t>(blockIdx.x) * (kDropoutThreads / 32) + (threadIdx.x >> 5);
    const int64_t chunks = (n + 256 * kFlatVectors - 1) / (256 * kFlatVectors);
    // (row, col) of the lane's first element of the chunk
    const int64_t start = chunk * (256 * kFlatVectors) + lane * 8;
    int64_t row0 = start / hidden;
    uint32_t col0 = static_cast<uint32_t>(start - row0 * hidden);
    for (; chunk < chunks; chunk += warps) {
        const int64_t v0 = chunk * (32 * kFlatVectors) + lane;
        V xv[kFlatVectors], rv[kFlatVectors];
#pragma unroll
        for (int i = 0; i < kFlatVectors; ++i) {
            if ((v0 + 32 * i) * 8 + 8 <= n) {
                ld_block_stream(x, v0 + 32 * i, xv[i]);
                if constexpr (ADD)
                    ld_block_stream(r, v0 + 32 * i, rv[i]);
            }
        }
        uint32_t row = static_cast<uint32_t>(row0), col = col0;
        uint4 mine = drop_bits(a.drop, offset, col >> 3, row);
#pragma unroll
        for (int i = 0; i < kFlatVectors; ++i) {
            // the next vector's place, and its first block
            uint32_t next_row = row + vec_rows, next_col = col + vec_cols;
            if (next_col >= hidden) {
                next_col -= hidden;
                ++next_row;
            }
            uint4 after = mine;
            if (i + 1 < kFlatVectors)
                after = drop_bits(a.drop, offset, next_col >> 3, next_row);
            // block col / 8 + 1 of the row: the next lane's, where it is in the same row
            uint4 second;
            second.x = __shfl_down_sync(0xFFFFFFFFu, mine.x, 1);
            second.y = __shfl_down_sync(0xFFFFFFFFu, mine.y, 1);
            second.z = __shfl_down_sync(0xFFFFFFFFu, mine.z, 1);
            second.w = __shfl_down_sync(0xFFFFFFFFu, mine.w, 1);
            if (i + 1 < kFlatVectors) {
                const uint4 first = make_uint4(__shfl_sync(0xFFFFFFFFu, after.x, 0), __shfl_sync(0xFFFFFFFFu, after.y, 0),
                                               __shfl_sync(0xFFFFFFFFu, after.z, 0), __shfl_sync(0xFFFFFFFFu, after.w, 0));
                if (lane == 31)
                    second = first;
            } else if (lane == 31) {
                second = drop_bits(a.drop, offset, (col >> 3) + 1, row);
            }
            uint4 bits = halves_from(mine, second, col & 7);
            if (col + 8 >= hidden) {
                // the last hidden - col elements of a row, then the first of
                // the next (whose numbers the next lane has, not this row's)
                const uint4 ours = drop_bits(a.drop, offset, (col >> 3) + 1, row);
                const uint4 theirs = drop_bits(a.drop, offset, 0, row + 1);
                const uint32_t here = hidden - col;  // 1 .. 8
                bits = halves_from(mine, ours, col & 7);
                const uint4 shifted = halves_from(make_uint4(0u, 0u, 0u, 0u), theirs, 8 - here);
                const uint32_t odd = (here & 1) ? 0x0000FFFFu : 0u;  // of word here / 2: the low half is ours
                uint32_t* b = &bits.x;
                const uint32_t* t = &shifted.x;
#pragma unroll
                for (uint32_t k = 0; k < 4; ++k) {
                    const uint32_t keep = k < (here >> 1) ? 0xFFFFFFFFu : k == (here >> 1) ? odd : 0u;
                    b[k] = (b[k] & keep) | (t[k] & ~keep);
                }
            }
            const int64_t v = v0 + 32 * i;
            if (v * 8 + 8 <= n) {
                float f[8];
                Elem<E>::unpack(xv[i], f);
                if (a.drop.drops) {
#pragma unroll
                    for (int e = 0; e < 8; e += 2) {
                        mul2_rn(f[e], f[e + 1], a.drop.scale, a.drop.scale, f[e], f[e + 1]);
                        f[e] = kept(bits, e, a.drop.limit) ? f[e] : 0.0f;
                        f[e + 1] = kept(bits, e + 1, a.drop.limit) ? f[e + 1] : 0.0f;
                    }
                }
                if constexpr (ADD) {
                    float g[8];
                    Elem<E>::unpack(rv[i], g);
#pragma unroll
                    for (int e = 0; e < 8; e += 2)
                        add2_rn(g[e], g[e + 1], f[e], f[e + 1], f[e], f[e + 1]);
                }
                st_block_stream(out, v, Elem<E>::pack(f));
            } else if (v * 8 < n) {
                // the tensor's last elements
                for (int e = 0; e < static_cast<int>(n - v * 8); ++e) {
                    const uint32_t word = e < 2 ? bits.x : e < 4 ? bits.y : e < 6 ? bits.z : bits.w;
                    const bool keep = !a.drop.drops || ((e & 1) ? word : word << 16) > a.drop.limit;
                    float f = keep ? __fmul_rn(Elem<E>::widen(x[v * 8 + e]), a.drop.scale) : 0.0f;
                    if constexpr (ADD)
                        f = __fadd_rn(Elem<E>::widen(r[v * 8 + e]), f);
                    out[v * 8 + e] = Elem<E>::narrow(f);
                }
            }
            row = next_row;
            col = next_col;
            mine = after;
        }
        row0 += step_rows;
        col0 += step_cols;
        if (col0 >= hidden) {
            col0 -= hidden;
            ++row0;
        }
    }
}

// ------------------------------------------------------- any layout at all
// A warp takes 256 columns of a row.  Lane l draws
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
cudaError_t launch_dropout_of(const DropoutArgs& a, DropoutLayout layout, int sm_count, cudaStream_t stream)
{
    const int64_t per_row = layout == kDropoutBlocks ? a.hidden >> 3 : (a.hidden + 255) / 256;
    const int64_t per_cta = layout == kDropoutBlocks ? kDropoutThreads : kDropoutThreads / 32;
    const int64_t units = layout == kDropoutFlat
                              ? (a.n_rows * a.hidden + 256 * kFlatVectors - 1) / (256 * kFlatVectors)
                              : a.n_rows * per_row;
    const int64_t wanted = (units + per_cta - 1) / per_cta;
    const int64_t most = static_cast<int64_t>(sm_count) * kDropoutCtasPerSm;
    const int grid = static_cast<int>(wanted < most ? wanted : most);
    const int64_t step = grid * per_cta;
    if (layout == kDropoutFlat) {
        const int64_t elements = step * 256 * kFlatVectors;
        return launch(dropout_flat_kernel<E, ADD>, grid, kDropoutThreads, 0, false, stream, a, elements / a.hidden,
                      static_cast<uint32_t>(elements % a.hidden), static_cast<uint32_t>(256 / a.hidden),
                      static_cast<uint32_t>(256 % a.hidden));
    }
    // rows and blocks are 32-bit in the kernels: both, and one step more, fit
    const uint32_t span = static_cast<uint32_t>(per_row);
    const uint32_t step_rows = static_cast<uint32_t>(step / per_row), rest = static_cast<uint32_t>(step % per_row);
    return launch(layout == kDropoutBlocks ? dropout_blocks_kernel<E, ADD> : dropout_ragged_kernel<E, ADD>, grid,
                  kDropoutThreads, 0, false, stream, a, span, step_rows, rest);
}

}  // namespace

cudaError_t launch_dropout(const DropoutArgs& a, int elem, DropoutLayout layout, int sm_count, cudaStream_t stream)
{
    const bool add = a.residual != nullptr;
    switch (elem) {
    case kElemBf16:
        return add ? launch_dropout_of<kElemBf16, true>(a, layout, sm_count, stream)
                   : launch_dropout_of<kElemBf16, false>(a, layout, sm_count, stream);
    case kElemF16:
        return add ? launch_dropout_of<kElemF16, true>(a, layout, sm_count, stream)
                   : launch_dropout_of<kElemF16, false>(a, layout, sm_count, stream);
    case kElemF32:
        return add ? launch_dropout_of<kElemF32, true>(a, layout, sm_count, stream)
                   : launch_dropout_of<kElemF32, false>(a, layout, sm_count, stream);
    default:
        return cudaErrorInvalidValue;
    }
}

}  // namespace dradd
