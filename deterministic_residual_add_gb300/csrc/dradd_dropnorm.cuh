// dradd_dropnorm.cuh -- dropout + residual add + RMSNorm, and its gradients.
//
// Forward, per row (the row function of add_rmsnorm_fwd with the dropout in
// front of it, so p = 0 gives its bits):
//   acc = residual + (kept ? RN(x scale) : 0); residual_out = E(acc)
//   out = E((acc * inv) * w), inv = 1 / sqrt(S / hidden + eps),
// S the canonical pairwise sum of acc^2 (see dradd_kernels.cuh).
//
// Backward from h = residual_out (the rounded sum is what a training step
// keeps), with g = dout * w:
//   S1 = sum h^2, S2 = sum g h, in a fixed order
//   inv from S1; c = -inv * (inv * (S2 / hidden))
//   d = dresidual_out + inv * (g + h * c)
//   dresidual = E(d); dx = E(kept ? d scale : 0)
//   dweight[i] = sum over rows of dout * (h * inv), in fp32: every CTA (part)
//   adds its rows in order and a second kernel adds the parts in a fixed
//   order, so the bits depend on the shape and the element type alone.
//
// Bound by the memory: 4 elements of traffic an element forward, 5 backward.
// Rows of P > 256 (P: hidden rounded up to a power of two; backward, 2-byte
// types, P > 1024) go through shared memory, one CTA a row, staged `stages`
// rows ahead by bulk copies.  The forward keeps acc in registers between its
// two passes; the backward pass keeps h and dout there up to two blocks of 8
// a thread, so that the slot is refilled at once, and reads longer rows from
// the slot again.  Narrower rows take a warp (or 8 or 16 lanes) each, with
// the next rows on their way into shared memory that only their lane reads.
//
// Measured on GB300 (device time, inputs and outputs of every pass its own;
// share of the 6.79 TB/s a copy reaches): forward bf16 4096 x 8192 42.2 us (94
// %), 16384 x 4096 88.0 (90 %), 4096 x 1024 6.5 (76 %), fp32 8192 x 4096 84.5
// (93 %); backward bf16 8192 x 8192 109.8 us (90 %), 4096 x 4096 33.2 (74 %),
// 4096 x 1024 13.0 (47 %; the sums of dweight's parts are 3 us of any call),
// fp32 1999 x 5120 37.9 (80 %).  The sweeps noted in the code shared their
// outputs between passes, which reads up to 3 us lower.
#pragma once

#include "dradd_elem.cuh"
#include "dradd_internal.h"
#include "dradd_kernels.cuh"
#include "dradd_train_internal.h"

namespace dradd {

// ------------------------------------------------------------- block helpers
// acc of one block; the residual sum is stored.
template <int E>
__device__ __forceinline__ void fwd_block(const DropNormArgs& a, const uint2& offset,
                                          const typename Elem<E>::Block& xv, const typename Elem<E>::Block& rv,
                                          int64_t row, int b, float (&acc)[8])
{
    using T = typename Elem<E>::T;
    float r[8];
    Elem<E>::unpack(xv, acc);
    Elem<E>::unpack(rv, r);
    if (a.drop.drops)
        drop8(acc, a.drop, offset, static_cast<uint32_t>(b), static_cast<uint32_t>(row));
#pragma unroll
    for (int e = 0; e < 8; e += 2)
        add2_rn(acc[e], acc[e + 1], r[e], r[e + 1], acc[e], acc[e + 1]);
    st_block_stream(static_cast<T*>(a.residual_out) + row * a.hidden, b, Elem<E>::pack(acc));
}

// out of one block.
template <int E>
__device__ __forceinline__ void fwd_finish(const DropNormArgs& a, float (&acc)[8], float inv,
                                           const typename Elem<E>::Block& wv, int64_t row, int b)
{
    using T = typename Elem<E>::T;
    float w[8];
    Elem<E>::unpack(wv, w);
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
        mul2_rn(acc[e], acc[e + 1], inv, inv, acc[e], acc[e + 1]);
        mul2_rn(acc[e], acc[e + 1], w[e], w[e + 1], acc[e], acc[e + 1]);
    }
    st_block_stream(static_cast<T*>(a.out) + row * a.hidden, b, Elem<E>::pack(acc));
}

// The block's parts of sum h^2 and sum g h (g = dout w): two chains of fused
// multiply-adds each, two to an instruction, then their sum.
template <int E>
__device__ __forceinline__ void bwd_sums(const float (&h)[8], const float (&dout)[8],
                                         const typename Elem<E>::Block& wv, float& s1, float& s2)
{
    float g[8];
    Elem<E>::unpack(wv, g);
#pragma unroll
    for (int e = 0; e < 8; e += 2)
        mul2_rn(dout[e], dout[e + 1], g[e], g[e + 1], g[e], g[e + 1]);
    float a0, a1, b0, b1;
    mul2_rn(h[0], h[1], h[0], h[1], a0, a1);
    mul2_rn(h[0], h[1], g[0], g[1], b0, b1);
#pragma unroll
    for (int e = 2; e < 8; e += 2) {
        fma2_rn(h[e], h[e + 1], h[e], h[e + 1], a0, a1, a0, a1);
        fma2_rn(h[e], h[e + 1], g[e], g[e + 1], b0, b1, b0, b1);
    }
    s1 = __fadd_rn(a0, a1);
    s2 = __fadd_rn(b0, b1);
}

// The gradients of one block, and its rows' share of dweight.
template <int E>
__device__ __forceinline__ void bwd_finish(const DropNormArgs& a, const uint2& offset, const float (&h)[8],
                                           const float (&dout)[8], const typename Elem<E>::Block& wv,
                                           const typename Elem<E>::Block& dv, float inv, float c, int64_t row, int b,
                                           float (&dw)[8])
{
    using T = typename Elem<E>::T;
    float w[8], d[8];
    Elem<E>::unpack(wv, w);
    Elem<E>::unpack(dv, d);
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
        float x0, x1;
        mul2_rn(h[e], h[e + 1], inv, inv, x0, x1);
        fma2_rn(dout[e], dout[e + 1], x0, x1, dw[e], dw[e + 1], dw[e], dw[e + 1]);
        mul2_rn(dout[e], dout[e + 1], w[e], w[e + 1], w[e], w[e + 1]);
        fma2_rn(h[e], h[e + 1], c, c, w[e], w[e + 1], w[e], w[e + 1]);
        fma2_rn(w[e], w[e + 1], inv, inv, d[e], d[e + 1], d[e], d[e + 1]);
    }
    st_block_stream(static_cast<T*>(a.dresidual) + row * a.hidden, b, Elem<E>::pack(d));
    if (a.dx) {
        if (a.drop.drops)
            drop8(d, a.drop, offset, static_cast<uint32_t>(b), static_cast<uint32_t>(row));
        st_block_stream(static_cast<T*>(a.dx) + row * a.hidden, b, Elem<E>::pack(d));
    }
}

// c of the row: -inv^2 S2 / hidden.
__device__ __forceinline__ float bwd_coefficient(const DropNormArgs& a, float s2, float inv)
{
    const float mean = a.inv_hidden != 0.0f ? __fmul_rn(s2, a.inv_hidden)
                                            : __fdiv_rn(s2, static_cast<float>(a.hidden));
    return -__fmul_rn(inv, __fmul_rn(inv, mean));
}

// ------------------------------------------------------------- narrow rows
// L lanes a row (8, 16 or 32), K blocks of 8 a lane: P = 8 L K, up to 256
// (K = 1), backward up to 1024 for 2-byte types.  A CTA takes (threads x 32 / L) rows at a time.  Every thread copies its
// blocks of the next rows into a ring of shared memory that only it reads.
constexpr int kNarrowThreads = 256;

// N tensors, K blocks each: slots of the ring, and its bytes.
template <int E, int N, int K>
struct NarrowRing {
    static constexpr uint32_t kPiece = kNarrowThreads * 16;
    static constexpr int kVec = E == kElemF32 ? 2 : 1;
    static constexpr uint32_t kSlotBytes = N * K * kVec * kPiece;
    static constexpr int kSlots = narrow_slots(E, N, K);
    static constexpr uint32_t kBytes = kSlots * kSlotBytes;
    static_assert(kBytes == narrow_ring_bytes(E, N, K), "the host sizes the same ring");
    static __device__ __forceinline__ uint32_t at(uint32_t slot, int tensor, int j)
    {
        return slot + (tensor * K + j) * kVec * kPiece;
    }
    static __device__ __forceinline__ uint32_t after(uint32_t slot, uint32_t ring)
    {
        return slot == ring + (kSlots - 1) * kSlotBytes ? ring : slot + kSlotBytes;
    }
};

// Copies row `row` of the tensors into a slot, or nothing past the last row.
template <int E, int N, int L, int K>
__device__ __forceinline__ void narrow_issue(const void* const (&src)[N], int64_t row, const DropNormArgs& a,
                                             uint32_t slot, int t)
{
    using T = typename Elem<E>::T;
    using Ring = NarrowRing<E, N, K>;
    if (row < a.n_rows) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if (!src[i])
                continue;
            const T* p = static_cast<const T*>(src[i]) + row * a.hidden + t * 8;
#pragma unroll
            for (int j = 0; j < K; ++j)
                if (8 * (t + j * L) < a.hidden)
                    copy_ahead_block(Ring::at(slot, i, j), Ring::kPiece, p + j * L * 8);
        }
    }
    copy_ahead_commit();
}

template <int E, int L>
__global__ void __launch_bounds__(kNarrowThreads) drop_norm_fwd_narrow(const DropNormArgs a)
{
    using T = typename Elem<E>::T;
    using V = typename Elem<E>::Block;
    using Ring = NarrowRing<E, 2, 1>;
    extern __shared__ __align__(128) unsigned char stage_mem[];
    const int t = threadIdx.x & (L - 1);
    const int nblocks = a.hidden >> 3;
    const uint32_t ring = smem_u32(stage_mem) + threadIdx.x * 16;
    const int64_t step = static_cast<int64_t>(gridDim.x) * (kNarrowThreads / L);
    const int64_t first = static_cast<int64_t>(blockIdx.x) * (kNarrowThreads / L) + threadIdx.x / L;
    // rows of one warp start together, so every lane of it makes the same
    // number of steps and takes part in the shuffles
    const int64_t lead = first - (threadIdx.x & 31) / L;
    wait_prior_grids();
    allow_next_grid();
    const void* const src[2] = {a.x, a.residual};
    uint32_t in = ring, slot = ring;
#pragma unroll
    for (int i = 0; i < Ring::kSlots - 1; ++i) {
        narrow_issue<E, 2, L, 1>(src, first + i * step, a, in, t);
        in = Ring::after(in, ring);
    }
    const uint2 offset = drop_offset(a.drop);
    V wv = V{};
    if (t < nblocks)
        ld_block(static_cast<const T*>(a.weight), t, wv);
    for (int64_t base = 0; lead + base < a.n_rows; base += step) {
        const int64_t row = first + base;
        narrow_issue<E, 2, L, 1>(src, row + (Ring::kSlots - 1) * step, a, in, t);
        in = Ring::after(in, ring);
        copy_ahead_wait<Ring::kSlots - 1>();
        const bool in_row = row < a.n_rows && t < nblocks;
        float acc[8], part = 0.0f;
        if (in_row) {
            V xv, rv;
            lds_block(Ring::at(slot, 0, 0), Ring::kPiece, xv);
            lds_block(Ring::at(slot, 1, 0), Ring::kPiece, rv);
            fwd_block<E>(a, offset, xv, rv, row, t, acc);
            part = fold8_squares(acc);
        }
        const float inv = inv_rms(butterfly_sum(part, L), a.hidden, a.inv_hidden, a.eps);
        if (in_row)
            fwd_finish<E>(a, acc, inv, wv, row, t);
        slot = Ring::after(slot, ring);
    }
}

template <int E, int L, int K>
__global__ void __launch_bounds__(kNarrowThreads, 2) drop_norm_bwd_narrow(const DropNormArgs a)
{
    using T = typename Elem<E>::T;
    using V = typename Elem<E>::Block;
    using Ring = NarrowRing<E, 3, K>;
    extern __shared__ __align__(128) unsigned char stage_mem[];
    const int t = threadIdx.x & (L - 1);
    const int nblocks = a.hidden >> 3;
    const uint32_t ring = smem_u32(stage_mem) + threadIdx.x * 16;
    const int64_t step = static_cast<int64_t>(gridDim.x) * (kNarrowThreads / L);
    const int64_t first = static_cast<int64_t>(blockIdx.x) * (kNarrowThreads / L) + threadIdx.x / L;
    const int64_t lead = first - (threadIdx.x & 31) / L;  // as in the forward
    wait_prior_grids();
    allow_next_grid();
    const void* const src[3] = {a.h, a.dout, a.dresidual_out};
    uint32_t in = ring, slot = ring;
#pragma unroll
    for (int i = 0; i < Ring::kSlots - 1; ++i) {
        narrow_issue<E, 3, L, K>(src, first + i * step, a, in, t);
        in = Ring::after(in, ring);
    }
    const uint2 offset = drop_offset(a.drop);
    __shared__ V weights[L * K];
    for (int i = threadIdx.x; i < L * K; i += kNarrowThreads) {
        V v = V{};
        if (i < nblocks)
            ld_block(static_cast<const T*>(a.weight), i, v);
        weights[i] = v;
    }
    __syncthreads();
    float dw[K][8] = {};
    for (int64_t base = 0; lead + base < a.n_rows; base += step) {
        const int64_t row = first + base;
        const bool active = row < a.n_rows;
        narrow_issue<E, 3, L, K>(src, row + (Ring::kSlots - 1) * step, a, in, t);
        in = Ring::after(in, ring);
        copy_ahead_wait<Ring::kSlots - 1>();
        float p1[K], p2[K];
#pragma unroll
        for (int j = 0; j < K; ++j) {
            // a slot that was not filled is read all the same and counts nothing
            V hv, gv;
            lds_block(Ring::at(slot, 0, j), Ring::kPiece, hv);
            lds_block(Ring::at(slot, 1, j), Ring::kPiece, gv);
            float h[8], g[8];
            Elem<E>::unpack(hv, h);
            Elem<E>::unpack(gv, g);
            bwd_sums<E>(h, g, weights[t + j * L], p1[j], p2[j]);
            const bool in_row = active && t + j * L < nblocks;
            p1[j] = in_row ? p1[j] : 0.0f;
            p2[j] = in_row ? p2[j] : 0.0f;
        }
        const float inv =
            inv_rms(butterfly_sum(fold_k<K>(p1), L), a.hidden, a.inv_hidden, a.eps);
        const float c = bwd_coefficient(a, butterfly_sum(fold_k<K>(p2), L), inv);
#pragma unroll
        for (int j = 0; j < K; ++j) {
            const int b = t + j * L;
            if (active && b < nblocks) {
                V hv, gv, dv = V{};
                lds_block(Ring::at(slot, 0, j), Ring::kPiece, hv);
                lds_block(Ring::at(slot, 1, j), Ring::kPiece, gv);
                if (a.dresidual_out)
                    lds_block(Ring::at(slot, 2, j), Ring::kPiece, dv);
                float h[8], g[8];
                Elem<E>::unpack(hv, h);
                Elem<E>::unpack(gv, g);
                bwd_finish<E>(a, offset, h, g, weights[b], dv, inv, c, row, b, dw[j]);
            }
        }
        slot = Ring::after(slot, ring);
    }
    if (!a.partials)
        return;
    // the CTA's part: a warp's groups by butterfly, then the warps in order
    copy_ahead_wait<0>();
    __syncthreads();
    float* const sums = reinterpret_cast<float*>(stage_mem);
    constexpr int P = 8 * L * K;
#pragma unroll
    for (int j = 0; j < K; ++j) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float v = dw[j][e];
#pragma unroll
            for (int d = L; d < 32; d <<= 1)
                v = __fadd_rn(v, __shfl_xor_sync(0xFFFFFFFFu, v, d));
            if ((threadIdx.x & 31) < L)
                sums[(threadIdx.x >> 5) * P + (t + j * L) * 8 + e] = v;
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < a.hidden; i += kNarrowThreads) {
        float v = sums[i];
#pragma unroll
        for (int k = 1; k < kNarrowThreads / 32; ++k)
            v = __fadd_rn(v, sums[k * P + i]);
        a.partials[static_cast<int64_t>(blockIdx.x) * a.hidden + i] = v;
    }
}

// --------------------------------------------------------------- wide rows
// One CTA a row, T threads of K blocks: P = 8 T K.  Rows reach the threads
// through stages of shared memory (STAGED) or straight from global memory
// (buffers that are not device memory, rows of which two do not fit).

// The forward's T threads cover the padded row exactly, as the canonical
// tree wants; the backward pass, whose sums have no such order to keep,
// takes as many whole warps as the row has work for.
//
// Resident CTAs per SM the kernels are compiled for: forward 1024 threads of
// 64 registers, or 512 of 128; backward likewise, and 640 of about 100 for
// two blocks a thread in CTAs of 256 to 320 threads (2-byte types).
constexpr int fwd_min_blocks(int T, int K) { return K <= 2 ? 1024 / T : 512 / T; }
// Between its two passes the backward kernel holds h and dout in registers,
// widened; more than two blocks a thread it reads from the stage again (held
// as they came, four blocks: 61.8 us against 57.8 at 2048 x 16384 bf16).
__host__ __device__ constexpr bool bwd_holds(int K) { return K <= 2; }

// N arrays of rows staged in turn: a ring of `stages` slots, each one row of
// every array, filled by thread 0.
template <int N>
struct RowRing {
    unsigned char* mem;
    uint64_t* bars;
    const unsigned char* src[N];
    uint32_t row_bytes;
    int stages;
    uint64_t policy;

    __device__ __forceinline__ const unsigned char* slot(int s) const
    {
        return mem + static_cast<size_t>(s) * N * row_bytes;
    }
    // The row's lines into L2, while the previous grid finishes: a hint that
    // moves nothing to the SM, so the copies issued after the wait still read
    // what the memory holds then.
    __device__ __forceinline__ void prefetch(int64_t row) const
    {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (src[i])
                prefetch_l2(src[i] + row * static_cast<int64_t>(row_bytes), row_bytes);
    }
    __device__ __forceinline__ void issue(int s, int64_t row) const
    {
        unsigned char* dst = mem + static_cast<size_t>(s) * N * row_bytes;
        uint32_t bytes = 0;
#pragma unroll
        for (int i = 0; i < N; ++i)
            bytes += src[i] ? row_bytes : 0u;
        mbar_arrive_expect_tx(&bars[s], bytes);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if (src[i])
                bulk_copy_g2s(dst + i * row_bytes, src[i] + row * static_cast<int64_t>(row_bytes), row_bytes,
                              &bars[s], policy);
        }
    }
};

// After an expired wait: thread 0 records it and waits, with a limit, for
// the copies of slots that were filled and not yet taken (`pending` of them
// from slot s), so that none lands after the CTA has gone.
__device__ __forceinline__ void give_up(const DropNormArgs& a, uint64_t* bars, int s, uint32_t parity, int64_t pending)
{
    atomicOr(a.status, kDeviceStatusTimeout);
    for (int64_t i = 0; i < pending; ++i) {
        bool landed = false;
        for (int r = 0; r < kDrainRounds && !landed; ++r)
            landed = mbar_wait_bounded(&bars[s], parity, a.wait_limit_ns);
        if (!landed)
            atomicOr(a.status, kDeviceStatusUndrained);
        if (++s == a.stages) {
            s = 0;
            parity ^= 1u;
        }
    }
}

template <int E, int T, int K, bool STAGED>
__global__ void __launch_bounds__(T, fwd_min_blocks(T, K)) drop_norm_fwd_wide(const DropNormArgs a)
{
    using X = typename Elem<E>::T;
    using V = typename Elem<E>::Block;
    constexpr int W = T / 32;
    extern __shared__ __align__(128) unsigned char stage_mem[];
    __shared__ float red[2][K * W];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int nblocks = a.hidden >> 3;
    const int64_t stride = gridDim.x;
    RowRing<2> ring;
    if constexpr (STAGED) {
        ring.mem = stage_mem;
        ring.row_bytes = static_cast<uint32_t>(a.hidden * sizeof(X));
        ring.stages = a.stages;
        ring.bars = reinterpret_cast<uint64_t*>(stage_mem + static_cast<size_t>(a.stages) * 2 * ring.row_bytes);
        ring.src[0] = static_cast<const unsigned char*>(a.x);
        ring.src[1] = static_cast<const unsigned char*>(a.residual);
        ring.policy = l2_policy_evict_first();
        if (tid == 0) {
            ring.prefetch(blockIdx.x);
            for (int s = 0; s < a.stages; ++s)
                mbar_init(&ring.bars[s], 1);
            fence_mbar_init();
        }
        __syncthreads();
    }
    wait_prior_grids();
    allow_next_grid();
    if constexpr (STAGED) {
        if (tid == 0) {
            for (int s = 0; s < a.stages && blockIdx.x + s * stride < a.n_rows; ++s)
                ring.issue(s, blockIdx.x + s * stride);
        }
    }
    const uint2 offset = drop_offset(a.drop);
    V wv[K];
#pragma unroll
    for (int j = 0; j < K; ++j) {
        const int b = tid + j * T;
        if (block_in_row<K>(j, b, nblocks))
            ld_block(static_cast<const X*>(a.weight), b, wv[j]);
    }
    int s = 0, buf = 0;
    uint32_t parity = 0;
    for (int64_t row = blockIdx.x; row < a.n_rows; row += stride) {
        bool ok = true;
        const X *xs, *rs;
        if constexpr (STAGED) {
            ok = mbar_wait_bounded(&ring.bars[s], parity, a.wait_limit_ns);
            xs = reinterpret_cast<const X*>(ring.slot(s));
            rs = xs + a.hidden;
        } else {
            xs = static_cast<const X*>(a.x) + row * a.hidden;
            rs = static_cast<const X*>(a.residual) + row * a.hidden;
        }
        float acc[K][8], part[K];
#pragma unroll
        for (int j = 0; j < K; ++j) {
            const int b = tid + j * T;
            part[j] = 0.0f;
            if (block_in_row<K>(j, b, nblocks)) {
                V xv, rv;
                ld_block(xs, b, xv);
                ld_block(rs, b, rv);
                fwd_block<E>(a, offset, xv, rv, row, b, acc[j]);
                part[j] = fold8_squares(acc[j]);
            }
        }
        int jsub;
        const float v = warp_halving_sum<K>(part, lane, jsub);
        if (lane < K)
            red[buf][jsub * W + warp] = v;
        if constexpr (STAGED) {
            // every thread has read the slot; an expired wait ends the CTA
            if (__syncthreads_or(!ok)) {
                if (tid == 0) {
                    const int64_t left = (a.n_rows - row + stride - 1) / stride;
                    give_up(a, ring.bars, s, parity, left < a.stages ? left : a.stages);
                }
                return;
            }
            if (tid == 0 && row + a.stages * stride < a.n_rows) {
                fence_proxy_async_smem();
                ring.issue(s, row + a.stages * stride);
            }
        } else {
            __syncthreads();
        }
        const float inv = inv_rms(cross_warp_sum<K, W>(red[buf], lane), a.hidden, a.inv_hidden, a.eps);
#pragma unroll
        for (int j = 0; j < K; ++j) {
            const int b = tid + j * T;
            if (block_in_row<K>(j, b, nblocks))
                fwd_finish<E>(a, acc[j], inv, wv[j], row, b);
        }
        buf ^= 1;
        if constexpr (STAGED) {
            if (++s == a.stages) {
                s = 0;
                parity ^= 1u;
            }
        }
    }
}

// MAXT threads at most, MINB CTAs an SM.
template <int E, int K, int MAXT, int MINB, bool STAGED>
__global__ void __launch_bounds__(MAXT, MINB) drop_norm_bwd_wide(const DropNormArgs a)
{
    using X = typename Elem<E>::T;
    using V = typename Elem<E>::Block;
    constexpr bool HOLD = bwd_holds(K);
    constexpr int H = HOLD ? K : 1;
    extern __shared__ __align__(128) unsigned char stage_mem[];
    __shared__ float red1[2][16], red2[2][16];
    const int T = blockDim.x, W = T >> 5;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int nblocks = a.hidden >> 3;
    const int64_t stride = gridDim.x;
    RowRing<3> ring;
    if constexpr (STAGED) {
        ring.mem = stage_mem;
        ring.row_bytes = static_cast<uint32_t>(a.hidden * sizeof(X));
        ring.stages = a.stages;
        ring.bars = reinterpret_cast<uint64_t*>(stage_mem + static_cast<size_t>(a.stages) * 3 * ring.row_bytes);
        ring.src[0] = static_cast<const unsigned char*>(a.h);
        ring.src[1] = static_cast<const unsigned char*>(a.dout);
        ring.src[2] = static_cast<const unsigned char*>(a.dresidual_out);
        ring.policy = l2_policy_evict_first();
        if (tid == 0) {
            ring.prefetch(blockIdx.x);
            for (int s = 0; s < a.stages; ++s)
                mbar_init(&ring.bars[s], 1);
            fence_mbar_init();
        }
        __syncthreads();
    }
    wait_prior_grids();
    allow_next_grid();
    if constexpr (STAGED) {
        if (tid == 0) {
            for (int s = 0; s < a.stages && blockIdx.x + s * stride < a.n_rows; ++s)
                ring.issue(s, blockIdx.x + s * stride);
        }
    }
    const uint2 offset = drop_offset(a.drop);
    const X* wrow = static_cast<const X*>(a.weight);
    // fp32 weights stay in registers too where the row does: shared memory
    // leaves the L1 cache too small for them (2048 x 4096 31.6 us, read again
    // every row 33.5); 2-byte ones fit, and the registers do more elsewhere
    // (16384 x 4096 bf16 110 us, held 117).
    constexpr bool HOLD_WEIGHTS = HOLD && E == kElemF32;
    V wv[H];
    if constexpr (HOLD_WEIGHTS) {
#pragma unroll
        for (int j = 0; j < K; ++j)
            ld_block(wrow, j < K - 1 || tid + j * T < nblocks ? tid + j * T : nblocks - 1, wv[j]);
    }
    float dw[K][8] = {};
    int s = 0, buf = 0;
    uint32_t parity = 0;
    for (int64_t row = blockIdx.x; row < a.n_rows; row += stride) {
        bool ok = true;
        const X *hs, *gs, *ds;
        if constexpr (STAGED) {
            ok = mbar_wait_bounded(&ring.bars[s], parity, a.wait_limit_ns);
            hs = reinterpret_cast<const X*>(ring.slot(s));
            gs = hs + a.hidden;
            ds = gs + a.hidden;
        } else {
            hs = static_cast<const X*>(a.h) + row * a.hidden;
            gs = static_cast<const X*>(a.dout) + row * a.hidden;
            ds = static_cast<const X*>(a.dresidual_out) + row * a.hidden;
        }
        float h[H][8], g[H][8];
        V dv[H];
        const auto load = [&](int b, int i) {
            V v;
            ld_block(hs, b, v);
            Elem<E>::unpack(v, h[i]);
            ld_block(gs, b, v);
            Elem<E>::unpack(v, g[i]);
            if constexpr (!HOLD_WEIGHTS)
                ld_block(wrow, b, wv[i]);
        };
        // T is nblocks / K rounded up to whole warps, so only the last of a
        // thread's blocks may lie past the row; it is then read from the last
        // block and counts nothing, which keeps the loads free of branches.
        float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
        for (int j = 0; j < K; ++j) {
            const int i = HOLD ? j : 0;
            const bool in_row = j < K - 1 || tid + j * T < nblocks;
            const int b = in_row ? tid + j * T : nblocks - 1;
            load(b, i);
            if constexpr (HOLD) {
                dv[i] = V{};
                if (a.dresidual_out)
                    ld_block(ds, b, dv[i]);
            }
            float p1, p2;
            bwd_sums<E>(h[i], g[i], wv[i], p1, p2);
            s1 = __fadd_rn(s1, in_row ? p1 : 0.0f);
            s2 = __fadd_rn(s2, in_row ? p2 : 0.0f);
        }
        s1 = butterfly_sum(s1, 32);
        s2 = butterfly_sum(s2, 32);
        if (lane == 0) {
            red1[buf][warp] = s1;
            red2[buf][warp] = s2;
        }
        if constexpr (STAGED) {
            if (__syncthreads_or(!ok)) {
                if (tid == 0) {
                    // filled and not taken: this row's slot and those after it;
                    // without HOLD, short of the row before's (not refilled yet)
                    const int64_t left = (a.n_rows - row + stride - 1) / stride;
                    const int64_t filled = HOLD || row == blockIdx.x ? a.stages : a.stages - 1;
                    give_up(a, ring.bars, s, parity, left < filled ? left : filled);
                }
                return;
            }
            if constexpr (HOLD) {
                // every thread has taken this row into registers
                if (tid == 0 && row + a.stages * stride < a.n_rows) {
                    fence_proxy_async_smem();
                    ring.issue(s, row + a.stages * stride);
                }
            } else {
                // Past this barrier every thread is done with the row before
                // this one, so its slot takes the next row: no second barrier
                // a row, at the price of one slot's depth.
                if (tid == 0 && row != blockIdx.x && row + (a.stages - 1) * stride < a.n_rows) {
                    fence_proxy_async_smem();
                    ring.issue(s == 0 ? a.stages - 1 : s - 1, row + (a.stages - 1) * stride);
                }
            }
        } else {
            __syncthreads();
        }
        s1 = butterfly_sum((lane & 15) < W ? red1[buf][lane & 15] : 0.0f, 16);
        s2 = butterfly_sum((lane & 15) < W ? red2[buf][lane & 15] : 0.0f, 16);
        const float inv = inv_rms(s1, a.hidden, a.inv_hidden, a.eps);
        const float c = bwd_coefficient(a, s2, inv);
#pragma unroll
        for (int j = 0; j < K; ++j) {
            const int b = tid + j * T;
            const int i = HOLD ? j : 0;
            if (j < K - 1 || b < nblocks) {
                if constexpr (!HOLD) {
                    load(b, i);
                    dv[i] = V{};
                    if (a.dresidual_out)
                        ld_block(ds, b, dv[i]);
                }
                bwd_finish<E>(a, offset, h[i], g[i], wv[i], dv[i], inv, c, row, b, dw[j]);
            }
        }
        buf ^= 1;
        if constexpr (STAGED) {
            if (++s == a.stages) {
                s = 0;
                parity ^= 1u;
            }
        }
    }
    if (!a.partials)
        return;
    float* part = a.partials + static_cast<int64_t>(blockIdx.x) * a.hidden;
#pragma unroll
    for (int j = 0; j < K; ++j) {
        const int b = tid + j * T;
        if (j < K - 1 || b < nblocks) {
            float4* p = reinterpret_cast<float4*>(part) + 2 * b;
            p[0] = make_float4(dw[j][0], dw[j][1], dw[j][2], dw[j][3]);
            p[1] = make_float4(dw[j][4], dw[j][5], dw[j][6], dw[j][7]);
        }
    }
}

// ------------------------------------------------------------------- launch
template <auto FN>
cudaError_t launch_sized(const DropNormArgs& a, const DropNormPlan& p, cudaStream_t stream)
{
    if (p.smem > 40 * 1024) {  // with the kernels' own shared memory, past the 48 KB of a plain launch
        const cudaError_t e = allow_all_shared<FN>();
        if (e != cudaSuccess)
            return e;
    }
    return launch(FN, p.grid, p.threads, p.smem, false, stream, a);
}

template <int E, int T, int K>
cudaError_t launch_fwd_wide(const DropNormArgs& a, const DropNormPlan& p, cudaStream_t stream)
{
    return p.staged ? launch_sized<drop_norm_fwd_wide<E, T, K, true>>(a, p, stream)
                    : launch_sized<drop_norm_fwd_wide<E, T, K, false>>(a, p, stream);
}

template <int E, int K, int MAXT, int MINB>
cudaError_t launch_bwd_wide(const DropNormArgs& a, const DropNormPlan& p, cudaStream_t stream)
{
    return p.staged ? launch_sized<drop_norm_bwd_wide<E, K, MAXT, MINB, true>>(a, p, stream)
                    : launch_sized<drop_norm_bwd_wide<E, K, MAXT, MINB, false>>(a, p, stream);
}

template <int E, int L>
cudaError_t launch_narrow(const DropNormArgs& a, const DropNormPlan& p, bool backward, cudaStream_t stream)
{
    return backward ? launch_sized<drop_norm_bwd_narrow<E, L, 1>>(a, p, stream)
                    : launch_sized<drop_norm_fwd_narrow<E, L>>(a, p, stream);
}

template <int E>
cudaError_t launch_drop_norm_of(const DropNormArgs& a, const DropNormPlan& p, bool backward, cudaStream_t stream)
{
    if (p.warp) {
        if constexpr (E != kElemF32) {
            if (p.K > 1)
                return p.K == 2 ? launch_sized<drop_norm_bwd_narrow<E, 32, 2>>(a, p, stream)
                                : launch_sized<drop_norm_bwd_narrow<E, 32, 4>>(a, p, stream);
        }
        return p.lanes == 8    ? launch_narrow<E, 8>(a, p, backward, stream)
               : p.lanes == 16 ? launch_narrow<E, 16>(a, p, backward, stream)
                               : launch_narrow<E, 32>(a, p, backward, stream);
    }
    if (backward) {
        switch (p.K) {
        case 1:
            return launch_bwd_wide<E, 1, 256, 4>(a, p, stream);
        case 2:
            if (p.threads <= 256)
                return launch_bwd_wide<E, 2, 256, 2>(a, p, stream);
            if constexpr (bwd_pair_threads(E) > 256) {
                if (p.threads <= bwd_pair_threads(E))
                    return launch_bwd_wide<E, 2, bwd_pair_threads(E), 2>(a, p, stream);
            }
            return launch_bwd_wide<E, 2, 512, 1>(a, p, stream);
        case 4:
            return launch_bwd_wide<E, 4, 512, 1>(a, p, stream);
        default:
            return launch_bwd_wide<E, 8, 512, 1>(a, p, stream);
        }
    }
    constexpr bool wide_type = E == kElemF32;
    switch (p.threads * 8 * p.K) {
    case 512:
        return launch_fwd_wide<E, wide_type ? 64 : 32, wide_type ? 1 : 2>(a, p, stream);
    case 1024:
        return launch_fwd_wide<E, wide_type ? 128 : 32, wide_type ? 1 : 4>(a, p, stream);
    case 2048:
        return launch_fwd_wide<E, 128, 2>(a, p, stream);
    case 4096:
        return launch_fwd_wide<E, 128, 4>(a, p, stream);
    case 8192:
        return launch_fwd_wide<E, 256, 4>(a, p, stream);
    case 16384:
        return launch_fwd_wide<E, 512, 4>(a, p, stream);
    default:
        return launch_fwd_wide<E, 512, 8>(a, p, stream);
    }
}

}  // namespace dradd
