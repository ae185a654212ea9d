// dradd_rope.cuh -- rotary positions of q and k in one launch, plain or
// behind a per-head RMSNorm, and the gradients of the latter.
//
// Pair i < rot / 2 of a head, columns (i, i + rot / 2) (halves layout) or
// (2 i, 2 i + 1) (interleaved), turns by theta = position * inv_freq[i]:
//   (a, b) -> (a C - b S, a S + b C), C = scale cos theta, S = scale sin theta,
// the inverse (and gradient) by -theta.  Columns rot .. dim - 1 pass.
//
// Angles: inv_freq / 2 pi, less its whole turns, is held as a 64-bit
// fraction of a turn; position times it modulo 2^64 is then the angle modulo
// one turn, exact up to the fraction's own rounding (below position * 2^-53
// turns for frequencies up to one radian), for positions of either sign.
// Its top 32 bits go to sincospif.  fp32 angles would lose far positions:
// at 2^20 they are off by 2^-5 radians.  Three integer multiplies and no
// fp64 outside the one conversion a CTA makes.
//
// Work layout.  A unit is 16 columns of a head: in the halves layout 8
// columns and their partners, or 16 that pass; interleaved 16 consecutive
// ones.  A head's units go to `group` neighbouring lanes (a power of two, so
// the norm's sums are butterflies within the group); the CTA's groups walk
// the heads of q and of k of `tokens_per_step` tokens, whose cosines and
// sines the CTA computes once into shared memory.  Bound by the memory (2
// elements of traffic an element, the gradient 3).
#pragma once

#include "dradd_elem.cuh"
#include "dradd_internal.h"
#include "dradd_train_internal.h"

namespace dradd {

// Turns per position as a 64-bit fraction.
__device__ __forceinline__ uint64_t turn_fraction(double inv_freq)
{
    const double turns = inv_freq * 0.15915494309189533577;  // 1 / (2 pi)
    return __double2ull_rd((turns - floor(turns)) * 18446744073709551616.0);
}

// (cos, sin) of position * fraction turns.
__device__ __forceinline__ void turn_cos_sin(uint64_t fraction, int64_t position, float& c, float& s)
{
    const uint64_t turns = fraction * static_cast<uint64_t>(position);
    const int32_t top = static_cast<int32_t>(static_cast<uint32_t>(turns >> 32));
    sincospif(static_cast<float>(top) * 0x1p-31f, &s, &c);
}

// The two 8-column runs of unit u: first columns, and how many of each lie
// in the head.
struct UnitColumns {
    int a, b, na, nb;
    int pairs;  // how many of its 8 pairs turn
};

template <bool INTER>
__device__ __forceinline__ UnitColumns unit_columns(const RopeArgs& p, int u)
{
    UnitColumns c;
    auto clip = [](int n) { return n < 0 ? 0 : n > 8 ? 8 : n; };
    if (INTER) {
        c.a = 16 * u;
        c.b = c.a + 8;
        c.pairs = clip((p.rot >> 1) - 8 * u);
        c.na = clip(p.dim - c.a);
        c.nb = clip(p.dim - c.b);
    } else if (u < p.rot_units) {
        const int half = p.rot >> 1;
        c.a = 8 * u;
        c.b = half + 8 * u;
        c.na = c.nb = c.pairs = clip(half - 8 * u);
    } else {
        c.a = p.rot + 16 * (u - p.rot_units);
        c.b = c.a + 8;
        c.pairs = 0;
        c.na = clip(p.dim - c.a);
        c.nb = clip(p.dim - c.b);
    }
    if (u >= p.units)
        c.na = c.nb = c.pairs = 0;
    return c;
}

// BLOCKS: every run is a whole, 16-byte aligned block of 8.
template <int E, bool BLOCKS>
__device__ __forceinline__ void load_unit(const void* base, int64_t at, const UnitColumns& c, float (&a)[8],
                                          float (&b)[8])
{
    using T = typename Elem<E>::T;
    const T* p = static_cast<const T*>(base) + at;
    if constexpr (BLOCKS) {
        typename Elem<E>::Block va, vb;
        if (c.na) {
            ld_block_stream(p + c.a, 0, va);
            Elem<E>::unpack(va, a);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                a[e] = 0.0f;
        }
        if (c.nb) {
            ld_block_stream(p + c.b, 0, vb);
            Elem<E>::unpack(vb, b);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                b[e] = 0.0f;
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            a[e] = e < c.na ? Elem<E>::widen(__ldcs(p + c.a + e)) : 0.0f;
            b[e] = e < c.nb ? Elem<E>::widen(__ldcs(p + c.b + e)) : 0.0f;
        }
    }
}

template <int E, bool BLOCKS>
__device__ __forceinline__ void store_unit(void* base, int64_t at, const UnitColumns& c, const float (&a)[8],
                                           const float (&b)[8])
{
    using T = typename Elem<E>::T;
    T* p = static_cast<T*>(base) + at;
    if constexpr (BLOCKS) {
        if (c.na)
            st_block_stream(p + c.a, 0, Elem<E>::pack(a));
        if (c.nb)
            st_block_stream(p + c.b, 0, Elem<E>::pack(b));
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if (e < c.na)
                __stcs(p + c.a + e, Elem<E>::narrow(a[e]));
            if (e < c.nb)
                __stcs(p + c.b + e, Elem<E>::narrow(b[e]));
        }
    }
}

// 16 floats of shared memory as two runs of 8.
__device__ __forceinline__ void load_shared16(const float* p, float (&a)[8], float (&b)[8])
{
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float4 va = *reinterpret_cast<const float4*>(p + 4 * i);
        const float4 vb = *reinterpret_cast<const float4*>(p + 8 + 4 * i);
        a[4 * i] = va.x; a[4 * i + 1] = va.y; a[4 * i + 2] = va.z; a[4 * i + 3] = va.w;
        b[4 * i] = vb.x; b[4 * i + 1] = vb.y; b[4 * i + 2] = vb.z; b[4 * i + 3] = vb.w;
    }
}

// Turns the unit's first `pairs` pairs by their cosines and sines (cs: 8
// cosines, then 8 sines); the others stay, whatever they hold.  In the
// halves layout a unit's pairs all turn or lie outside the head.
template <bool INTER>
__device__ __forceinline__ void turn_unit(const float* cs, int pairs, float (&a)[8], float (&b)[8])
{
    float c[8], s[8];
    load_shared16(cs, c, s);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        float& x = INTER ? (e < 4 ? a[(2 * e) & 7] : b[(2 * e) & 7]) : a[e];
        float& y = INTER ? (e < 4 ? a[(2 * e + 1) & 7] : b[(2 * e + 1) & 7]) : b[e];
        const float x1 = __fmaf_rn(x, c[e], -__fmul_rn(y, s[e]));
        const float y1 = __fmaf_rn(x, s[e], __fmul_rn(y, c[e]));
        if (!INTER || e < pairs) {
            x = x1;
            y = y1;
        }
    }
}

// The weights of q and of k in fp32, table[side][unit][16] in the order of
// the unit's columns (0 past the head).
template <int E, bool INTER>
__device__ __forceinline__ void fill_weights(const RopeArgs& p, float* table)
{
    using T = typename Elem<E>::T;
    for (int i = threadIdx.x; i < 2 * p.units * 16; i += kRopeThreads) {
        const int side = i >= p.units * 16;
        const int r = i - side * p.units * 16;
        const UnitColumns c = unit_columns<INTER>(p, r >> 4);
        const int e = r & 7;
        const bool second = (r & 8) != 0;
        const T* w = static_cast<const T*>(side ? p.k.weight : p.q.weight);
        float v = 0.0f;
        if (w && e < (second ? c.nb : c.na))
            v = Elem<E>::widen(__ldg(w + (second ? c.b : c.a) + e));
        table[i] = v;
    }
}

// The CTA's angles: table[token][unit][8 cosines, 8 sines], for the units
// that rotate (cosine 1 and sine 0 past rot / 2, never used).
__device__ __forceinline__ void fill_angles(const RopeArgs& p, float* table, int64_t first, int n_tokens)
{
    const int pairs = 8 * p.rot_units;
    for (int i = threadIdx.x; i < n_tokens * pairs; i += kRopeThreads) {
        const int j = i / pairs, pair = i - j * pairs;
        const int64_t token = first + j;
        float c = 1.0f, s = 0.0f;
        if (pair < (p.rot >> 1)) {
            const int64_t pos = p.positions ? __ldg(p.positions + token) : p.position0 + token % p.seq;
            turn_cos_sin(turn_fraction(__ldg(p.inv_freq + pair)), pos, c, s);
            c = __fmul_rn(c, p.scale);
            s = __fmul_rn(s, __fmul_rn(p.scale, p.sign));
        }
        float* at = table + (j * p.rot_units + (pair >> 3)) * 16 + (pair & 7);
        at[0] = c;
        at[8] = s;
    }
}

__device__ __forceinline__ float fold8(const float (&p)[8])
{
    return __fadd_rn(__fadd_rn(__fadd_rn(p[0], p[1]), __fadd_rn(p[2], p[3])),
                     __fadd_rn(__fadd_rn(p[4], p[5]), __fadd_rn(p[6], p[7])));
}

// Forward: plain (NORM false; also the inverse) or behind the norm
//   z = (x * inv) * w, inv = 1 / sqrt(sum x^2 / dim + eps).
template <int E, bool NORM, bool INTER, bool BLOCKS>
__global__ void __launch_bounds__(kRopeThreads) rope_fwd_kernel(const RopeArgs p)
{
    extern __shared__ __align__(16) float table[];
    wait_prior_grids();
    allow_next_grid();
    const int64_t first = static_cast<int64_t>(blockIdx.x) * p.tokens_per_step;
    const int n_tokens = static_cast<int>(p.tokens - first < p.tokens_per_step ? p.tokens - first : p.tokens_per_step);
    fill_angles(p, table, first, n_tokens);
    float* const weights = table + p.tokens_per_step * p.rot_units * 16;
    if constexpr (NORM)
        fill_weights<E, INTER>(p, weights);
    __syncthreads();
    const int u = threadIdx.x & (p.group - 1);
    const int groups = kRopeThreads / p.group;
    const int own = u < p.units ? u : 0;  // lanes past the units carry zeros
    const UnitColumns cols = unit_columns<INTER>(p, u);
    const int heads = p.q.heads + p.k.heads;
    const int items = n_tokens * heads;
    // lanes of one warp start together and leave together (the norm's sums
    // are shuffles of the whole warp)
    const int mine = threadIdx.x / p.group;
    const int lead = mine - (threadIdx.x & 31) / p.group;
    for (int base = 0; lead + base < items; base += groups) {
        const int item = mine + base;
        const bool active = item < items;
        const int j = active ? item / heads : 0;
        const int head = active ? item - j * heads : 0;
        const bool is_k = head >= p.q.heads;
        const RopeSide& side = is_k ? p.k : p.q;
        const int hd = is_k ? head - p.q.heads : head;
        const int64_t token = first + j;
        const int64_t bi = token / p.seq, si = token - bi * p.seq;
        UnitColumns c = cols;
        if (!active || (side.skip_rest && c.pairs == 0))
            c.na = c.nb = 0;
        float a[8], b[8];
        load_unit<E, BLOCKS>(side.in, bi * side.in_b + si * side.in_s + hd * side.in_h, c, a, b);
        if constexpr (NORM) {
            float sq = __fadd_rn(fold8_squares(a), fold8_squares(b));
            sq = butterfly_sum(sq, p.group);
            const float inv = inv_rms(sq, p.dim, p.inv_dim, side.eps);
            float wa[8], wb[8];
            load_shared16(weights + ((is_k ? p.units : 0) + own) * 16, wa, wb);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                a[e] = __fmul_rn(__fmul_rn(a[e], inv), wa[e]);
                b[e] = __fmul_rn(__fmul_rn(b[e], inv), wb[e]);
            }
        }
        if (c.pairs)
            turn_unit<INTER>(table + (j * p.rot_units + u) * 16, c.pairs, a, b);
        store_unit<E, BLOCKS>(side.out, bi * side.out_b + si * side.out_s + hd * side.out_h, c, a, b);
    }
}

// The gradients of the fused call, with g = turn(-theta) dy:
//   S1 = sum x^2, S2 = sum (g w) x; c = inv (inv (S2 / dim))
//   dx = inv (g w - x c); dweight += g (x inv), over tokens and heads.
// A CTA walks its token steps in order, q heads then k heads of each, every
// group adding its own heads' shares in registers; at the end the groups'
// sums are added in group order into the CTA's part.
template <int E, bool INTER, bool BLOCKS>
__device__ __forceinline__ void rope_bwd_side(const RopeArgs& p, const RopeSide& side, const float* table, const float* weights,
                                              int64_t first, int n_tokens, const UnitColumns& cols, int u,
                                              float (&da)[8], float (&db)[8])
{
    const int groups = kRopeThreads / p.group;
    const int items = n_tokens * side.heads;
    const int mine = threadIdx.x / p.group;
    const int lead = mine - (threadIdx.x & 31) / p.group;
    for (int base = 0; lead + base < items; base += groups) {
        const int item = mine + base;
        const bool active = item < items;
        const int j = active ? item / side.heads : 0;
        const int hd = active ? item - j * side.heads : 0;
        const int64_t token = first + j;
        const int64_t bi = token / p.seq, si = token - bi * p.seq;
        UnitColumns c = cols;
        if (!active)
            c.na = c.nb = 0;
        float a[8], b[8], ga[8], gb[8], wa[8], wb[8];
        load_unit<E, BLOCKS>(side.in, bi * side.in_b + si * side.in_s + hd * side.in_h, c, a, b);
        load_unit<E, BLOCKS>(side.grad, bi * side.grad_b + si * side.grad_s + hd * side.grad_h, c, ga, gb);
        if (c.pairs)
            turn_unit<INTER>(table + (j * p.rot_units + u) * 16, c.pairs, ga, gb);
        load_shared16(weights + (u < p.units ? u : 0) * 16, wa, wb);
        float ta[8], tb[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            wa[e] = __fmul_rn(ga[e], wa[e]);
            wb[e] = __fmul_rn(gb[e], wb[e]);
            ta[e] = __fmul_rn(wa[e], a[e]);
            tb[e] = __fmul_rn(wb[e], b[e]);
        }
        const float s1 = butterfly_sum(__fadd_rn(fold8_squares(a), fold8_squares(b)), p.group);
        const float s2 = butterfly_sum(__fadd_rn(fold8(ta), fold8(tb)), p.group);
        const float inv = inv_rms(s1, p.dim, p.inv_dim, side.eps);
        const float mean = p.inv_dim != 0.0f ? __fmul_rn(s2, p.inv_dim) : __fdiv_rn(s2, static_cast<float>(p.dim));
        const float k = __fmul_rn(inv, __fmul_rn(inv, mean));
        if (active) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                da[e] = __fmaf_rn(ga[e], __fmul_rn(a[e], inv), da[e]);
                db[e] = __fmaf_rn(gb[e], __fmul_rn(b[e], inv), db[e]);
                ta[e] = __fmul_rn(inv, __fmaf_rn(-a[e], k, wa[e]));
                tb[e] = __fmul_rn(inv, __fmaf_rn(-b[e], k, wb[e]));
            }
        }
        store_unit<E, BLOCKS>(side.out, bi * side.out_b + si * side.out_s + hd * side.out_h, c, ta, tb);
    }
}

template <int E, bool INTER, bool BLOCKS>
__global__ void __launch_bounds__(kRopeThreads) rope_bwd_kernel(const RopeArgs p)
{
    extern __shared__ __align__(16) float table[];
    wait_prior_grids();
    allow_next_grid();
    const int u = threadIdx.x & (p.group - 1);
    const int group = threadIdx.x / p.group;
    const int groups = kRopeThreads / p.group;
    const UnitColumns cols = unit_columns<INTER>(p, u);
    float dq[2][8] = {}, dk[2][8] = {};
    float* const weights = table + p.tokens_per_step * p.rot_units * 16;
    fill_weights<E, INTER>(p, weights);
    const int64_t step = static_cast<int64_t>(gridDim.x) * p.tokens_per_step;
    for (int64_t first = static_cast<int64_t>(blockIdx.x) * p.tokens_per_step; first < p.tokens; first += step) {
        const int n = static_cast<int>(p.tokens - first < p.tokens_per_step ? p.tokens - first : p.tokens_per_step);
        fill_angles(p, table, first, n);
        __syncthreads();
        rope_bwd_side<E, INTER, BLOCKS>(p, p.q, table, weights, first, n, cols, u, dq[0], dq[1]);
        rope_bwd_side<E, INTER, BLOCKS>(p, p.k, table, weights + p.units * 16, first, n, cols, u, dk[0], dk[1]);
        __syncthreads();
    }
    if (!p.partials)
        return;
    // The table's memory now takes the head's column sums: q, then k.
    float* part = p.partials + static_cast<int64_t>(blockIdx.x) * 2 * p.dim;
    for (int side = 0; side < 2; ++side) {
        for (int g = 0; g < groups; ++g) {
            if (group == g) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float va = side ? dk[0][e] : dq[0][e], vb = side ? dk[1][e] : dq[1][e];
                    if (e < cols.na)
                        table[cols.a + e] = g == 0 ? va : __fadd_rn(table[cols.a + e], va);
                    if (e < cols.nb)
                        table[cols.b + e] = g == 0 ? vb : __fadd_rn(table[cols.b + e], vb);
                }
            }
            __syncthreads();
        }
        for (int i = threadIdx.x; i < p.dim; i += kRopeThreads)
            part[side * p.dim + i] = table[i];
        __syncthreads();
    }
}

template <int E, bool INTER, bool BLOCKS>
cudaError_t launch_rope_as(const RopeArgs& p, int mode, int grid, cudaStream_t stream)
{
    const size_t angles = static_cast<size_t>(p.tokens_per_step) * p.rot_units * 16 * sizeof(float);
    const size_t both = angles + static_cast<size_t>(p.units) * 32 * sizeof(float);  // >= dim floats
    if (mode == kRopeNormBwd)
        return launch(rope_bwd_kernel<E, INTER, BLOCKS>, grid, kRopeThreads, both, false, stream, p);
    return mode == kRopeNorm
               ? launch(rope_fwd_kernel<E, true, INTER, BLOCKS>, grid, kRopeThreads, both, false, stream, p)
               : launch(rope_fwd_kernel<E, false, INTER, BLOCKS>, grid, kRopeThreads, angles, false, stream, p);
}

template <int E>
cudaError_t launch_rope_of(const RopeArgs& p, int mode, bool interleaved, bool blocks, int grid, cudaStream_t stream)
{
    if (interleaved)
        return blocks ? launch_rope_as<E, true, true>(p, mode, grid, stream)
                      : launch_rope_as<E, true, false>(p, mode, grid, stream);
    return blocks ? launch_rope_as<E, false, true>(p, mode, grid, stream)
                  : launch_rope_as<E, false, false>(p, mode, grid, stream);
}

}  // namespace dradd
