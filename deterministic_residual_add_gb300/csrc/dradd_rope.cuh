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
// the norm's sums are butterflies within the group), so a warp takes
// 32 / group heads at a time; one such step is all of q or all of k.  A warp
// takes a token, computes its cosines and sines once, two or so a lane, into
// shared memory of its own, and goes through `per_warp` steps of heads with
// the loads of the next ones in flight; no barrier but the CTA's first.
// Bound by the memory (2 elements of traffic an element, the gradient 3).
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

// BLOCKS, below: every run is a whole, 16-byte aligned block of 8.

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
    for (int e = 0; e < 8; e += 2) {
        // pairs e and e + 1
        float& x0 = INTER ? (e < 4 ? a[(2 * e) & 7] : b[(2 * e) & 7]) : a[e];
        float& y0 = INTER ? (e < 4 ? a[(2 * e + 1) & 7] : b[(2 * e + 1) & 7]) : b[e];
        float& x1 = INTER ? (e < 4 ? a[(2 * e + 2) & 7] : b[(2 * e + 2) & 7]) : a[e + 1];
        float& y1 = INTER ? (e < 4 ? a[(2 * e + 3) & 7] : b[(2 * e + 3) & 7]) : b[e + 1];
        float p0, p1, q0, q1;
        mul2_rn(y0, y1, s[e], s[e + 1], p0, p1);
        mul2_rn(y0, y1, c[e], c[e + 1], q0, q1);
        fma2_rn(x0, x1, s[e], s[e + 1], q0, q1, q0, q1);
        p0 = __fmaf_rn(x0, c[e], -p0);
        p1 = __fmaf_rn(x1, c[e + 1], -p1);
        if (!INTER || e < pairs) {
            x0 = p0;
            y0 = q0;
        }
        if (!INTER || e + 1 < pairs) {
            x1 = p1;
            y1 = q1;
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

// A unit as it comes from memory.
template <int E, bool BLOCKS>
struct RawUnit {
    typename Elem<E>::Block a, b;
};
template <int E>
struct RawUnit<E, false> {
    typename Elem<E>::T a[8], b[8];
};

template <int E, bool BLOCKS>
__device__ __forceinline__ void load_raw(const void* base, int64_t at, const UnitColumns& c, bool active,
                                         RawUnit<E, BLOCKS>& r)
{
    using T = typename Elem<E>::T;
    const T* p = static_cast<const T*>(base) + at;
    if constexpr (BLOCKS) {
        r.a = r.b = typename Elem<E>::Block{};
        if (active && c.na)
            ld_block_stream(p + c.a, 0, r.a);
        if (active && c.nb)
            ld_block_stream(p + c.b, 0, r.b);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            r.a[e] = active && e < c.na ? __ldcs(p + c.a + e) : T{};
            r.b[e] = active && e < c.nb ? __ldcs(p + c.b + e) : T{};
        }
    }
}

template <int E, bool BLOCKS>
__device__ __forceinline__ void widen_unit(const RawUnit<E, BLOCKS>& r, float (&a)[8], float (&b)[8])
{
    if constexpr (BLOCKS) {
        Elem<E>::unpack(r.a, a);
        Elem<E>::unpack(r.b, b);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            a[e] = Elem<E>::widen(r.a[e]);
            b[e] = Elem<E>::widen(r.b[e]);
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

__device__ __forceinline__ float fold8(const float (&p)[8])
{
    return __fadd_rn(__fadd_rn(__fadd_rn(p[0], p[1]), __fadd_rn(p[2], p[3])),
                     __fadd_rn(__fadd_rn(p[4], p[5]), __fadd_rn(p[6], p[7])));
}

// The CTA's shared memory: the pairs' fractions, the weights (norm only),
// then every warp's cosines and sines, table[unit][8 cosines, 8 sines].
struct RopeShared {
    uint64_t* fractions;
    float* weights;
    float* table;  // this warp's
};

template <int E, bool NORM, bool INTER>
__device__ __forceinline__ RopeShared rope_prologue(const RopeArgs& p, unsigned char* mem)
{
    RopeShared sh;
    sh.fractions = reinterpret_cast<uint64_t*>(mem);
    sh.weights = reinterpret_cast<float*>(sh.fractions + 8 * p.rot_units);
    sh.table = sh.weights + (NORM ? 32 * p.units : 0) + (threadIdx.x >> 5) * 16 * p.rot_units;
    for (int i = threadIdx.x; i < (p.rot >> 1); i += kRopeThreads)
        sh.fractions[i] = turn_fraction(__ldg(p.inv_freq + i));
    if constexpr (NORM)
        fill_weights<E, INTER>(p, sh.weights);
    __syncthreads();
    return sh;
}

// The warp's table for one position.  What lies past rot / 2 is never used.
__device__ __forceinline__ void fill_angles(const RopeArgs& p, const RopeShared& sh, int64_t position, int lane)
{
    __syncwarp();
    for (int i = lane; i < (p.rot >> 1); i += 32) {
        float c, s;
        turn_cos_sin(sh.fractions[i], position, c, s);
        float* at = sh.table + (i >> 3) * 16 + (i & 7);
        at[0] = __fmul_rn(c, p.scale);
        at[8] = __fmul_rn(s, __fmul_rn(p.scale, p.sign));
    }
    __syncwarp();
}

// One step of a warp's work: the heads of q or of k its groups take, and
// where this lane's head begins.
struct RopeStep {
    bool is_k, active;
    int head;
};

__device__ __forceinline__ RopeStep rope_step(const RopeArgs& p, int step, int group_in_warp)
{
    RopeStep r;
    r.is_k = step >= p.q_steps;
    r.head = (step - (r.is_k ? p.q_steps : 0)) * p.heads_per_step + group_in_warp;
    r.active = r.head < (r.is_k ? p.k.heads : p.q.heads);
    if (!r.active)
        r.head = 0;
    return r;
}

// The token and the steps of work item w of the call.
struct RopeWork {
    int64_t bi, si, position;
    int first, last;
};

__device__ __forceinline__ RopeWork rope_work(const RopeArgs& p, uint32_t w)
{
    RopeWork r;
    const uint32_t token = w / static_cast<uint32_t>(p.warps_per_token);
    const int part = static_cast<int>(w - token * static_cast<uint32_t>(p.warps_per_token));
    const uint32_t b = token / static_cast<uint32_t>(p.seq);
    r.bi = b;
    r.si = token - b * static_cast<uint32_t>(p.seq);
    r.position = p.positions ? __ldg(p.positions + token) : p.position0 + r.si;
    r.first = part * p.steps_per_warp;
    const int steps = p.q_steps + p.k_steps;
    r.last = r.first + p.steps_per_warp < steps ? r.first + p.steps_per_warp : steps;
    return r;
}

// Forward: plain (NORM false; also the inverse) or behind the norm
//   z = (x * inv) * w, inv = 1 / sqrt(sum x^2 / dim + eps).
template <int E, bool NORM, bool INTER, bool BLOCKS>
__global__ void __launch_bounds__(kRopeThreads, E == kElemF32 || !BLOCKS ? 2 : 3) rope_fwd_kernel(const RopeArgs p)
{
    extern __shared__ __align__(16) unsigned char mem[];
    wait_prior_grids();
    allow_next_grid();
    const RopeShared sh = rope_prologue<E, NORM, INTER>(p, mem);
    const int lane = threadIdx.x & 31;
    const int u = lane & (p.group - 1);
    const int g = lane / p.group;
    const UnitColumns cols = unit_columns<INTER>(p, u);
    const float* const turn = sh.table + (cols.pairs ? u : 0) * 16;
    const float* const weight = sh.weights + (u < p.units ? u : 0) * 16;
    const uint32_t warps = gridDim.x * (kRopeThreads / 32);
    for (uint32_t w = blockIdx.x * (kRopeThreads / 32) + (threadIdx.x >> 5); w < p.n_work; w += warps) {
        const RopeWork work = rope_work(p, w);
        auto load = [&](int step, RawUnit<E, BLOCKS>& raw) {
            const RopeStep st = rope_step(p, step, g);
            const RopeSide& side = st.is_k ? p.k : p.q;
            load_raw<E, BLOCKS>(side.in, work.bi * side.in_b + work.si * side.in_s + st.head * side.in_h, cols,
                                st.active && step < work.last, raw);
        };
        RawUnit<E, BLOCKS> next0, next1;
        load(work.first, next0);
        load(work.first + 1, next1);
        fill_angles(p, sh, work.position, lane);
        for (int step = work.first; step < work.last; ++step) {
            float a[8], b[8];
            widen_unit<E, BLOCKS>(next0, a, b);
            next0 = next1;
            load(step + 2, next1);
            const RopeStep st = rope_step(p, step, g);
            const RopeSide& side = st.is_k ? p.k : p.q;
            if constexpr (NORM) {
                float sq = __fadd_rn(fold8_squares(a), fold8_squares(b));
                sq = butterfly_sum(sq, p.group);
                const float inv = inv_rms(sq, p.dim, p.inv_dim, side.eps);
                float wa[8], wb[8];
                load_shared16(weight + (st.is_k ? p.units * 16 : 0), wa, wb);
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    mul2_rn(a[e], a[e + 1], inv, inv, a[e], a[e + 1]);
                    mul2_rn(b[e], b[e + 1], inv, inv, b[e], b[e + 1]);
                    mul2_rn(a[e], a[e + 1], wa[e], wa[e + 1], a[e], a[e + 1]);
                    mul2_rn(b[e], b[e + 1], wb[e], wb[e + 1], b[e], b[e + 1]);
                }
            }
            if (cols.pairs)
                turn_unit<INTER>(turn, cols.pairs, a, b);
            UnitColumns c = cols;
            if (!st.active || (side.skip_rest && cols.pairs == 0))
                c.na = c.nb = 0;
            store_unit<E, BLOCKS>(side.out, work.bi * side.out_b + work.si * side.out_s + st.head * side.out_h, c, a,
                                  b);
        }
    }
}

// The gradients of the fused call, with g = turn(-theta) dy:
//   S1 = sum x^2, S2 = sum (g w) x; c = inv (inv (S2 / dim))
//   dx = inv (g w - x c); dweight += g (x inv), over tokens and heads.
// Every lane adds the shares of its warp's work in order in registers; at
// the end a warp's groups are added by butterfly and the CTA's warps in
// order into the CTA's part.
template <int E, bool INTER, bool BLOCKS>
__global__ void __launch_bounds__(kRopeThreads, 2) rope_bwd_kernel(const RopeArgs p)
{
    extern __shared__ __align__(16) unsigned char mem[];
    wait_prior_grids();
    allow_next_grid();
    const RopeShared sh = rope_prologue<E, true, INTER>(p, mem);
    const int lane = threadIdx.x & 31;
    const int u = lane & (p.group - 1);
    const int g = lane / p.group;
    const UnitColumns cols = unit_columns<INTER>(p, u);
    const float* const turn = sh.table + (cols.pairs ? u : 0) * 16;
    const float* const weight = sh.weights + (u < p.units ? u : 0) * 16;
    float dq[2][8] = {}, dk[2][8] = {};
    const uint32_t warps = gridDim.x * (kRopeThreads / 32);
    for (uint32_t w = blockIdx.x * (kRopeThreads / 32) + (threadIdx.x >> 5); w < p.n_work; w += warps) {
        const RopeWork work = rope_work(p, w);
        auto load = [&](int step, RawUnit<E, BLOCKS>& x, RawUnit<E, BLOCKS>& dy) {
            const RopeStep st = rope_step(p, step, g);
            const RopeSide& side = st.is_k ? p.k : p.q;
            const bool active = st.active && step < work.last;
            load_raw<E, BLOCKS>(side.in, work.bi * side.in_b + work.si * side.in_s + st.head * side.in_h, cols, active,
                                x);
            load_raw<E, BLOCKS>(side.grad, work.bi * side.grad_b + work.si * side.grad_s + st.head * side.grad_h, cols,
                                active, dy);
        };
        RawUnit<E, BLOCKS> next_x, next_dy;
        load(work.first, next_x, next_dy);
        fill_angles(p, sh, work.position, lane);
        for (int step = work.first; step < work.last; ++step) {
            const RopeStep st = rope_step(p, step, g);
            const RopeSide& side = st.is_k ? p.k : p.q;
            float a[8], b[8], ga[8], gb[8], wa[8], wb[8], ta[8], tb[8];
            widen_unit<E, BLOCKS>(next_x, a, b);
            widen_unit<E, BLOCKS>(next_dy, ga, gb);
            load(step + 1, next_x, next_dy);
            if (cols.pairs)
                turn_unit<INTER>(turn, cols.pairs, ga, gb);
            load_shared16(weight + (st.is_k ? p.units * 16 : 0), wa, wb);
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
                mul2_rn(ga[e], ga[e + 1], wa[e], wa[e + 1], wa[e], wa[e + 1]);
                mul2_rn(gb[e], gb[e + 1], wb[e], wb[e + 1], wb[e], wb[e + 1]);
                mul2_rn(wa[e], wa[e + 1], a[e], a[e + 1], ta[e], ta[e + 1]);
                mul2_rn(wb[e], wb[e + 1], b[e], b[e + 1], tb[e], tb[e + 1]);
            }
            const float s1 = butterfly_sum(__fadd_rn(fold8_squares(a), fold8_squares(b)), p.group);
            const float s2 = butterfly_sum(__fadd_rn(fold8(ta), fold8(tb)), p.group);
            const float inv = inv_rms(s1, p.dim, p.inv_dim, side.eps);
            const float mean =
                p.inv_dim != 0.0f ? __fmul_rn(s2, p.inv_dim) : __fdiv_rn(s2, static_cast<float>(p.dim));
            const float k = -__fmul_rn(inv, __fmul_rn(inv, mean));
            if (st.active) {
                float xa[8], xb[8];
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    mul2_rn(a[e], a[e + 1], inv, inv, xa[e], xa[e + 1]);
                    mul2_rn(b[e], b[e + 1], inv, inv, xb[e], xb[e + 1]);
                    fma2_rn(a[e], a[e + 1], k, k, wa[e], wa[e + 1], ta[e], ta[e + 1]);
                    fma2_rn(b[e], b[e + 1], k, k, wb[e], wb[e + 1], tb[e], tb[e + 1]);
                    mul2_rn(ta[e], ta[e + 1], inv, inv, ta[e], ta[e + 1]);
                    mul2_rn(tb[e], tb[e + 1], inv, inv, tb[e], tb[e + 1]);
                }
                if (st.is_k) {
#pragma unroll
                    for (int e = 0; e < 8; e += 2) {
                        fma2_rn(ga[e], ga[e + 1], xa[e], xa[e + 1], dk[0][e], dk[0][e + 1], dk[0][e], dk[0][e + 1]);
                        fma2_rn(gb[e], gb[e + 1], xb[e], xb[e + 1], dk[1][e], dk[1][e + 1], dk[1][e], dk[1][e + 1]);
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 8; e += 2) {
                        fma2_rn(ga[e], ga[e + 1], xa[e], xa[e + 1], dq[0][e], dq[0][e + 1], dq[0][e], dq[0][e + 1]);
                        fma2_rn(gb[e], gb[e + 1], xb[e], xb[e + 1], dq[1][e], dq[1][e + 1], dq[1][e], dq[1][e + 1]);
                    }
                }
                store_unit<E, BLOCKS>(side.out, work.bi * side.out_b + work.si * side.out_s + st.head * side.out_h,
                                      cols, ta, tb);
            }
        }
    }
    if (!p.partials)
        return;
    // warp sums [warp][side][unit][16] over the memory used so far
    float* const sums = reinterpret_cast<float*>(mem);
    const int stride = 32 * p.units;
    __syncthreads();
#pragma unroll
    for (int side = 0; side < 2; ++side) {
        float* at = sums + (threadIdx.x >> 5) * stride + (side * p.units + u) * 16;
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            float v = side ? dk[e >> 3][e & 7] : dq[e >> 3][e & 7];
            for (int d = p.group; d < 32; d <<= 1)
                v = __fadd_rn(v, __shfl_xor_sync(0xFFFFFFFFu, v, d));
            if (g == 0 && u < p.units)
                at[e] = v;
        }
    }
    __syncthreads();
    float* part = p.partials + static_cast<int64_t>(blockIdx.x) * 2 * p.dim;
    for (int i = threadIdx.x; i < stride; i += kRopeThreads) {
        const int side = i >= 16 * p.units;
        const int r = i - side * 16 * p.units;
        const UnitColumns c = unit_columns<INTER>(p, r >> 4);
        const int e = r & 7;
        const bool second = (r & 8) != 0;
        if (e >= (second ? c.nb : c.na))
            continue;
        float v = sums[i];
#pragma unroll
        for (int k = 1; k < kRopeThreads / 32; ++k)
            v = __fadd_rn(v, sums[k * stride + i]);
        part[side * p.dim + (second ? c.b : c.a) + e] = v;
    }
}

template <int E, bool INTER, bool BLOCKS>
cudaError_t launch_rope_as(const RopeArgs& p, int mode, int grid, cudaStream_t stream)
{
    const bool norm = mode != kRopePlain;
    size_t smem = static_cast<size_t>(p.rot_units) * 64 * (1 + kRopeThreads / 32) + (norm ? p.units * 128 : 0);
    const size_t sums = static_cast<size_t>(p.units) * 128 * (kRopeThreads / 32);
    if (mode == kRopeNormBwd)
        return launch(rope_bwd_kernel<E, INTER, BLOCKS>, grid, kRopeThreads, smem > sums ? smem : sums, false, stream,
                      p);
    return norm ? launch(rope_fwd_kernel<E, true, INTER, BLOCKS>, grid, kRopeThreads, smem, false, stream, p)
                : launch(rope_fwd_kernel<E, false, INTER, BLOCKS>, grid, kRopeThreads, smem, false, stream, p);
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
