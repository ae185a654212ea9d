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
// Its top 32 bits (2^-32 turns), rounded to fp32 (2^-26 turns at most), go to
// sincospif.  fp32 angles would lose far positions: at 2^20 they are off by
// 2^-5 radians.  Three integer multiplies and no fp64 outside the one
// conversion a CTA makes.
//
// Work layout.  A unit is 16 columns of a head: in the halves layout 8
// columns and their partners, or 16 that pass; interleaved 16 consecutive
// ones.  A head's units go to `group` neighbouring lanes (a power of two, so
// the norm's sums are butterflies within the group), so a warp takes
// 32 / group heads at a time: of one token, or, where that would leave lanes
// idle, one head each of several tokens.  One such step is all of q or all of
// k.  A warp takes steps_per_warp steps in a row, across tokens, and computes
// the cosines and sines of the tokens it comes to, two or so a lane, into
// shared memory of its own; no barrier but the CTA's first.
//
// Bound by the memory (2 elements of traffic an element, the gradient 3), so
// the bytes on their way count: every lane copies its vectors of the next
// steps, across tokens, into slots of shared memory that only it reads
// (cp.async, so no barrier and no registers).
//
// Measured on GB300 (device time, inputs and outputs of every pass its own;
// share of the 6.79 TB/s a copy reaches), 32 + 8 heads of 128, bf16: rotation
// of 4096 tokens 16.4 us (75 %), of 8192 28.9 (85 %), behind the norm of 8192
// tokens 29.9 us (83 %), its gradient for 4096 tokens 26.6 us (70 %); fp32
// 38.3 (64 %), 69.2 (71 %) and, the gradient, 72.7 (51 %).  The sweeps noted
// in the code shared their outputs between passes, which reads 1 to 3 us
// lower.  What holds the norm's kernels back: about 250 and 290 instructions a
// warp and step against 160 for the rotation alone, at an issue rate of 73 %
// with 32 warps an SM; 56 % with the gradient's 16 (128 registers: the 32 sums
// of both weights' gradients live there; fp32 spills 56 to 76 bytes), which do
// not cover their latency.  Three CTAs of 80 registers spill (62.6 us); a
// chunk of two steps with one look at the walk took fewer instructions and
// more time; so did one walk for loads and stores, whose notes of the steps
// between cost more than a second walk.
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
    const auto clip = [](int n) { return n < 0 ? 0 : n > 8 ? 8 : n; };
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
        c.a = c.b = c.na = c.nb = c.pairs = 0;
    if (c.nb == 0)
        c.b = c.a;  // never used, but inside the head
    return c;
}

// BLOCKS, below: every run is a whole, 16-byte aligned block of 8.

// A table of 16 floats a unit in shared memory, in four planes of one
// 16-byte quad a unit, so that neighbouring lanes (units) read neighbouring
// quads without bank conflicts: element i of unit u of n lies at
// table_at(n, u, i), and `units` below is n.
__host__ __device__ constexpr int table_at(int n, int u, int i) { return ((i >> 2) * n + u) * 4 + (i & 3); }

// The unit's 16 floats as two runs of 8; p points at its first quad.
__device__ __forceinline__ void load_table(const float* p, int units, float (&a)[8], float (&b)[8])
{
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float4 va = *reinterpret_cast<const float4*>(p + i * units * 4);
        const float4 vb = *reinterpret_cast<const float4*>(p + (i + 2) * units * 4);
        a[4 * i] = va.x; a[4 * i + 1] = va.y; a[4 * i + 2] = va.z; a[4 * i + 3] = va.w;
        b[4 * i] = vb.x; b[4 * i + 1] = vb.y; b[4 * i + 2] = vb.z; b[4 * i + 3] = vb.w;
    }
}

// Turns the unit's first `pairs` pairs by their cosines and sines (its table
// entry: 8 cosines, then 8 sines); the others stay, whatever they hold.  In the
// halves layout a unit's pairs all turn or lie outside the head: those are
// turned by what the table holds past rot / 2, and come out finite only where
// that is.
template <bool INTER>
__device__ __forceinline__ void turn_unit(const float* entry, int units, int pairs, float (&a)[8], float (&b)[8])
{
    float c[8], s[8];
    load_table(entry, units, c, s);
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

// The weights of q and of k in fp32, a table each, in the order of the
// unit's columns (0 past the head).
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
        table[side * p.units * 16 + table_at(p.units, r >> 4, r & 15)] = v;
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

// The unit behind p (its first run; the second `second` bytes on), element by
// element; zeros where the head ends.
template <int E>
__device__ __forceinline__ void load_elements(const char* p, int second, const UnitColumns& c, bool active,
                                              RawUnit<E, false>& r)
{
    using T = typename Elem<E>::T;
    const T* a = reinterpret_cast<const T*>(p);
    const T* b = reinterpret_cast<const T*>(p + second);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        r.a[e] = active && e < c.na ? __ldcs(a + e) : T{};
        r.b[e] = active && e < c.nb ? __ldcs(b + e) : T{};
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
__device__ __forceinline__ void store_unit(const char* at, int second, const UnitColumns& c, bool active,
                                           const float (&a)[8], const float (&b)[8])
{
    using T = typename Elem<E>::T;
    T* pa = reinterpret_cast<T*>(const_cast<char*>(at));
    T* pb = reinterpret_cast<T*>(const_cast<char*>(at) + second);
    if constexpr (BLOCKS) {
        if (active && c.na)
            st_block_stream(pa, 0, Elem<E>::pack(a));
        if (active && c.nb)
            st_block_stream(pb, 0, Elem<E>::pack(b));
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if (active && e < c.na)
                __stcs(pa + e, Elem<E>::narrow(a[e]));
            if (active && e < c.nb)
                __stcs(pb + e, Elem<E>::narrow(b[e]));
        }
    }
}

// The lane's share of sum x y over its two runs: four chains of fused
// multiply-adds, two to an instruction, then their sum.
__device__ __forceinline__ float unit_dot(const float (&xa)[8], const float (&xb)[8], const float (&ya)[8],
                                          const float (&yb)[8])
{
    float a0, a1, b0, b1;
    mul2_rn(xa[0], xa[1], ya[0], ya[1], a0, a1);
    mul2_rn(xb[0], xb[1], yb[0], yb[1], b0, b1);
#pragma unroll
    for (int e = 2; e < 8; e += 2) {
        fma2_rn(xa[e], xa[e + 1], ya[e], ya[e + 1], a0, a1, a0, a1);
        fma2_rn(xb[e], xb[e + 1], yb[e], yb[e + 1], b0, b1, b0, b1);
    }
    add2_rn(a0, a1, b0, b1, a0, a1);
    return __fadd_rn(a0, a1);
}

// 1 / sqrt(v): the reciprocal square root approximation (within 2^-22.9)
// with one Newton step, r + r (1/2 - v/2 r r), which leaves less than 2^-23
// relative.  v = 0 and v = inf keep the approximation's inf and 0.
__device__ __forceinline__ float inv_sqrt(float v)
{
    float r;
    asm("rsqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(v));
    const float h = __fmul_rn(-0.5f, v);
    const float e = __fmaf_rn(__fmul_rn(h, r), r, 0.5f);
    const float n = __fmaf_rn(r, e, r);
    return v > 0.0f && v < __int_as_float(0x7f800000) ? n : r;
}

// The mean over a head of a sum over it.
__device__ __forceinline__ float head_mean(const RopeArgs& p, float sum)
{
    return __fmul_rn(sum, p.inv_dim);
}

// A lane's ring of shared memory: kSlots steps, one being computed while the
// others are on their way; a step is the 16-byte pieces of N tensors' runs,
// then the position.  Two steps ahead measured best: q and k of 8192 tokens
// behind the norm 29.7 us, one ahead 30.3, three 30.4, four 31.5 (more
// shared memory leaves less of it as cache).
template <int E, int N>
struct RopeRing {
    static constexpr int kVec = E == kElemF32 ? 2 : 1;  // pieces of a run
    static constexpr int kPieces = 2 * N * kVec;
    static constexpr int kPosition = kPieces * 512;
    static constexpr int kStepBytes = kPosition + 256;
    static constexpr int kSlots = 3;
    static constexpr int kBytes = kSlots * kStepBytes * (kRopeThreads / 32);
    static __device__ __forceinline__ uint32_t after(uint32_t slot, uint32_t ring)
    {
        return slot == ring + (kSlots - 1) * kStepBytes ? ring : slot + kStepBytes;
    }
    static __device__ __forceinline__ uint32_t before(uint32_t slot, uint32_t ring)
    {
        return slot == ring ? ring + (kSlots - 1) * kStepBytes : slot - kStepBytes;
    }
};

// The CTA's shared memory: the warps' rings (BLOCKS only), the pairs'
// fractions, the weights (norm only), then every warp's tables of cosines and
// sines.
struct RopeShared {
    unsigned char* ring;  // this warp's
    uint64_t* fractions;
    float* weights;
    float* table;  // this warp's
};

// Tables of cosines and sines a warp keeps.
template <bool TOK>
__host__ __device__ __forceinline__ int rope_tables(const RopeArgs& p)
{
    return TOK ? 32 / p.group : 1;
}

template <bool NORM, bool TOK>
__device__ __forceinline__ RopeShared rope_shared(const RopeArgs& p, unsigned char* mem, int ring_bytes)
{
    const int warp = threadIdx.x >> 5;
    RopeShared sh;
    sh.ring = mem + warp * (ring_bytes / (kRopeThreads / 32));
    sh.fractions = reinterpret_cast<uint64_t*>(mem + ring_bytes);
    sh.weights = reinterpret_cast<float*>(sh.fractions + 8 * p.rot_units);
    sh.table = sh.weights + (NORM ? 32 * p.units : 0) + warp * rope_tables<TOK>(p) * 16 * p.rot_units;
    return sh;
}

template <int E, bool NORM, bool INTER>
__device__ __forceinline__ void rope_prologue(const RopeArgs& p, const RopeShared& sh)
{
    for (int i = threadIdx.x; i < (p.rot >> 1); i += kRopeThreads)
        sh.fractions[i] = turn_fraction(__ldg(p.inv_freq + i));
    if constexpr (NORM)
        fill_weights<E, INTER>(p, sh.weights);
    __syncthreads();
}

// Zeros in all of the warp's tables, for a kernel whose sums take in the
// columns outside the head too (after turn_unit in the halves layout, where
// rot / 2 is no multiple of 8): shared memory may hold NaN, and 0 * NaN would
// reach every column of the head.
template <bool TOK>
__device__ __forceinline__ void clear_tables(const RopeArgs& p, const RopeShared& sh, int lane)
{
    for (int i = lane; i < rope_tables<TOK>(p) * 16 * p.rot_units; i += 32)
        sh.table[i] = 0.0f;
}

// The table of the lane's token, filled by the warp together, or by each
// lane group for its own token.  What lies past rot / 2 is left as it is.
template <bool TOK>
__device__ __forceinline__ void fill_angles(const RopeArgs& p, const RopeShared& sh, int64_t position, int lane,
                                            int group)
{
    float* const table = sh.table + (TOK ? (lane / group) * 16 * p.rot_units : 0);
    __syncwarp();
    for (int i = TOK ? lane & (group - 1) : lane; i < (p.rot >> 1); i += TOK ? group : 32) {
        float c, s;
        turn_cos_sin(sh.fractions[i], position, c, s);
        table[table_at(p.rot_units, i >> 3, i & 7)] = __fmul_rn(c, p.scale);
        table[table_at(p.rot_units, i >> 3, 8 + (i & 7))] = __fmul_rn(s, __fmul_rn(p.scale, p.sign));
    }
    __syncwarp();
}

// A warp's steps: `count` of them from step `first` of item `item` on.
struct WarpRange {
    uint32_t item;
    int first, count;
};

__device__ __forceinline__ WarpRange warp_range(const RopeArgs& p, uint32_t warp)
{
    const int64_t from = static_cast<int64_t>(warp) * p.steps_per_warp;
    const int64_t left = p.n_steps - from;
    const uint32_t steps = static_cast<uint32_t>(p.q_steps + p.k_steps);
    WarpRange r = {0, 0, 0};
    if (left > 0) {
        r.count = left < p.steps_per_warp ? static_cast<int>(left) : p.steps_per_warp;
        r.item = p.n_steps >> 32 ? static_cast<uint32_t>(from / steps) : static_cast<uint32_t>(from) / steps;
        r.first = static_cast<int>(from - static_cast<int64_t>(r.item) * steps);
    }
    return r;
}

// One lane's way through the steps of an item in the tensors W: first
// its heads of q, then those of k.  Everything but the addresses and `left`
// is uniform over the warp; with TOK the token is the lane group's own.
template <bool TOK, int... W>
struct HeadWalk {
    static constexpr int N = sizeof...(W);
    const char* at[N];  // the lane's first column in its head of this step
    int steps;          // left of the item, this one included
    int side_steps;     // left of q, or of k
    int left;           // heads of this side from the lane's on; <= 0: none
    bool is_k;
    bool real;          // TOK: the lane's token is one of the call's
    uint32_t b, s;      // the lane's token

    __device__ __forceinline__ int64_t token(const RopeArgs& p) const { return b * p.seq + s; }
    __device__ __forceinline__ void side(const RopeArgs& p, const RopeSide& sd, int step, int per_step, int g,
                                         int first_byte)
    {
        constexpr int which[N] = {W...};
        const int head = step * per_step + (TOK ? 0 : g);
        left = !TOK || real ? sd.heads - head : 0;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const HeadsView& v = sd.t[which[i]];
            at[i] = v.data + b * v.batch + s * v.seq + head * v.head + first_byte;
        }
    }
    // To step `first` of an item, for `most` steps or to its end.
    __device__ __forceinline__ void begin(const RopeArgs& p, uint32_t item, int first, int most, int per_step, int g,
                                          int first_byte)
    {
        uint32_t token = item;
        if constexpr (TOK) {
            token = item * (32u / p.group) + g;
            real = token < p.tokens;
            if (!real)
                token = item * (32u / p.group);  // not read, but an address inside the tensor
        }
        b = token / static_cast<uint32_t>(p.seq);
        s = token - b * static_cast<uint32_t>(p.seq);
        const int all = p.q_steps + p.k_steps - first;
        steps = all < most ? all : most;
        side_steps = p.q_steps - first;
        is_k = side_steps <= 0;
        if (is_k)
            side(p, p.k, -side_steps, per_step, g, first_byte);
        else
            side(p, p.q, first, per_step, g, first_byte);
    }
    __device__ __forceinline__ bool active() const { return left > 0; }
    // On to the next step; false when this one was the last.
    __device__ __forceinline__ bool advance(const RopeArgs& p, int per_step, int g, int first_byte)
    {
        if (--steps == 0)
            return false;
        if (--side_steps == 0) {
            is_k = true;
            side(p, p.k, 0, per_step, g, first_byte);
            return true;
        }
        constexpr int which[N] = {W...};
        left -= per_step;
#pragma unroll
        for (int i = 0; i < N; ++i)
            at[i] += is_k ? p.k.t[which[i]].step : p.q.t[which[i]].step;
        return true;
    }
};

// The copies ahead of the computation: the tensors W of the warp's steps,
// one by one, into the lane's slots.  A run the lane's head does
// not have is never copied (its slot keeps the zeros it starts with); a head
// the step does not have leaves what was there, which nobody uses.
template <int E, bool TOK, int... W>
struct RopeAhead {
    static constexpr int N = sizeof...(W);
    using Ring = RopeRing<E, N>;
    HeadWalk<TOK, W...> walk;
    uint32_t item;
    bool fresh;  // the walk stands at an item's first step for this warp

    __device__ __forceinline__ void begin(const RopeArgs& p, const WarpRange& r, int per_step, int g,
                                          int first_byte)
    {
        item = r.item;
        fresh = true;
        if (r.count > 0)
            walk.begin(p, item, r.first, r.count, per_step, g, first_byte);
    }
    // Copies one step into a slot, or nothing when no work is left.  rest:
    // the warp's steps from this one on; slot: of the lane's 16-byte pieces.
    __device__ __forceinline__ void issue(const RopeArgs& p, int rest, uint32_t slot, int lane, int per_step, int g,
                                          int first_byte, int second, bool has_a, bool has_b)
    {
        if (rest > 0) {
            if (walk.active()) {
#pragma unroll
                for (int i = 0; i < N; ++i) {
#pragma unroll
                    for (int v = 0; v < Ring::kVec; ++v) {
                        const uint32_t dst = slot + (2 * i * Ring::kVec + v) * 512;
                        if (has_a)
                            copy_ahead16(dst, walk.at[i] + 16 * v);
                        if (has_b)
                            copy_ahead16(dst + Ring::kVec * 512, walk.at[i] + second + 16 * v);
                    }
                }
            }
            if (fresh && p.positions)
                copy_ahead8(slot + Ring::kPosition - 8 * lane, p.positions + walk.token(p));
            fresh = !walk.advance(p, per_step, g, first_byte);
            if (fresh && rest > 1)
                walk.begin(p, ++item, 0, rest - 1, per_step, g, first_byte);
        }
        copy_ahead_commit();
    }
};

template <int E, int N>
__device__ __forceinline__ void read_slot(uint32_t slot, int i, RawUnit<E, true>& r)
{
    using Ring = RopeRing<E, N>;
    const uint32_t at = slot + 2 * i * Ring::kVec * 512;
    if constexpr (Ring::kVec == 1) {
        r.a = lds16(at);
        r.b = lds16(at + 512);
    } else {
        r.a.lo = lds16(at);
        r.a.hi = lds16(at + 512);
        r.b.lo = lds16(at + 1024);
        r.b.hi = lds16(at + 1536);
    }
}

template <typename Ring>
__device__ __forceinline__ void clear_ring(unsigned char* ring, int lane)
{
    for (int i = lane; i < Ring::kSlots * Ring::kStepBytes / 16; i += 32)
        reinterpret_cast<uint4*>(ring)[i] = make_uint4(0u, 0u, 0u, 0u);
    __syncwarp();
}

// G: lanes per head, or 0 for p.group (element-wise kernels, which have
// more to do than a butterfly's branches).
template <int G>
__device__ __forceinline__ float head_sum(float v, int group)
{
    return butterfly_sum(v, G ? G : group);
}

// Forward: plain (NORM false; also the inverse) or behind the norm
//   z = (x * inv) * w, inv = 1 / sqrt(sum x^2 / dim + eps).
template <int E, bool NORM, bool INTER, int G, bool TOK>
__global__ void __launch_bounds__(kRopeThreads, E == kElemF32 ? 3 : 4) rope_fwd_kernel(const RopeArgs p)
{
    constexpr bool BLOCKS = G != 0;
    using T = typename Elem<E>::T;
    using Ring = RopeRing<E, 1>;
    extern __shared__ __align__(16) unsigned char mem[];
    const RopeShared sh = rope_shared<NORM, TOK>(p, mem, BLOCKS ? Ring::kBytes : 0);
    const int lane = threadIdx.x & 31;
    const int group = G ? G : p.group;
    const int per_step = TOK ? 1 : G ? 32 / (G ? G : 1) : p.heads_per_step;
    const int u = lane & (group - 1);
    const int g = lane / group;
    const UnitColumns cols = unit_columns<INTER>(p, u);
    const bool has_a = cols.na != 0, has_b = cols.nb != 0;
    const int first_byte = cols.a * static_cast<int>(sizeof(T));
    const int second = (cols.b - cols.a) * static_cast<int>(sizeof(T));
    WarpRange range = warp_range(p, blockIdx.x * (kRopeThreads / 32) + (threadIdx.x >> 5));
    const uint32_t ring = smem_u32(sh.ring) + lane * 16;
    wait_prior_grids();
    allow_next_grid();
    RopeAhead<E, TOK, kRopeIn> ahead;
    if constexpr (BLOCKS) {
        clear_ring<Ring>(sh.ring, lane);
        ahead.begin(p, range, per_step, g, first_byte);
#pragma unroll
        for (int i = 0; i < Ring::kSlots - 1; ++i)
            ahead.issue(p, range.count - i, ring + i * Ring::kStepBytes, lane, per_step, g, first_byte, second, has_a, has_b);
    }
    rope_prologue<E, NORM, INTER>(p, sh);
    const float* const turn = sh.table + (TOK ? g * 16 * p.rot_units : 0) + (cols.pairs ? u : 0) * 4;
    const float* const weight = sh.weights + (u < p.units ? u : 0) * 4;
    const bool rest = cols.pairs == 0;
    const bool skip_q = rest && p.q.skip_rest, skip_k = rest && p.k.skip_rest;
    uint32_t slot = ring;
    // The slot to fill, the one before `slot`: kept behind the norm (8192
    // tokens of 32 + 8 heads 29.3 us, computed 30.4), computed without it
    // (4096 tokens 13.0, kept 14.2: a register spills).
    uint32_t into = ring + (Ring::kSlots - 1) * Ring::kStepBytes;
    HeadWalk<TOK, kRopeOut, kRopeIn> walk;  // out, and x where it is not copied ahead
    while (range.count > 0) {
        walk.begin(p, range.item, range.first, range.count, per_step, g, first_byte);
        bool fresh = true;
        do {
            if constexpr (BLOCKS) {
                ahead.issue(p, range.count - (Ring::kSlots - 1), NORM ? into : Ring::before(slot, ring), lane, per_step, g,
                            first_byte, second, has_a, has_b);
                into = Ring::after(into, ring);
                copy_ahead_wait<Ring::kSlots - 1>();
            }
            if (fresh) {
                int64_t position = p.position0 + walk.s;
                if (p.positions)
                    position = BLOCKS ? lds8(slot + Ring::kPosition - 8 * lane) : __ldg(p.positions + walk.token(p));
                fill_angles<TOK>(p, sh, position, lane, group);
                fresh = false;
            }
            const float eps = walk.is_k ? p.k.eps : p.q.eps;
            const float* const w_side = weight + (walk.is_k ? p.units * 16 : 0);
            const bool skip = walk.is_k ? skip_k : skip_q;
            const bool active = walk.active();
            RawUnit<E, BLOCKS> x;
            if constexpr (BLOCKS)
                read_slot<E, 1>(slot, 0, x);
            else
                load_elements<E>(walk.at[1], second, cols, active, x);
            float a[8], b[8];
            widen_unit<E, BLOCKS>(x, a, b);
            if constexpr (NORM) {
                const float sq = head_sum<G>(unit_dot(a, b, a, b), group);
                const float inv = inv_sqrt(__fadd_rn(head_mean(p, sq), eps));
                float wa[8], wb[8];
                load_table(w_side, p.units, wa, wb);
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    mul2_rn(a[e], a[e + 1], inv, inv, a[e], a[e + 1]);
                    mul2_rn(b[e], b[e + 1], inv, inv, b[e], b[e + 1]);
                    mul2_rn(a[e], a[e + 1], wa[e], wa[e + 1], a[e], a[e + 1]);
                    mul2_rn(b[e], b[e + 1], wb[e], wb[e + 1], b[e], b[e + 1]);
                }
            }
            if (!rest)
                turn_unit<INTER>(turn, p.rot_units, cols.pairs, a, b);
            store_unit<E, BLOCKS>(walk.at[0], second, cols, active && !skip, a, b);
            slot = Ring::after(slot, ring);
            --range.count;
        } while (walk.advance(p, per_step, g, first_byte));
        ++range.item;
        range.first = 0;
    }
}

// The gradients of the fused call, with g = turn(-theta) dy:
//   S1 = sum x^2, S2 = sum (g w) x; c = inv (inv (S2 / dim))
//   dx = inv (g w - x c); dweight += g (x inv), over tokens and heads.
// Every lane adds the shares of its warp's work in order in registers; at
// the end a warp's groups are added by butterfly and the CTA's warps in
// order into the CTA's part.
template <int E, bool INTER, int G, bool TOK>
__global__ void __launch_bounds__(kRopeThreads, 2) rope_bwd_kernel(const RopeArgs p)
{
    constexpr bool BLOCKS = G != 0;
    using T = typename Elem<E>::T;
    using Ring = RopeRing<E, 2>;
    extern __shared__ __align__(16) unsigned char mem[];
    const RopeShared sh = rope_shared<true, TOK>(p, mem, BLOCKS ? Ring::kBytes : 0);
    const int lane = threadIdx.x & 31;
    const int group = G ? G : p.group;
    const int per_step = TOK ? 1 : G ? 32 / (G ? G : 1) : p.heads_per_step;
    const int u = lane & (group - 1);
    const int g = lane / group;
    const UnitColumns cols = unit_columns<INTER>(p, u);
    const bool has_a = cols.na != 0, has_b = cols.nb != 0;
    const int first_byte = cols.a * static_cast<int>(sizeof(T));
    const int second = (cols.b - cols.a) * static_cast<int>(sizeof(T));
    WarpRange range = warp_range(p, blockIdx.x * (kRopeThreads / 32) + (threadIdx.x >> 5));
    const uint32_t ring = smem_u32(sh.ring) + lane * 16;
    wait_prior_grids();
    allow_next_grid();
    RopeAhead<E, TOK, kRopeIn, kRopeGrad> ahead;
    if constexpr (BLOCKS) {
        clear_ring<Ring>(sh.ring, lane);
        ahead.begin(p, range, per_step, g, first_byte);
#pragma unroll
        for (int i = 0; i < Ring::kSlots - 1; ++i)
            ahead.issue(p, range.count - i, ring + i * Ring::kStepBytes, lane, per_step, g, first_byte, second, has_a, has_b);
    }
    if constexpr (!BLOCKS && !INTER)
        clear_tables<TOK>(p, sh, lane);
    rope_prologue<E, true, INTER>(p, sh);
    const float* const turn = sh.table + (TOK ? g * 16 * p.rot_units : 0) + (cols.pairs ? u : 0) * 4;
    const float* const weight = sh.weights + (u < p.units ? u : 0) * 4;
    float dq[2][8] = {}, dk[2][8] = {};
    uint32_t slot = ring;
    HeadWalk<TOK, kRopeOut, kRopeIn, kRopeGrad> walk;
    while (range.count > 0) {
        walk.begin(p, range.item, range.first, range.count, per_step, g, first_byte);
        bool fresh = true;
        do {
            if constexpr (BLOCKS) {
                ahead.issue(p, range.count - (Ring::kSlots - 1), Ring::before(slot, ring), lane, per_step, g, first_byte,
                            second, has_a, has_b);
                copy_ahead_wait<Ring::kSlots - 1>();
            }
            if (fresh) {
                int64_t position = p.position0 + walk.s;
                if (p.positions)
                    position = BLOCKS ? lds8(slot + Ring::kPosition - 8 * lane) : __ldg(p.positions + walk.token(p));
                fill_angles<TOK>(p, sh, position, lane, group);
                fresh = false;
            }
            const float eps = walk.is_k ? p.k.eps : p.q.eps;
            const float* const w_side = weight + (walk.is_k ? p.units * 16 : 0);
            const bool active = walk.active();
            RawUnit<E, BLOCKS> x, dy;
            if constexpr (BLOCKS) {
                read_slot<E, 2>(slot, 0, x);
                read_slot<E, 2>(slot, 1, dy);
            } else {
                load_elements<E>(walk.at[1], second, cols, active, x);
                load_elements<E>(walk.at[2], second, cols, active, dy);
            }
            float a[8], b[8], ga[8], gb[8], wa[8], wb[8];
            widen_unit<E, BLOCKS>(x, a, b);
            widen_unit<E, BLOCKS>(dy, ga, gb);
            if (cols.pairs)
                turn_unit<INTER>(turn, p.rot_units, cols.pairs, ga, gb);
            load_table(w_side, p.units, wa, wb);
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
                mul2_rn(ga[e], ga[e + 1], wa[e], wa[e + 1], wa[e], wa[e + 1]);
                mul2_rn(gb[e], gb[e + 1], wb[e], wb[e + 1], wb[e], wb[e + 1]);
            }
            const float s1 = head_sum<G>(unit_dot(a, b, a, b), group);
            const float s2 = head_sum<G>(unit_dot(a, b, wa, wb), group);
            const float inv = inv_sqrt(__fadd_rn(head_mean(p, s1), eps));
            const float c = -__fmul_rn(inv, __fmul_rn(inv, head_mean(p, s2)));
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
                fma2_rn(a[e], a[e + 1], c, c, wa[e], wa[e + 1], wa[e], wa[e + 1]);
                fma2_rn(b[e], b[e + 1], c, c, wb[e], wb[e + 1], wb[e], wb[e + 1]);
                mul2_rn(wa[e], wa[e + 1], inv, inv, wa[e], wa[e + 1]);
                mul2_rn(wb[e], wb[e + 1], inv, inv, wb[e], wb[e + 1]);
                mul2_rn(a[e], a[e + 1], inv, inv, a[e], a[e + 1]);
                mul2_rn(b[e], b[e + 1], inv, inv, b[e], b[e + 1]);
            }
            if (active) {  // a lane without a head adds nothing
                if (walk.is_k) {
#pragma unroll
                    for (int e = 0; e < 8; e += 2) {
                        fma2_rn(ga[e], ga[e + 1], a[e], a[e + 1], dk[0][e], dk[0][e + 1], dk[0][e], dk[0][e + 1]);
                        fma2_rn(gb[e], gb[e + 1], b[e], b[e + 1], dk[1][e], dk[1][e + 1], dk[1][e], dk[1][e + 1]);
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 8; e += 2) {
                        fma2_rn(ga[e], ga[e + 1], a[e], a[e + 1], dq[0][e], dq[0][e + 1], dq[0][e], dq[0][e + 1]);
                        fma2_rn(gb[e], gb[e + 1], b[e], b[e + 1], dq[1][e], dq[1][e + 1], dq[1][e], dq[1][e + 1]);
                    }
                }
            }
            store_unit<E, BLOCKS>(walk.at[0], second, cols, active, wa, wb);
            slot = Ring::after(slot, ring);
            --range.count;
        } while (walk.advance(p, per_step, g, first_byte));
        ++range.item;
        range.first = 0;
    }
    if (!p.partials)
        return;
    // warp sums [warp][side][unit][16] over the memory used so far
    copy_ahead_wait<0>();
    float* const sums = reinterpret_cast<float*>(mem);
    const int stride = 32 * p.units;
    __syncthreads();
#pragma unroll
    for (int side = 0; side < 2; ++side) {
        float* at = sums + (threadIdx.x >> 5) * stride + (side * p.units + u) * 16;
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            float v = side ? dk[e >> 3][e & 7] : dq[e >> 3][e & 7];
            for (int d = group; d < 32; d <<= 1)
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
        const bool upper = (r & 8) != 0;
        if (e >= (upper ? c.nb : c.na))
            continue;
        float v = sums[i];
#pragma unroll
        for (int k = 1; k < kRopeThreads / 32; ++k)
            v = __fadd_rn(v, sums[k * stride + i]);
        part[side * p.dim + (upper ? c.b : c.a) + e] = v;
    }
}

// ------------------------------------------------------------------- launch
template <auto FN>
cudaError_t launch_rope_kernel(const RopeArgs& p, int grid, size_t smem, cudaStream_t stream)
{
    if (smem > 48 * 1024) {
        const cudaError_t e = allow_all_shared<FN>();
        if (e != cudaSuccess)
            return e;
    }
    return launch(FN, grid, kRopeThreads, smem, false, stream, p);
}

template <int E, bool INTER, int G, bool TOK>
cudaError_t launch_rope_as(const RopeArgs& p, int mode, int grid, cudaStream_t stream)
{
    constexpr bool BLOCKS = G != 0;
    const bool norm = mode != kRopePlain;
    const int per_cta = 1 + rope_tables<TOK>(p) * (kRopeThreads / 32);  // the fractions, the tables
    const size_t tables = static_cast<size_t>(p.rot_units) * 64 * per_cta + (norm ? p.units * 128 : 0);
    if (mode == kRopeNormBwd) {
        const size_t all = tables + (BLOCKS ? RopeRing<E, 2>::kBytes : 0);
        const size_t sums = static_cast<size_t>(p.units) * 128 * (kRopeThreads / 32);
        return launch_rope_kernel<rope_bwd_kernel<E, INTER, G, TOK>>(p, grid, all > sums ? all : sums, stream);
    }
    const size_t all = tables + (BLOCKS ? RopeRing<E, 1>::kBytes : 0);
    return norm ? launch_rope_kernel<rope_fwd_kernel<E, true, INTER, G, TOK>>(p, grid, all, stream)
                : launch_rope_kernel<rope_fwd_kernel<E, false, INTER, G, TOK>>(p, grid, all, stream);
}

// With 32 lanes a head a warp has one lane group, so TOK does not arise.
template <int E, bool INTER, int G>
cudaError_t launch_rope_group(const RopeArgs& p, int mode, int grid, cudaStream_t stream)
{
    return p.by_token ? launch_rope_as<E, INTER, G, true>(p, mode, grid, stream)
                      : launch_rope_as<E, INTER, G, false>(p, mode, grid, stream);
}

template <int E, bool INTER>
cudaError_t launch_rope_layout(const RopeArgs& p, int mode, bool blocks, int grid, cudaStream_t stream)
{
    if (!blocks)
        return launch_rope_group<E, INTER, 0>(p, mode, grid, stream);
    switch (p.group) {
    case 4:
        return launch_rope_group<E, INTER, 4>(p, mode, grid, stream);
    case 8:
        return launch_rope_group<E, INTER, 8>(p, mode, grid, stream);
    case 16:
        return launch_rope_group<E, INTER, 16>(p, mode, grid, stream);
    default:
        return launch_rope_as<E, INTER, 32, false>(p, mode, grid, stream);
    }
}

template <int E>
cudaError_t launch_rope_of(const RopeArgs& p, int mode, bool interleaved, bool blocks, int grid, cudaStream_t stream)
{
    return interleaved ? launch_rope_layout<E, true>(p, mode, blocks, grid, stream)
                       : launch_rope_layout<E, false>(p, mode, blocks, grid, stream);
}

}  // namespace dradd
