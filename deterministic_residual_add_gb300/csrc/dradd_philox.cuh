// dradd_philox.cuh -- the counter-based generator behind every dropout mask.
//
// Philox4x32 with 7 rounds (Salmon, Moraes, Dror and Shaw, "Parallel random
// numbers: as easy as 1, 2, 3", 2011, who report 7 rounds as the fewest that
// pass BigCrush).  A mask bit is a pure function of (seed, offset, row,
// column): the key is the seed, the counter is (column / 8, row, offset low,
// offset high), and the 128 bits are cut into eight 16-bit numbers, one for
// each of the 8 columns of the block, i.e. one call for each 16-byte vector
// of 2-byte elements.  No state, no stored mask, and no dependence on the
// launch, so the backward pass draws the same bits again.
//
// Why 16 bits and 7 rounds: the generator is 32 x 32 -> 64-bit multiplies,
// and one call for 4 elements of 32 bits each is bound by them.  Dropout of
// 2^27 bf16 elements, same kernel otherwise: 32 bits an element 127 us with
// 10 rounds and 99 us with 7; 16 bits 92 us with 10 and 84 us with 7; a
// plain copy 80 us.
#pragma once

#include <cstdint>

#include "dradd_device.cuh"

namespace dradd {

constexpr int kPhiloxRounds = 7;

// What a kernel needs to draw a mask.  An element is kept when its 16 bits
// are >= t (0: all are kept, 65536: none), and then multiplied by scale =
// 65536 / (65536 - t), so the mean is the input's.  The rounds' keys are laid
// out by the host: in the kernel's constants they cost no instructions.
struct DropParams {
    uint32_t key[2 * kPhiloxRounds];
    uint64_t offset;
    const int64_t* step;  // device memory, added to offset; or NULL
    uint32_t drops;       // whether t > 0
    uint32_t limit;       // t * 65536 - 1: a 32-bit word is above it when its high half is >= t
    float scale;
};

inline DropParams make_drop_params(uint64_t seed, uint64_t offset, const int64_t* step, uint32_t t, float scale)
{
    DropParams d = {};
    uint32_t k0 = static_cast<uint32_t>(seed), k1 = static_cast<uint32_t>(seed >> 32);
    for (int i = 0; i < kPhiloxRounds; ++i) {
        d.key[2 * i] = k0;
        d.key[2 * i + 1] = k1;
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    d.offset = offset;
    d.step = step;
    d.drops = t > 0;
    d.limit = (t << 16) - 1u;
    d.scale = scale;
    return d;
}

// The offset of this run.
__device__ __forceinline__ uint2 drop_offset(const DropParams& d)
{
    uint64_t off = d.offset;
    if (d.step)
        off += static_cast<uint64_t>(*d.step);
    return make_uint2(static_cast<uint32_t>(off), static_cast<uint32_t>(off >> 32));
}

__device__ __forceinline__ uint4 drop_bits(const DropParams& d, const uint2& offset, uint32_t block, uint32_t row)
{
    uint32_t c0 = block, c1 = row, c2 = offset.x, c3 = offset.y;
#pragma unroll
    for (int i = 0; i < kPhiloxRounds; ++i) {
        const uint64_t a = static_cast<uint64_t>(0xD2511F53u) * c0;
        const uint64_t b = static_cast<uint64_t>(0xCD9E8D57u) * c2;
        c0 = static_cast<uint32_t>(b >> 32) ^ c1 ^ d.key[2 * i];
        c1 = static_cast<uint32_t>(b);
        c2 = static_cast<uint32_t>(a >> 32) ^ c3 ^ d.key[2 * i + 1];
        c3 = static_cast<uint32_t>(a);
    }
    return make_uint4(c0, c1, c2, c3);
}

// Element e of a block is kept (its 16 bits: word e / 2, low half first).
__device__ __forceinline__ bool kept(const uint4& bits, int e, uint32_t limit)
{
    const uint32_t word = e < 2 ? bits.x : e < 4 ? bits.y : e < 6 ? bits.z : bits.w;
    return ((e & 1) ? word : word << 16) > limit;
}

// v = kept ? RN(v * scale) : +0 for the 8 elements of block `block` of a row.
// A dropped element is +0 whatever it held (infinities and NaN included).
__device__ __forceinline__ void drop8(float (&v)[8], const DropParams& d, const uint2& offset, uint32_t block,
                                      uint32_t row)
{
    const uint4 bits = drop_bits(d, offset, block, row);
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
        mul2_rn(v[e], v[e + 1], d.scale, d.scale, v[e], v[e + 1]);
        v[e] = kept(bits, e, d.limit) ? v[e] : 0.0f;
        v[e + 1] = kept(bits, e + 1, d.limit) ? v[e + 1] : 0.0f;
    }
}

}  // namespace dradd
