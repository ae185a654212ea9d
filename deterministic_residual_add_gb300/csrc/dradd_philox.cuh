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

namespace dradd {

// What a kernel needs to draw a mask.  An element is kept when its 16 bits
// are >= threshold (0: all are kept, 65536: none), and then multiplied by
// scale = 65536 / (65536 - threshold), so the mean is the input's.
struct DropParams {
    uint32_t seed_lo, seed_hi;
    uint64_t offset;
    const int64_t* step;  // device memory, added to offset; or NULL
    uint32_t threshold;
    float scale;
};

struct DropKey {
    uint32_t k0, k1, c2, c3;
    uint32_t threshold;
    float scale;
};

__device__ __forceinline__ DropKey make_drop_key(const DropParams& d)
{
    uint64_t off = d.offset;
    if (d.step)
        off += static_cast<uint64_t>(*d.step);
    return DropKey{d.seed_lo, d.seed_hi, static_cast<uint32_t>(off), static_cast<uint32_t>(off >> 32),
                   d.threshold, d.scale};
}

__device__ __forceinline__ uint4 philox4x32_7(uint32_t c0, uint32_t c1, uint32_t c2, uint32_t c3, uint32_t k0,
                                              uint32_t k1)
{
#pragma unroll
    for (int i = 0; i < 7; ++i) {
        const uint64_t a = static_cast<uint64_t>(0xD2511F53u) * c0;
        const uint64_t b = static_cast<uint64_t>(0xCD9E8D57u) * c2;
        c0 = static_cast<uint32_t>(b >> 32) ^ c1 ^ k0;
        c1 = static_cast<uint32_t>(b);
        c2 = static_cast<uint32_t>(a >> 32) ^ c3 ^ k1;
        c3 = static_cast<uint32_t>(a);
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return make_uint4(c0, c1, c2, c3);
}

// Element e of a block is kept (its 16 bits: word e / 2, low half first).
__device__ __forceinline__ bool kept(const uint4& bits, int e, uint32_t threshold)
{
    const uint32_t word = e < 2 ? bits.x : e < 4 ? bits.y : e < 6 ? bits.z : bits.w;
    return ((e & 1) ? word >> 16 : word & 0xFFFFu) >= threshold;
}

// v = kept ? RN(v * scale) : +0 for the 8 elements of block `block` of a row.
// A dropped element is +0 whatever it held (infinities and NaN included).
__device__ __forceinline__ void drop8(float (&v)[8], const DropKey& k, uint32_t block, uint32_t row)
{
    const uint4 bits = philox4x32_7(block, row, k.c2, k.c3, k.k0, k.k1);
#pragma unroll
    for (int e = 0; e < 8; ++e)
        v[e] = kept(bits, e, k.threshold) ? __fmul_rn(v[e], k.scale) : 0.0f;
}

}  // namespace dradd
