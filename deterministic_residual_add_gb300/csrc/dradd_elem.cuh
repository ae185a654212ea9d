// dradd_elem.cuh -- element types of the training and rotary kernels: bf16,
// fp16 and fp32 tensors, moved in blocks of 8 elements (16 or 32 bytes) and
// computed in fp32.  Stores round to nearest, ties to even.
#pragma once

#include <cuda_fp16.h>

#include "dradd_device.cuh"

namespace dradd {

// The values of DRADD_BF16, DRADD_F16 and DRADD_F32.
enum ElemKind : int { kElemBf16 = 0, kElemF16 = 1, kElemF32 = 2 };

template <int E>
struct Elem;

template <>
struct Elem<kElemBf16> {
    using T = uint16_t;
    using Block = uint4;
    static __device__ __forceinline__ float widen(T v) { return __uint_as_float(static_cast<uint32_t>(v) << 16); }
    static __device__ __forceinline__ T narrow(float f) { return static_cast<T>(pack_rne(f, 0.0f)); }
    static __device__ __forceinline__ void unpack(const Block& b, float (&f)[8]) { unpack8(b, f); }
    static __device__ __forceinline__ Block pack(const float (&f)[8]) { return pack8_rne(f); }
};

template <>
struct Elem<kElemF16> {
    using T = uint16_t;
    using Block = uint4;
    static __device__ __forceinline__ float widen(T v) { return __half2float(__ushort_as_half(v)); }
    static __device__ __forceinline__ T narrow(float f) { return __half_as_ushort(__float2half_rn(f)); }
    static __device__ __forceinline__ void unpack(const Block& b, float (&f)[8])
    {
        const uint32_t w[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = widen(static_cast<T>(w[i] & 0xFFFFu));
            f[2 * i + 1] = widen(static_cast<T>(w[i] >> 16));
        }
    }
    static __device__ __forceinline__ uint32_t pack2(float lo, float hi)
    {
        uint32_t d;
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
        return d;
    }
    static __device__ __forceinline__ Block pack(const float (&f)[8])
    {
        return make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
    }
};

struct F32Block {
    uint4 lo, hi;
};

template <>
struct Elem<kElemF32> {
    using T = float;
    using Block = F32Block;
    static __device__ __forceinline__ float widen(T v) { return v; }
    static __device__ __forceinline__ T narrow(float f) { return f; }
    static __device__ __forceinline__ void unpack(const Block& b, float (&f)[8])
    {
        const uint32_t w[8] = {b.lo.x, b.lo.y, b.lo.z, b.lo.w, b.hi.x, b.hi.y, b.hi.z, b.hi.w};
#pragma unroll
        for (int i = 0; i < 8; ++i)
            f[i] = __uint_as_float(w[i]);
    }
    static __device__ __forceinline__ Block pack(const float (&f)[8])
    {
        F32Block b;
        b.lo = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
        b.hi = make_uint4(__float_as_uint(f[4]), __float_as_uint(f[5]), __float_as_uint(f[6]), __float_as_uint(f[7]));
        return b;
    }
};

// Block `i` of 8 elements behind a 16-byte aligned pointer.  stream: read or
// written once (evict first); plain: shared memory, or data read again.
__device__ __forceinline__ void ld_block_stream(const uint16_t* p, int64_t i, uint4& b)
{
    b = ld_stream(reinterpret_cast<const uint4*>(p) + i);
}
__device__ __forceinline__ void ld_block_stream(const float* p, int64_t i, F32Block& b)
{
    b.lo = ld_stream(reinterpret_cast<const uint4*>(p) + 2 * i);
    b.hi = ld_stream(reinterpret_cast<const uint4*>(p) + 2 * i + 1);
}
__device__ __forceinline__ void ld_block(const uint16_t* p, int64_t i, uint4& b)
{
    b = *(reinterpret_cast<const uint4*>(p) + i);
}
__device__ __forceinline__ void ld_block(const float* p, int64_t i, F32Block& b)
{
    b.lo = *(reinterpret_cast<const uint4*>(p) + 2 * i);
    b.hi = *(reinterpret_cast<const uint4*>(p) + 2 * i + 1);
}
__device__ __forceinline__ void st_block_stream(uint16_t* p, int64_t i, const uint4& b)
{
    st_stream(reinterpret_cast<uint4*>(p) + i, b);
}
__device__ __forceinline__ void st_block_stream(float* p, int64_t i, const F32Block& b)
{
    st_stream(reinterpret_cast<uint4*>(p) + 2 * i, b.lo);
    st_stream(reinterpret_cast<uint4*>(p) + 2 * i + 1, b.hi);
}

}  // namespace dradd
