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
// One 256-bit store where p allows it: two of 16 bytes write half sectors
// (rotation of 4096 tokens of 32 + 8 heads, fp32: 42.4 us, so 38.4; dropout
// 1999 x 5120 12.6, so 10.1).  Loads gain nothing from it.
__device__ __forceinline__ void st_block_stream(float* p, int64_t i, const F32Block& b)
{
    if (reinterpret_cast<uintptr_t>(p) % 32 == 0) {
        asm volatile("st.global.cs.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p + 8 * i), "r"(b.lo.x),
                     "r"(b.lo.y), "r"(b.lo.z), "r"(b.lo.w), "r"(b.hi.x), "r"(b.hi.y), "r"(b.hi.z), "r"(b.hi.w)
                     : "memory");
        return;
    }
    st_stream(reinterpret_cast<uint4*>(p) + 2 * i, b.lo);
    st_stream(reinterpret_cast<uint4*>(p) + 2 * i + 1, b.hi);
}

// ------------------------------------------------- lane-private copies ahead
// Asynchronous copies from global memory into shared memory that only the
// copying thread reads again, so that waiting for its own groups is all the
// synchronisation there is.  Ordinary loads to the memory system: any
// address a load could take.
__device__ __forceinline__ void copy_ahead16(uint32_t dst, const void* src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_ahead8(uint32_t dst, const void* src)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_ahead_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_ahead_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t at)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(at)
                 : "memory");
    return v;
}
__device__ __forceinline__ int64_t lds8(uint32_t at)
{
    int64_t v;
    asm volatile("ld.shared.s64 %0, [%1];" : "=l"(v) : "r"(at) : "memory");
    return v;
}

// A block of 8 elements in such memory: its 16-byte pieces `stride` bytes
// apart.
__device__ __forceinline__ void copy_ahead_block(uint32_t dst, uint32_t stride, const uint16_t* src)
{
    copy_ahead16(dst, src);
}
__device__ __forceinline__ void copy_ahead_block(uint32_t dst, uint32_t stride, const float* src)
{
    copy_ahead16(dst, src);
    copy_ahead16(dst + stride, src + 4);
}
__device__ __forceinline__ void lds_block(uint32_t at, uint32_t stride, uint4& b) { b = lds16(at); }
__device__ __forceinline__ void lds_block(uint32_t at, uint32_t stride, F32Block& b)
{
    b.lo = lds16(at);
    b.hi = lds16(at + stride);
}

}  // namespace dradd
