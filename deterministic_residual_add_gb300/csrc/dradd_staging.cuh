// dradd_staging.cuh -- the way of an epilogue warp's results out of a product
// kernel, and of what they are joined with in, through a box in shared memory.
#pragma once

#include <cstdint>

namespace dradd {

constexpr uint32_t kStagingBox = 4096;  // 32 rows and 64 columns of 16 bits

// An epilogue warp's box.  Lane i has row i.  A 16-byte piece lies at its
// place xor the row's lowest bits, as the tensor map's swizzle has it, and
// eight lanes that move a piece each touch all banks.
//
// Results stored by the lanes themselves, a 32-byte sector of a row each,
// took 5.6 us for a tile of 128 x 256 (8192 x 512 by 8192: 78 us); through
// here whole lines leave.
struct Staging {
    uint32_t at;     // shared address
    uint64_t* bar;   // counts what comes in
    uint64_t limit_ns;
    uint32_t phase;
    int lane;
    bool failed;
    bool coming;  // something is on its way in

    // Before the first of a box's columns is written: what was stored from
    // here has been read.
    __device__ __forceinline__ void acquire(int c)
    {
        if ((c & 63) != 0)
            return;
        if (lane == 0)
            bulk_wait_read();
        __syncwarp();
    }
    // The same, and then something comes in.
    __device__ __forceinline__ void load(const CUtensorMap* map, int x, int y)
    {
        if (failed)
            return;
        fence_proxy_async_smem();  // behind what was read and written here
        if (lane == 0)
            bulk_wait_read();
        __syncwarp();
        if (lane == 0) {
            mbar_arrive_expect_tx(bar, kStagingBox);
            copy_box<1>(at, map, x, y, bar);
        }
        coming = true;
    }
    // Waits for it; a wait that gave up ends the warp's work behind this tile,
    // whose results are then not to be used, and nothing more comes in.
    __device__ __forceinline__ void loaded()
    {
        if (failed)
            return;
        coming = failed = !arrived();
        phase ^= failed ? 0u : 1u;
    }
    __device__ __forceinline__ bool arrived() const
    {
        return __all_sync(0xffffffffu, mbar_wait_bounded(bar, phase, limit_ns));
    }
    // Before the warp leaves: what a wait gave up on, or what no tile's
    // results came for, is waited for once more.
    __device__ __forceinline__ bool drained()
    {
        return !coming || arrived();
    }
    // Columns c to c + 15 of the lane's row.
    __device__ __forceinline__ uint32_t piece(int c, int i) const
    {
        return at + lane * 128u + (((((c & 63) >> 3) + i) ^ (lane & 7)) << 4);
    }
    __device__ __forceinline__ void read(int c, uint32_t (&w)[8]) const
    {
        const uint4 a = ld_shared(piece(c, 0)), b = ld_shared(piece(c, 1));
        w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
        w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
    }
    __device__ __forceinline__ void write(int c, const uint32_t (&w)[8]) const
    {
        st_shared(piece(c, 0), w[0], w[1], w[2], w[3]);
        st_shared(piece(c, 1), w[4], w[5], w[6], w[7]);
    }
    // The box that column c is the last 16 of goes out, once it is full.
    __device__ __forceinline__ void store_full(const CUtensorMap* map, int c, int x, int y, bool inside) const
    {
        if ((c & 63) != 48)
            return;
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0 && inside) {
            store_box(map, x + c - 48, y, at);
            bulk_commit();
        }
    }
};

}  // namespace dradd
