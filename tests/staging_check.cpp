// The box of an epilogue warp on the host: a warp of one lane, a barrier that
// counts what comes in, and copies that land when they are told to.
#include <cassert>
#include <cstdint>
#include <cstdio>

#define __device__
#define __forceinline__ inline

struct CUtensorMap {};
struct uint4 {
    uint32_t x, y, z, w;
};

static int phases, expected, copies, waits;  // completed phases; arrivals that wait for bytes; calls
static bool lands;                           // whether a copy in flight has landed when it is waited for

static void mbar_arrive_expect_tx(uint64_t*, uint32_t bytes)
{
    assert(bytes == 4096);
    assert(expected == 0);  // a second arrival in one phase
    expected = 1;
}
template <int CG>
static void copy_box(uint32_t, const CUtensorMap*, int, int, uint64_t*)
{
    ++copies;
}
static bool mbar_wait_bounded(uint64_t*, uint32_t parity, uint64_t)
{
    ++waits;
    if (expected && lands) {
        expected = 0;
        ++phases;
    }
    return static_cast<uint32_t>(phases & 1) != parity;
}
static bool __all_sync(unsigned, bool p) { return p; }
static void __syncwarp() {}
static void fence_proxy_async_smem() {}
static void bulk_wait_read() {}
static void bulk_commit() {}
static void store_box(const CUtensorMap*, int, int, uint32_t) {}
static uint4 ld_shared(uint32_t) { return {}; }
static void st_shared(uint32_t, uint32_t, uint32_t, uint32_t, uint32_t) {}

#include "dradd_staging.cuh"

static dradd::Staging fresh()
{
    static uint64_t bar;
    phases = expected = copies = waits = 0;
    lands = true;
    return {0, &bar, 1, 0, 0, false, false};
}

int main()
{
    const CUtensorMap map;
    {  // tile after tile, each waited for in its own phase
        dradd::Staging s = fresh();
        for (int i = 0; i < 5; ++i) {
            s.load(&map, 0, 0);
            assert(expected == 1);
            s.loaded();
            assert(!s.failed && phases == i + 1);
        }
        waits = 0;
        assert(s.drained() && waits == 0);
    }
    {  // the products of a tile never came: what was asked for is waited for
        dradd::Staging s = fresh();
        s.load(&map, 0, 0);
        s.loaded();
        s.load(&map, 0, 0);
        lands = false;
        assert(!s.drained());
        lands = true;
        assert(s.drained() && expected == 0);
    }
    {  // the copy itself was waited for in vain: nothing more is asked for, and it is waited for again
        dradd::Staging s = fresh();
        lands = false;
        s.load(&map, 0, 0);
        s.loaded();
        assert(s.failed);
        s.load(&map, 64, 0);
        waits = 0;
        s.loaded();
        assert(copies == 1 && waits == 0 && s.failed);
        assert(!s.drained());
        lands = true;
        assert(s.drained() && expected == 0);
    }
    {  // nothing ever came in
        dradd::Staging s = fresh();
        s.acquire(0);
        assert(s.drained() && waits == 0);
    }
    std::puts("ok");
}
