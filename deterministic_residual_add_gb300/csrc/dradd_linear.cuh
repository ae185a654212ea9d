// dradd_linear.cuh -- the matrix product kernel of dradd_linear.h.
//
// C[m, n] = sum over k of A[m, k] B[n, k] in 16-bit operands and fp32 sums.
// A persistent grid of CTAs (CG = 1) or CTA pairs (CG = 2) walks the tiles.
// In a CTA one thread copies operands through a ring in shared memory, one
// thread (CG = 2: of the pair's first CTA) issues the products into one of
// two accumulators in tensor memory, and 8 or 16 warps turn the other one
// into the call's results, so that the epilogue runs beside the next tile's
// products.  What the epilogue does is the template's argument E, which sees
// 16 columns of a row at a time, the next ones already on their way.
//
// A pair of CTAs works on 256 x 256: each brings its own 128 rows of A and
// half of B, which halves what B's tile costs shared memory.  One CTA on 128
// x 256 has to move 192 bytes a cycle through it for the products to run at
// full rate, more than there are: 8192 x 4096 by 4096 took 190 us against 147.
// Single CTAs serve up to 128 rows, and gradients that they divide up better.
#pragma once

#include <atomic>

#include "dradd_elem.cuh"
#include "dradd_internal.h"
#include "dradd_linear_internal.h"
#include "dradd_mma.cuh"
#include "dradd_staging.cuh"
#include "dradd_train_internal.h"

namespace dradd {

// A copying warp, an issuing one, two spare, and those of the epilogue.
template <class E>
constexpr int kProductThreads = 128 + 32 * E::kWarps;
constexpr uint32_t kBoxBytes = 64 * 64 * 2;  // 64 rows of 128 bytes

__host__ __device__ constexpr uint32_t product_stage_bytes(int CG) { return (2u + 4u / CG) * kBoxBytes; }

// What 16-bit results take on their way out (and the residual, or the
// gradient that comes in, on its way in): a box of 32 rows and 64 columns for
// every warp of an epilogue that is `staged`.
//
// Such an epilogue comes in two forms.  Sums of at least kDeepSteps steps a
// tile leave it time, so 8 warps with two boxes of columns each do, and 32
// more KB go to the ring, a sixth stage for a pair of CTAs; short sums want
// 16 warps and leave five.  8192 x 4096 by 4096: 142.3 us with 8 warps, 147.4
// with 16 (the sixth stage alone is 4 us of 643 for 8192 x 16384 by 4096).
// 8192 x 512 by 8192 with silu: 94.5 us with 8 warps, 65.6 with 16.
constexpr int kDeepSteps = 32;
template <class E>
__host__ __device__ constexpr uint32_t staging_bytes()
{
    return E::kStaged ? E::kWarps * kStagingBox : 0;
}
template <int CG, class E>
__host__ __device__ constexpr int product_stages()
{
    return static_cast<int>((225u * 1024u - staging_bytes<E>()) / product_stage_bytes(CG));
}
template <int CG, class E>
constexpr uint32_t product_smem()
{
    return product_stages<CG, E>() * product_stage_bytes(CG) + staging_bytes<E>() + 1024u;
}

// Waits that have given up end every role's loop; the CTA then drains what
// it has in flight and returns.
struct ProductBars {
    uint64_t full[8], empty[8], acc_full[2], acc_empty[2], drain, loaded[16];
    uint32_t tmem;
};

struct TileAt {
    int problem, m, n, split, k0, k1;
};

// The i-th tile of a worker, or -1 behind its last.  The first problem's
// tiles go round the workers; where they do not come out even, the workers
// that got one less first take as many tiles of the second problem as one of
// the first is worth.
template <class K>
__device__ __forceinline__ int tile_of(const ProductArgs<K>& a, int worker, int workers, int i)
{
    int t = worker + i * workers;
    if constexpr (K::kProblems == 1)
        return t < a.tiles ? t : -1;
    if (t < a.tiles0)
        return t;
    const int odd = a.odd;
    i -= a.rounds + (worker < odd);
    t = worker + i * workers;
    if (odd > 0) {
        const int rest = workers - odd;
        if (worker >= odd) {
            t = i < a.worth ? worker - odd + i * rest : rest * a.worth + worker + (i - a.worth) * workers;
        } else {
            t += rest * a.worth;
        }
    }
    t += a.tiles0;
    return t < a.tiles ? t : -1;
}

// Tiles of one problem: splits outermost, then bands of tile rows that are
// walked down column by column, so that the tiles at work at one time share
// few rows and columns.
template <class K>
__device__ __forceinline__ TileAt tile_at(const ProductArgs<K>& a, int t)
{
    TileAt r;
    r.problem = K::kProblems > 1 && t >= a.tiles0 ? 1 : 0;
    if (r.problem)
        t -= a.tiles0;
    const ProductShape& s = a.shape[K::kProblems > 1 ? r.problem : 0];
    r.split = s.per_split.divide(t);
    t -= r.split * s.per_split.d;
    const int band = s.per_band.divide(t);
    t -= band * s.per_band.d;
    const bool last = (band + 1) * s.band > s.tiles_m;
    r.n = last ? s.in_last.divide(t) : s.in_band.divide(t);
    r.m = band * s.band + t - r.n * (last ? s.in_last.d : s.in_band.d);
    r.k0 = r.split * s.k_each;
    r.k1 = min(r.k0 + s.k_each, s.k_blocks);
    return r;
}

// Sums that are broken (E::kRun steps at most are added without a break): the
// tensor cores cut off what does not fit their fp32 sum instead of rounding
// it, so what they add up comes out short by about 1e-9 of its size a term.
// Where results are differences of such sums, to more digits than a 16-bit
// type has, a tile's sum is taken out of tensor memory in runs, and those are
// added with rounding in the registers of the epilogue: 128 columns a lane.
// These do not fit the 168 registers a thread that 12 warps share, so the four
// warps that need few hand theirs over.
constexpr int kOtherRegisters = 56, kSumRegisters = 224;
constexpr int kLaunchRegisters = 65536 / 384 / 8 * 8;
static_assert(128 * kOtherRegisters + 256 * kSumRegisters <= 384 * kLaunchRegisters,
              "the epilogue's warps would wait for registers that there are not");

// Steps of a sum that an epilogue's wait has its limit for.
constexpr int kWaitSteps = 1 << 18;

// Where the run of a tile's sum that begins at step k ends.
template <class E>
__device__ __forceinline__ int run_end(const TileAt& at, int k)
{
    return E::kRun > 0 && at.k1 - k > E::kRun ? k + E::kRun : at.k1;
}

// sums += v, fp32
__device__ __forceinline__ void add16(uint32_t (&sums)[16], const uint32_t (&v)[16])
{
#pragma unroll
    for (int j = 0; j < 16; j += 2) {
        float a, b;
        add2_rn(__uint_as_float(sums[j]), __uint_as_float(sums[j + 1]), __uint_as_float(v[j]),
                __uint_as_float(v[j + 1]), a, b);
        sums[j] = __float_as_uint(a);
        sums[j + 1] = __float_as_uint(b);
    }
}

template <int CG, class E>
__global__ void __launch_bounds__(kProductThreads<E>, 1)
    product_kernel(const __grid_constant__ ProductArgs<typename E::Kind> a)
{
    constexpr int kStages = product_stages<CG, E>();
    constexpr uint32_t kStageBytes = product_stage_bytes(CG);
    constexpr uint32_t kBytesA = 2 * kBoxBytes;
    constexpr int kRowsB = kTileCols / CG;
    extern __shared__ unsigned char smem_raw[];
    __shared__ ProductBars bars;
    const uint32_t ring = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = CG == 2 ? cluster_ctarank() : 0;
    const int worker = static_cast<int>(blockIdx.x) / CG, workers = static_cast<int>(gridDim.x) / CG;

    if (warp == 0 && lane == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&bars.full[i], 1);
            mbar_init(&bars.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars.acc_full[i], 1);
            mbar_init(&bars.acc_empty[i], E::kWarps * CG);
        }
        for (int i = 0; i < E::kWarps; ++i)
            mbar_init(&bars.loaded[i], 1);
        mbar_init(&bars.drain, 1);
        fence_mbar_init();
        for (int i = 0; i < E::Kind::kProblems && (i == 0 || a.tiles > a.tiles0); ++i) {
            prefetch_map(&a.shape[i].a);
            prefetch_map(&a.shape[i].b);
        }
    }
    if (warp == 2)
        tmem_alloc<CG>(&bars.tmem, 512);
    tmem_fence_before();
    __syncthreads();
    if constexpr (CG == 2)
        cluster_sync_all();
    tmem_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(&bars.tmem);
    if constexpr (CG == 1) {
        // Few rows: the second operand, the weights, is read once and its
        // bytes are what the product takes.  The first of them are asked into
        // L2 while the grid before ends: 12 steps a CTA, 60 MB in all.
        const int t = tile_of(a, worker, workers, 0);
        if (warp == 3 && lane == 0 && a.prefetch && t >= 0) {
            const TileAt at = tile_at(a, t);
            for (int k = at.k0; k < at.k1 && k < at.k0 + 12; ++k)
                prefetch_box(&a.shape[0].b, k * kTileDepth, at.n * kTileCols);
        }
    }
    allow_next_grid();
    if (!a.early || warp >= 4)
        wait_prior_grids();

    const auto wait = [&](uint64_t* bar, uint32_t parity) {
        if (mbar_wait_bounded(bar, parity, a.wait_limit_ns))
            return true;
        atomicOr(a.status, kDeviceStatusTimeout);
        return false;
    };

    const auto copy_operands = [&] {
        if (lane == 0) {
            int stage = 0;
            uint32_t phase = 0;
            bool ok = true;
            int64_t steps = 0;
            for (int i = 0, t; ok && (t = tile_of(a, worker, workers, i)) >= 0; ++i) {
                const TileAt at = tile_at(a, t);
                const ProductShape& s = a.shape[E::Kind::kProblems > 1 ? at.problem : 0];
                const int row = (at.m * CG + static_cast<int>(rank)) * kTileRows;
                const int col = at.n * kTileCols + static_cast<int>(rank) * kRowsB;
                for (int k = at.k0; k < at.k1; ++k) {
                    ok = wait(&bars.empty[stage], phase ^ 1u);
                    if (!ok)
                        break;
                    if (rank == 0)
                        mbar_arrive_expect_tx(&bars.full[stage], CG * kStageBytes);
                    const uint32_t to = ring + stage * kStageBytes;
                    uint64_t* bar = &bars.full[stage];
                    if (s.a_mn) {
#pragma unroll
                        for (int j = 0; j < kTileRows / 64; ++j)
                            copy_box<CG>(to + j * kBoxBytes, &s.a, row + j * 64, k * kTileDepth, bar);
                    } else {
                        copy_box<CG>(to, &s.a, k * kTileDepth, row, bar);
                    }
                    if (s.b_mn) {
#pragma unroll
                        for (int j = 0; j < kRowsB / 64; ++j)
                            copy_box<CG>(to + kBytesA + j * kBoxBytes, &s.b, col + j * 64, k * kTileDepth, bar);
                    } else {
                        copy_box<CG>(to + kBytesA, &s.b, k * kTileDepth, col, bar);
                    }
                    ++steps;
                    if (++stage == kStages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            // The last products have let go of every slot: nothing arrives
            // on this CTA's barriers after it has gone.
            for (int j = 0; ok && j < kStages && j < steps; ++j) {
                if (--stage < 0) {
                    stage = kStages - 1;
                    phase ^= 1u;
                }
                ok = wait(&bars.empty[stage], phase);
            }
            // Copies of this CTA (of the pair, where the barriers are) that
            // may still be in flight after a wait gave up.
            if (!ok && rank == 0) {
                for (int j = 0; j < kStages && j < steps; ++j) {
                    if (--stage < 0) {
                        stage = kStages - 1;
                        phase ^= 1u;
                    }
                    if (!mbar_wait_bounded(&bars.full[stage], phase, a.wait_limit_ns))
                        atomicOr(a.status, kDeviceStatusUndrained);
                }
            }
        }
    };
    // A whole warp, so that what one lane issues is known to be the same for
    // all: by a lone lane the four products of a step took 320 of its 512
    // cycles to issue, and every run's first waits stopped the tensor cores
    // (4096 x 4096 over 128000 words: 3838 k cycles, so 3532).
    const auto issue_products = [&] {
        if (rank == 0) {
            const bool chosen = elect_one();
            int stage = 0, acc = 0;
            uint32_t phase = 0, acc_phase = 0;
            bool ok = true;
            for (int i = 0, t; ok && (t = tile_of(a, worker, workers, i)) >= 0; ++i) {
                const TileAt at = tile_at(a, t);
                const ProductShape& s = a.shape[E::Kind::kProblems > 1 ? at.problem : 0];
                const uint32_t desc = product_desc(a.bf16, s.a_mn, s.b_mn, kTileRows * CG, kTileCols);
                // 16 of the summed dimension: 32 bytes along a row, or 16 rows
                const uint64_t step_a = s.a_mn ? 16 * 128 >> 4 : 32 >> 4, step_b = s.b_mn ? 16 * 128 >> 4 : 32 >> 4;
                for (int k0 = at.k0; ok && k0 < at.k1; k0 = run_end<E>(at, k0)) {
                    ok = __all_sync(0xffffffffu, wait(&bars.acc_empty[acc], acc_phase ^ 1u));
                    if (!ok)
                        break;
                    tmem_fence_after();
                    const uint32_t d = tmem + acc * kTileCols;
                    const int k1 = run_end<E>(at, k0);
                    for (int k = k0; k < k1; ++k) {
                        ok = __all_sync(0xffffffffu, wait(&bars.full[stage], phase));
                        if (!ok)
                            break;
                        tmem_fence_after();
                        const uint32_t from = ring + stage * kStageBytes;
                        const uint64_t da = operand_desc(from, kBoxBytes), db = operand_desc(from + kBytesA, kBoxBytes);
                        if (chosen) {
#pragma unroll
                            for (int j = 0; j < kTileDepth / 16; ++j)
                                mma_f16<CG>(d, da + j * step_a, db + j * step_b, desc, k > k0 || j > 0);
                            mma_commit<CG>(&bars.empty[stage]);
                        }
                        __syncwarp();
                        if (++stage == kStages) {
                            stage = 0;
                            phase ^= 1u;
                        }
                    }
                    if (!ok)
                        break;
                    if (chosen)
                        mma_commit<CG>(&bars.acc_full[acc]);
                    __syncwarp();
                    if (++acc == 2) {
                        acc = 0;
                        acc_phase ^= 1u;
                    }
                }
            }
            if (!ok && chosen) {
                mma_commit<CG>(&bars.drain);
                if (!mbar_wait_bounded(&bars.drain, 0, a.wait_limit_ns))
                    atomicOr(a.status, kDeviceStatusUndrained);
            }
        }
    };
    const auto finish_tiles = [&] {
        constexpr int kCols = kTileCols * 4 / E::kWarps;  // a warp's columns
        const int quadrant = warp & 3, part = (warp - 4) >> 2;
        int acc = 0;
        uint32_t acc_phase = 0;
        Staging staging = {ring + kStages * kStageBytes + (warp - 4) * kStagingBox,
                           &bars.loaded[warp - 4], a.wait_limit_ns, 0, lane, false, false};
        for (int i = 0, t; (t = tile_of(a, worker, workers, i)) >= 0; ++i) {
            const TileAt at = tile_at(a, t);
            const int row = (at.m * CG + static_cast<int>(rank)) * kTileRows + quadrant * 32 + lane;
            const int col = at.n * kTileCols + part * kCols;
            E epi(a.epi[E::Kind::kProblems > 1 ? at.problem : 0], a.bf16, row, col, at.split, staging);
            // The limit holds for every kWaitSteps of a sum: one over 2^28 rows
            // takes longer than a second.
            const auto arrived = [&](int steps) {
                bool ok = false;
                for (int s = 0; !ok && s < steps; s += kWaitSteps)
                    ok = mbar_wait_bounded(&bars.acc_full[acc], acc_phase, a.wait_limit_ns);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok && lane == 0)
                    atomicOr(a.status, kDeviceStatusTimeout);
                tmem_fence_after();
                return ok;
            };
            const auto let_go = [&] {
                tmem_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive_at(&bars.acc_empty[acc], 0);
            };
            const auto next_accumulator = [&] {
                if (++acc == 2) {
                    acc = 0;
                    acc_phase ^= 1u;
                }
            };
            const uint32_t own = tmem + (static_cast<uint32_t>(quadrant * 32) << 16) + part * kCols;
            uint32_t v0[16], v1[16];
            if constexpr (E::kRun > 0) {
                uint32_t sums[kCols / 16][16] = {};
                bool ok = true;
#pragma unroll 1
                for (int k = at.k0; k < at.k1; k = run_end<E>(at, k)) {
                    ok = arrived(E::kRun);
                    if (!ok)
                        break;
                    const uint32_t from = own + acc * kTileCols;
                    tmem_load16(from, v0);
#pragma unroll
                    for (int i = 0; i < kCols / 16; i += 2) {
                        tmem_wait(v0);
                        tmem_load16(from + i * 16 + 16, v1);
                        add16(sums[i], v0);
                        tmem_wait(v1);
                        if (i + 2 < kCols / 16)
                            tmem_load16(from + i * 16 + 32, v0);
                        else
                            let_go();
                        add16(sums[i + 1], v1);
                    }
                    next_accumulator();
                }
                if (!ok)
                    break;
                epi.whole(sums);
            } else {
                if (!arrived(at.k1 - at.k0))
                    break;
                const uint32_t from = own + acc * kTileCols;
                tmem_load16(from, v0);
#pragma unroll 1
                for (int c = 0; c < kCols; c += 32) {
                    tmem_wait(v0);
                    tmem_load16(from + c + 16, v1);
                    epi.columns(v0, c);
                    tmem_wait(v1);
                    if (c + 32 < kCols)
                        tmem_load16(from + c + 32, v0);
                    else
                        let_go();
                    epi.columns(v1, c + 16);
                }
                next_accumulator();
            }
            epi.end();
            if (staging.failed) {
                atomicOr(a.status, kDeviceStatusTimeout);
                break;
            }
        }
        if (E::kStaged) {
            if (!staging.drained() && lane == 0)
                atomicOr(a.status, kDeviceStatusUndrained);
            if (lane == 0)
                bulk_wait();
        }
    };
    if constexpr (E::kRun > 0) {
        if (warp < 4) {
            give_registers<kOtherRegisters>();
            if (warp == 0)
                copy_operands();
            else if (warp == 1)
                issue_products();
        } else {
            take_registers<kSumRegisters>();
            finish_tiles();
        }
    } else if (warp == 0) {
        copy_operands();
    } else if (warp == 1) {
        issue_products();
    } else if (warp >= 4) {
        finish_tiles();
    }
    tmem_fence_before();
    __syncthreads();
    if constexpr (CG == 2)
        cluster_sync_all();
    tmem_fence_after();
    if (warp == 2)
        tmem_free<CG>(tmem, 512);
}

template <int CG, class E>
cudaError_t launch_product_group(ProductArgs<typename E::Kind> a, int sm_count, cudaStream_t stream)
{
    constexpr auto fn = &product_kernel<CG, E>;
    cudaError_t e = allow_all_shared<product_kernel<CG, E>>();
    if (e != cudaSuccess)
        return e;
    if constexpr (E::kRun > 0) {
        static_assert(kProductThreads<E> == 384);
        // What the warps take is counted on the registers that the grid starts with.
        static std::atomic<int> registers{0};
        int r = registers.load(std::memory_order_acquire);
        if (r == 0) {
            cudaFuncAttributes attr;
            e = cudaFuncGetAttributes(&attr, reinterpret_cast<const void*>(fn));
            if (e != cudaSuccess)
                return e;
            registers.store(r = attr.numRegs, std::memory_order_release);
        }
        if (r != kLaunchRegisters)
            return cudaErrorInvalidConfiguration;
    }
    const int workers = a.tiles < sm_count / CG ? a.tiles : sm_count / CG;
    a.rounds = a.tiles0 / workers;
    a.odd = a.tiles0 % workers;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = CG;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(workers * CG));
    cfg.blockDim = dim3(kProductThreads<E>);
    cfg.dynamicSmemBytes = product_smem<CG, E>();
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, fn, a);
}

// Whether every tile's sum is long enough for the deep form of a staged epilogue.
template <class K>
bool long_sums(const ProductArgs<K>& a)
{
    for (int i = 0; i < K::kProblems; ++i)
        if ((i == 0 || a.tiles > a.tiles0) && a.shape[i].k_each < kDeepSteps)
            return false;
    return true;
}

template <class E>
cudaError_t launch_with(const ProductArgs<typename E::Kind>& a, int cta_group, int sm_count, cudaStream_t stream)
{
    return cta_group == 2 ? launch_product_group<2, E>(a, sm_count, stream)
                          : launch_product_group<1, E>(a, sm_count, stream);
}

// 16 values as eight pairs of a 16-bit type.
__device__ __forceinline__ void pack16(const float (&f)[16], bool bf16, uint32_t (&w)[8])
{
    if (bf16) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            w[i] = pack_rne(f[2 * i], f[2 * i + 1]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            w[i] = Elem<kElemF16>::pack2(f[2 * i], f[2 * i + 1]);
    }
}

__device__ __forceinline__ void store_sector(void* p, const uint32_t (&w)[8])
{
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}

__device__ __forceinline__ void unpack16(const uint32_t (&w)[8], bool bf16, float (&f)[16])
{
    if (bf16) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            f[2 * i] = bf16_lo(w[i]);
            f[2 * i + 1] = bf16_hi(w[i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            f[2 * i] = Elem<kElemF16>::widen(static_cast<uint16_t>(w[i] & 0xFFFFu));
            f[2 * i + 1] = Elem<kElemF16>::widen(static_cast<uint16_t>(w[i] >> 16));
        }
    }
}

__device__ __forceinline__ void prefetch_l1(const void* p)
{
    asm volatile("prefetch.global.L1 [%0];" ::"l"(p));
}

// 16 consecutive values of a 16-bit row, zeros past the n inside it.  An
// ordinary load: the grid in front may still write them when this one starts,
// so they are not read-only for its lifetime.
__device__ __forceinline__ void load16(const uint16_t* p, int n, uint32_t (&w)[8])
{
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        uint4 v = make_uint4(0, 0, 0, 0);
        if (8 * i < n)  // columns come in eights
            v = reinterpret_cast<const uint4*>(p)[i];
        w[4 * i] = v.x;
        w[4 * i + 1] = v.y;
        w[4 * i + 2] = v.z;
        w[4 * i + 3] = v.w;
    }
}

}  // namespace dradd
