// dradd_linear_loss.cu -- products whose results are logits: their rows'
// statistics, and the gradients with respect to them.
#include "dradd_act.cuh"
#include "dradd_linear.cuh"

namespace dradd {

// The words of a row that count in a part of 128 columns: a target, or the
// entries of a teacher in rising order, the one after the next on its way.
struct Words {
    const Entry* entry = nullptr;  // the next one
    int left = 0;                  // from it on
    int next = kHalfCols;          // its column in the part; kHalfCols or more: not in it
    float weight = 1.0f;

    __device__ __forceinline__ void target(int64_t word, int64_t col)
    {
        const int64_t at = word - col;
        next = at >= 0 && at < kHalfCols ? static_cast<int>(at) : kHalfCols;
    }
    __device__ __forceinline__ void teacher(const Entry* e, int first, int top, int64_t col)
    {
        entry = e + first;
        left = top - first;
        base = static_cast<int>(col);
        if (left > 0)
            ahead = entry[0];
        take();
    }
    __device__ __forceinline__ void advance()
    {
        ++entry;
        --left;
        take();
    }

private:
    int base = 0;
    Entry ahead;
    // Entries are not below the part's first column, and INT_MAX less that is
    // behind the part's last.
    __device__ __forceinline__ void take()
    {
        next = kHalfCols;
        if (left > 0) {
            next = ahead.word - base;
            weight = ahead.share;
            if (left > 1)
                ahead = entry[1];
        }
    }
};

// A row's 128 logits of a warp, once their sums are whole: their maximum and
// the sum of 2^(z - maximum), in units that take the temperature and the
// exponential's base into one factor, and the logits of the row's words.
// loss_kernel joins the parts in order.  A NaN stays out of the maximum and
// enters the sum.
//
// Losses are differences of logits, so their sums are broken.  32768
// exponentials a tile and SM take 2048 cycles of the special function units,
// the products of 4096 terms 32768: bound by the products (4096 x 4096 over
// 128000 words 2350 to 2430 us, 1770 to 1830 TFLOP/s under the power limit).
struct EpiStats {
    using Kind = StatsProduct;
    using Params = StatsParams;
    static constexpr int kWarps = 8;
    static constexpr bool kStaged = false;
    static constexpr int kRun = kLogitRun;
    const Params& p;
    const int row, col;
    const int part;
    Words words;
    float high = -INFINITY, sum = 0.0f, picked = 0.0f;
    bool found = false;

    __device__ __forceinline__ EpiStats(const Params& p_, int, int row_, int col_, int, Staging&)
        : p(p_), row(row_), col(col_), part(col_ / kHalfCols)
    {
        if (row < p.rows) {
            if (p.top == 0)
                words.target(p.target[row], col);
            else
                words.teacher(p.entries + static_cast<int64_t>(row) * p.top,
                              p.first[static_cast<int64_t>(row) * p.parts + part], p.top, col);
        }
    }
    __device__ __forceinline__ void whole(const uint32_t (&bits)[kHalfCols / 16][16])
    {
        float z[kHalfCols];
#pragma unroll
        for (int j = 0; j < kHalfCols; ++j)
            z[j] = __uint_as_float(bits[j >> 4][j & 15]);
#pragma unroll
        for (int c = 0; c < kHalfCols; c += 16) {
            while (words.next < c + 16) {
                const int at = words.next - c;
                float v = 0.0f;
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    v = j == at ? z[c + j] : v;
                picked = p.top == 0 ? v : fmaf(words.weight, v, picked);
                found = true;
                words.advance();
            }
        }
        const int n = p.vocab - col;
        if (n < kHalfCols) {
#pragma unroll
            for (int j = 0; j < kHalfCols; ++j)
                z[j] = j < n ? z[j] : -INFINITY;
        }
        float m[8];
#pragma unroll
        for (int j = 0; j < kHalfCols; ++j)
            m[j & 7] = j < 8 ? z[j] : fmaxf(m[j & 7], z[j]);
#pragma unroll
        for (int d = 4; d > 0; d >>= 1)
#pragma unroll
            for (int j = 0; j < d; ++j)
                m[j] = fmaxf(m[j], m[j + d]);
        high = m[0] * p.scale;
        const float shift = high == -INFINITY ? 0.0f : high;
        float s[8] = {};
#pragma unroll
        for (int j = 0; j < kHalfCols; ++j)
            s[j & 7] += exp2_fast(fmaf(z[j], p.scale, -shift));
        sum = ((s[0] + s[1]) + (s[2] + s[3])) + ((s[4] + s[5]) + (s[6] + s[7]));
    }
    __device__ __forceinline__ void end()
    {
        if (row >= p.rows)
            return;
        const int64_t at = static_cast<int64_t>(part) * p.rows + row;
        p.part[at] = make_float2(high, sum);
        if (p.top != 0)
            p.picked[at] = picked;
        else if (found)
            p.picked[row] = picked;
    }
};

// dz = coef.x exp(z - lse) - coef.y share, rounded to the operands' type: the
// tensor cores multiply nothing wider at this rate.  The rounding of each
// element is independent of the others' (2^-9 of it in bf16), so it adds to dx
// and dweight about as much as their own rounding does.  What the logits are
// short by is the same for a whole row and does not average out, so their sums
// are broken as the forward's: logits of 100 from 8192 terms of one sign left
// dx off by 6.8e-3 without, 2.7e-4 with the breaks (fp16), for 1 % of the time
// (gradients of 4096 tokens x 4096 over 65536 words 3840 us and 3811).  Rows
// whose two factors are 0 are zeros whatever their logits are.
struct EpiSlope {
    using Kind = SlopeProduct;
    using Params = SlopeParams;
    static constexpr int kWarps = 8;
    static constexpr bool kStaged = true;
    static constexpr int kRun = kLogitRun;
    const Params& p;
    const bool bf16;
    const int row, col;
    Staging& staging;
    Words words;
    float lse2 = 0.0f;
    float2 coef = make_float2(0.0f, 0.0f);
    bool live = false;

    __device__ __forceinline__ EpiSlope(const Params& p_, int bf16_, int row_, int col_, int, Staging& staging_)
        : p(p_), bf16(bf16_), row(row_), col(col_), staging(staging_)
    {
        if (row < p.rows) {
            lse2 = p.lse[row] * kLog2e;
            coef = p.coef[row];
            live = coef.x != 0.0f || coef.y != 0.0f;
            const int64_t at = static_cast<int64_t>(p.col0) + col;
            if (p.top == 0)
                words.target(p.target[row], at);
            else
                words.teacher(p.entries + static_cast<int64_t>(row) * p.top,
                              p.first[static_cast<int64_t>(row) * p.parts + at / kHalfCols], p.top, at);
        }
    }
    __device__ __forceinline__ void columns(const uint32_t (&bits)[16], int c)
    {
        const int n = p.vocab - col - c;
        float v[16];
#pragma unroll
        for (int j = 0; j < 16; ++j)
            v[j] = coef.x * exp2_fast(fmaf(__uint_as_float(bits[j]), p.scale, -lse2));
        while (words.next < c + 16) {
            const int at = words.next - c;
            const float less = coef.y * words.weight;
#pragma unroll
            for (int j = 0; j < 16; ++j)
                v[j] = j == at ? v[j] - less : v[j];
            words.advance();
        }
        if (n < 16 || !live) {
#pragma unroll
            for (int j = 0; j < 16; ++j)
                v[j] = live && j < n ? v[j] : 0.0f;
        }
        uint32_t w[8];
        pack16(v, bf16, w);
        staging.acquire(c);
        staging.write(c, w);
        staging.store_full(&p.out_map, c, col, row & ~31, (row & ~31) < p.rows);
    }
    template <int N>
    __device__ __forceinline__ void whole(const uint32_t (&bits)[N][16])
    {
#pragma unroll
        for (int i = 0; i < N; ++i)
            columns(bits[i], i * 16);
    }
    __device__ __forceinline__ void end() {}
};

template <>
cudaError_t launch_product<StatsProduct>(const ProductArgs<StatsProduct>& a, int cta_group, int sm_count,
                                         cudaStream_t stream)
{
    return launch_with<EpiStats>(a, cta_group, sm_count, stream);
}

template <>
cudaError_t launch_product<SlopeProduct>(const ProductArgs<SlopeProduct>& a, int cta_group, int sm_count,
                                         cudaStream_t stream)
{
    return launch_with<EpiSlope>(a, cta_group, sm_count, stream);
}

}  // namespace dradd
