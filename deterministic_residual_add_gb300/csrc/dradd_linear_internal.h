// dradd_linear_internal.h -- argument blocks and launchers of the matrix
// products of dradd_linear.h.  Not part of the public interface.
#pragma once

#include <cstddef>
#include <cstdint>

#include <cuda.h>
#include <cuda_runtime.h>

namespace dradd {

// Tiles: 128 rows a CTA (a pair of CTAs: 256) by 256 columns, summed in
// steps of 64.
constexpr int kTileRows = 128;
constexpr int kTileCols = 256;
constexpr int kTileDepth = 64;
constexpr int kHalfCols = kTileCols / 2;  // the columns of one epilogue warp

// A logit's sum is broken every so many steps (run_end): 512 terms, which the
// tensor cores leave short by up to 2e-6 of their size and 0.5e-6 as a rule.
// The relative errors of losses of 1024 tokens x 8192 over 32000 words, and of
// distillation from 64 words x 4096, against fp64: 2.1e-7 and 5.6e-7 (fp32 sums
// 6.8e-7 and 4.9e-7); with 16 steps 4.3e-7 and 1.1e-6, without breaks 1.9e-6
// and 5.1e-6.  The breaks cost power: 4096 x 4096 over 128000 words take 2365 us
// and 2279 without.
constexpr int kLogitRun = 8;

// n / d for 0 <= n < 2^31 by a multiplication: the quotient of the round-up
// method (Granlund and Montgomery, 1994), m = floor(2^32 (2^s - d) / d) + 1
// with s = ceil(log2 d).
struct Divisor {
    uint32_t m, s;
    int d;
    static Divisor of(int d)
    {
        Divisor r = {0, 0, d < 1 ? 1 : d};
        while ((1ull << r.s) < static_cast<uint64_t>(r.d))
            ++r.s;
        r.m = static_cast<uint32_t>((((1ull << r.s) - r.d) << 32) / r.d + 1);
        return r;
    }
#ifdef __CUDACC__
    __device__ __forceinline__ int divide(int n) const
    {
        return static_cast<int>((__umulhi(static_cast<uint32_t>(n), m) + static_cast<uint32_t>(n)) >> s);
    }
#endif
};

// One product C[m, n] = sum over k of A[m, k] B[n, k].
struct ProductShape {
    CUtensorMap a, b;
    int a_mn, b_mn;        // 1: the operand's rows in memory run along k
    int tiles_m, tiles_n;
    int k_blocks;          // steps of 64
    int splits;            // parts of the k dimension, each a tile of its own
    int band;              // tile rows that are walked down together
    Divisor per_split, per_band, in_band, in_last;  // tiles of a split, of a band, of a band's column
    int k_each;            // steps of a split
};

// ------------------------------------------------------------- epilogues
// A partial sum of a split, fp32 [splits, rows, cols].
struct SplitParams {
    float* partials;
    int rows, cols;
};

// out = residual + act(z + bias), or dz = dout * act'(z + bias)
struct ActParams {
    void* out;
    int64_t out_stride;
    const void* bias;      // or NULL
    const void* other;     // residual or NULL; the gradient: dout
    int64_t other_stride;
    int rows, cols;
    int act;
    float* col_sums;       // the gradient: [rows / 32, cols] sums of dz over 32 rows each, or NULL
};

struct ActProductParams {
    ActParams act;
    CUtensorMap out_map, other_map;  // 32 rows of 64 columns
};

// One of a teacher's words in a row and its share.
struct alignas(8) Entry {
    int word;
    float share;
};

// Statistics of the logits' rows, a part of 128 columns at a time.
struct StatsParams {
    float2* part;            // [parts, rows]: maximum and sum of 2^(z scale - maximum), in base-2 units
    float* picked;           // cross entropy: [rows], the target's logit; distillation: [parts, rows], sums of
                             // share * logit
    const int64_t* target;   // cross entropy
    const Entry* entries;    // distillation: [rows, top] words in rising order, INT_MAX behind the last
    const uint16_t* first;   // [rows, parts] the first entry at or behind a part's first column
    int parts;
    int rows, vocab, top;
    float scale;             // log2(e) / temperature
};

// dz = coef.x * p - coef.y * share, one piece of the vocabulary at a time.
struct SlopeParams {
    const float* lse;        // [rows]
    const float2* coef;      // [rows]
    const int64_t* target;
    const Entry* entries;
    const uint16_t* first;
    int parts;
    int rows, vocab, top;    // vocab: the piece's words
    int col0;                // its first one, a multiple of 256
    float scale;
    CUtensorMap out_map;
};

// out = rounded(sum * factor), or into fp32 partials [splits, rows, cols].
struct GradParams {
    CUtensorMap out_map;
    int to_out;              // 16-bit results; else partials
    float* partials;
    const float* factor;     // device, or NULL: 1
    int rows, cols;
    int add;
};

// What a launch does with its products, and how many it makes.
template <class P, int N, int Variant = 0>
struct ProductKind {
    using Params = P;
    static constexpr int kProblems = N;
};
using ActProduct = ProductKind<ActProductParams, 1, 0>;
using ActGradProduct = ProductKind<ActProductParams, 1, 1>;
using SplitProduct = ProductKind<SplitParams, 1, 0>;
using LogitSplitProduct = ProductKind<SplitParams, 1, 1>;  // of sums that are broken
using StatsProduct = ProductKind<StatsParams, 1>;
using SlopeProduct = ProductKind<SlopeParams, 1>;
using GradProducts = ProductKind<GradParams, 2>;

template <class K>
struct ProductArgs {
    ProductShape shape[K::kProblems];
    typename K::Params epi[K::kProblems];
    int tiles0, tiles;       // of the first problem, of all
    int worth;               // tiles of the second problem that cost as much as one of the first
    int rounds, odd;         // tiles0 / workers and its remainder (set with the launch)
    int prefetch;            // one CTA a tile and few rows: see product_kernel
    int early;               // the operands are complete when this grid may start (run_product says when); only
                             // the epilogue waits
    int bf16;
    unsigned* status;
    uint64_t wait_limit_ns;
};

// Sums of splits, finished: out = rounded(sum * factor), or with the
// activation's parameters as EpiAct (grad: EpiActGrad) does.
struct FinishParams {
    const float* partials;   // [splits, rows, cols]
    int splits;
    const float* factor;     // device, or NULL: 1
    ActParams act;           // act.act < 0: the plain sum
    int grad;
    int bf16;
};
cudaError_t launch_finish(const FinishParams& p, cudaStream_t stream);

// The product for a few rows, its epilogue with it.
struct FewParams {
    const void* x;
    int64_t x_stride;
    const void* weight;
    int64_t weight_stride;
    int inner;
    ActParams act;
    int bf16;
    unsigned* status;
    uint64_t wait_limit_ns;
};
constexpr int kFewRows = 16;
cudaError_t launch_few(const FewParams& p, cudaStream_t stream);

// What the epilogues of logits do, from partial sums [splits, rows, pitch].
struct LogitParts {
    const float* partials;
    int splits;
    int64_t pitch;           // a multiple of 8
};
cudaError_t launch_stats(const LogitParts& l, const StatsParams& p, cudaStream_t stream);
cudaError_t launch_slope(const LogitParts& l, const SlopeParams& p, void* out, int64_t stride, int bf16,
                         cudaStream_t stream);

// Column sums of fp32 [parts, cols], rounded.
cudaError_t launch_bias(const float* partials, int parts, int cols, void* out, int bf16, cudaStream_t stream);

// Sums of a 16-bit matrix's columns over `chunks` parts of its rows, fp32
// [chunks, cols]; with `out` (and one chunk) rounded to it.
cudaError_t launch_row_sums(const void* x, int64_t stride, int rows, int cols, int bf16, int chunks, float* partials,
                            void* out, cudaStream_t stream);

// A teacher's entries in rising order of their words.
struct TeacherParams {
    const int64_t* index;    // [rows, top]
    const void* logits;      // [rows, top]
    int logits_type;         // DRADD_*
    Entry* entries;          // [rows, top]
    float2* entropy;         // [rows] sum of e d / sum of e, and sum of e, with d = logit - the highest and e = exp(d);
                             // or NULL
    uint16_t* first;         // [rows, parts]
    int rows, top, vocab, parts;
    float inv_temperature;
};
cudaError_t launch_teacher(const TeacherParams& p, cudaStream_t stream);

// Row statistics joined: lse and loss.
struct LossParams {
    float* loss;
    float* lse;
    const float2* part;
    const float* picked;
    const int64_t* target;   // cross entropy
    int64_t ignore_index;
    const Entry* entries;    // distillation
    const float2* entropy;
    int rows, vocab, top, parts;
    float scale;             // log2(e) / temperature, as in StatsParams
};
cudaError_t launch_loss(const LossParams& p, cudaStream_t stream);

// A row's two factors, and x with the rows that count for nothing as zeros.
struct CoefParams {
    const float* dloss;
    int64_t dloss_stride;    // 0 or 1
    const float* dlse;       // or NULL
    int64_t dlse_stride;
    const int64_t* target;
    int64_t ignore_index;
    const Entry* entries;
    const void* x;
    int64_t x_stride;
    void* x_live;            // [rows, inner], or NULL
    float2* coef;
    float* factor;           // two numbers: what dz is scaled by, and its inverse; or NULL
    int rows, inner, vocab, top;
    float inv_temperature;
};
cudaError_t launch_coef(const CoefParams& p, cudaStream_t stream);

// Makes the map of a 16-bit matrix of `rows` rows of `cols` elements, `stride`
// apart, read in boxes of 64 elements by box_rows rows.
bool make_map(CUtensorMap* map, const void* base, int64_t rows, int64_t cols, int64_t stride, int box_rows);

template <class K>
cudaError_t launch_product(const ProductArgs<K>& a, int cta_group, int sm_count, cudaStream_t stream);

}  // namespace dradd
