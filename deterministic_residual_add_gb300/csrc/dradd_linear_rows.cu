// dradd_linear_rows.cu -- the passes around the products of dradd_linear.h:
// finishing split sums, column sums, a teacher's entries in order, row
// factors, and the joining of row statistics.
#include <climits>

#include "dradd_act.cuh"
#include "dradd_elem.cuh"
#include "dradd_internal.h"
#include "dradd_linear_internal.h"

namespace dradd {

namespace {

__device__ __forceinline__ void widen8(const uint4& v, bool bf16, float (&f)[8])
{
    if (bf16)
        Elem<kElemBf16>::unpack(v, f);
    else
        Elem<kElemF16>::unpack(v, f);
}

__device__ __forceinline__ uint4 narrow8(const float (&f)[8], bool bf16)
{
    return bf16 ? Elem<kElemBf16>::pack(f) : Elem<kElemF16>::pack(f);
}

}  // namespace

// --------------------------------------------------------------- split sums
// A thread takes 8 columns of a row and adds the splits in order, four of
// them on their way at a time.
__global__ void __launch_bounds__(256) finish_kernel(const FinishParams p)
{
    wait_prior_grids();
    allow_next_grid();
    const int blocks = p.act.cols >> 3;
    const int64_t all = static_cast<int64_t>(p.act.rows) * blocks;
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (i >= all)
        return;
    const int64_t row = i / blocks;
    const int col = static_cast<int>(i - row * blocks) * 8;
    const bool bf16 = p.bf16;
    uint4 other = make_uint4(0, 0, 0, 0), bias = other;
    if (p.act.act >= 0) {
        if (p.act.other)
            other = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.act.other) +
                                                    row * p.act.other_stride + col);
        if (p.act.bias)
            bias = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.act.bias) + col);
    }
    const int64_t step = static_cast<int64_t>(p.act.rows) * p.act.cols;
    const float* from = p.partials + row * p.act.cols + col;
    float z[8] = {};
    for (int s = 0; s < p.splits; s += 4) {
        float4 v[4][2];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const bool in = s + j < p.splits;
            v[j][0] = in ? *reinterpret_cast<const float4*>(from + (s + j) * step) : make_float4(0, 0, 0, 0);
            v[j][1] = in ? *reinterpret_cast<const float4*>(from + (s + j) * step + 4) : make_float4(0, 0, 0, 0);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            z[0] += v[j][0].x;
            z[1] += v[j][0].y;
            z[2] += v[j][0].z;
            z[3] += v[j][0].w;
            z[4] += v[j][1].x;
            z[5] += v[j][1].y;
            z[6] += v[j][1].z;
            z[7] += v[j][1].w;
        }
    }
    uint16_t* out = static_cast<uint16_t*>(p.act.out) + row * p.act.out_stride + col;
    if (p.act.act < 0) {
        const float factor = p.factor ? *p.factor : 1.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            z[j] *= factor;
    } else {
        float b[8], o[8];
        widen8(bias, bf16, b);
        widen8(other, bf16, o);
        if (p.act.bias) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                z[j] += b[j];
        }
        if (p.grad) {
            act_slopes(z, p.act.act);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                z[j] *= o[j];
        } else {
            act_values(z, p.act.act);
            if (p.act.other) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    z[j] += o[j];
            }
        }
    }
    *reinterpret_cast<uint4*>(out) = narrow8(z, bf16);
}

cudaError_t launch_finish(const FinishParams& p, cudaStream_t stream)
{
    const int64_t all = static_cast<int64_t>(p.act.rows) * (p.act.cols >> 3);
    return launch(finish_kernel, static_cast<int>((all + 255) / 256), 256, 0, false, stream, p);
}

// -------------------------------------------------------------- column sums
// A CTA takes 256 columns and one part of the rows, a warp every eighth row.
__global__ void __launch_bounds__(256) row_sums_kernel(const uint16_t* x, int64_t stride, int rows, int cols, int bf16,
                                                       int each, float* partials, uint16_t* out)
{
    __shared__ float sums[8][256];
    wait_prior_grids();
    allow_next_grid();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int col = blockIdx.x * 256 + lane * 8;
    const int r1 = min(rows, (static_cast<int>(blockIdx.y) + 1) * each);
    float s[8] = {};
    if (col < cols) {
        for (int r = blockIdx.y * each + warp; r < r1; r += 32) {
            uint4 v[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                v[j] = r + 8 * j < r1 ? *reinterpret_cast<const uint4*>(x + (r + 8 * j) * stride + col)
                                      : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float f[8];
                widen8(v[j], bf16, f);
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    s[k] += f[k];
            }
        }
    }
#pragma unroll
    for (int k = 0; k < 8; ++k)
        sums[warp][lane * 8 + k] = s[k];
    __syncthreads();
    const int c = blockIdx.x * 256 + threadIdx.x;
    if (c < cols) {
        float t = 0.0f;
#pragma unroll
        for (int w = 0; w < 8; ++w)
            t += sums[w][threadIdx.x];
        if (out)
            out[c] = bf16 ? Elem<kElemBf16>::narrow(t) : Elem<kElemF16>::narrow(t);
        else
            partials[static_cast<int64_t>(blockIdx.y) * cols + c] = t;
    }
}

cudaError_t launch_row_sums(const void* x, int64_t stride, int rows, int cols, int bf16, int chunks, float* partials,
                            void* out, cudaStream_t stream)
{
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((cols + 255) / 256), static_cast<unsigned>(chunks));
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, row_sums_kernel, static_cast<const uint16_t*>(x), stride, rows, cols, bf16,
                              (rows + chunks - 1) / chunks, partials, static_cast<uint16_t*>(out));
}

// A CTA takes 32 columns, a lane each; its warps every 32nd part.
__global__ void __launch_bounds__(1024) bias_kernel(const float* partials, int parts, int cols, uint16_t* out, int bf16)
{
    __shared__ float sums[32][33];
    wait_prior_grids();
    allow_next_grid();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int col = blockIdx.x * 32 + lane;
    float s = 0.0f;
    if (col < cols) {
        for (int i = warp; i < parts; i += 128) {
            float v[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                v[j] = i + 32 * j < parts ? partials[static_cast<int64_t>(i + 32 * j) * cols + col] : 0.0f;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                s += v[j];
        }
    }
    sums[warp][lane] = s;
    __syncthreads();
    // warp w now holds column w of the CTA, one warp's sum a lane
    s = butterfly_sum(sums[lane][warp], 32);
    const int c = blockIdx.x * 32 + warp;
    if (lane == 0 && c < cols)
        out[c] = bf16 ? Elem<kElemBf16>::narrow(s) : Elem<kElemF16>::narrow(s);
}

cudaError_t launch_bias(const float* partials, int parts, int cols, void* out, int bf16, cudaStream_t stream)
{
    return launch(bias_kernel, (cols + 31) / 32, 1024, 0, false, stream, partials, parts, cols,
                  static_cast<uint16_t*>(out), bf16);
}

// ------------------------------------------------------------------ teacher
// A CTA puts one row's entries into the order of (word, place), computes
// their shares and where each part of 128 columns begins.  An entry's place is
// the number of those before it, counted against the words in shared memory,
// four to a load.
constexpr int kTeacherMost = 256;  // threads

__device__ __forceinline__ float teacher_logit(const TeacherParams& p, int64_t at)
{
    if (p.logits_type == kElemF32)
        return static_cast<const float*>(p.logits)[at];
    const uint16_t v = static_cast<const uint16_t*>(p.logits)[at];
    return p.logits_type == kElemBf16 ? Elem<kElemBf16>::widen(v) : Elem<kElemF16>::widen(v);
}

// size: top rounded up to fours.
__global__ void __launch_bounds__(kTeacherMost) teacher_kernel(const TeacherParams p, int size)
{
    extern __shared__ __align__(16) uint32_t words[];  // size, then the logits, the ordered words and their shares
    __shared__ float red[3][kTeacherMost / 32];
    __shared__ int bad, counted_entries;
    wait_prior_grids();
    allow_next_grid();
    constexpr uint32_t kNone = 0xFFFFFFFFu;
    float* logits = reinterpret_cast<float*>(words + size);
    uint32_t* ordered = words + 2 * size;
    float* shares = reinterpret_cast<float*>(words + 3 * size);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int threads = blockDim.x, warps = threads >> 5;
    const int64_t row = blockIdx.x;
    if (tid == 0)
        bad = counted_entries = 0;
    __syncthreads();
    float high = -INFINITY;
    for (int i = tid; i < size; i += threads) {
        uint32_t key = kNone;
        float v = -INFINITY;
        if (i < p.top) {
            const int64_t word = p.index[row * p.top + i];
            if (word >= p.vocab)
                bad = 1;
            if (word >= 0 && word < p.vocab) {
                v = teacher_logit(p, row * p.top + i) * p.inv_temperature;
                key = static_cast<uint32_t>(word);
                high = v > high || v != v ? v : high;  // a NaN stays
            }
        }
        words[i] = key;
        logits[i] = v;
    }
    high = warp_max_nan(high);
    if (lane == 0)
        red[0][warp] = high;
    __syncthreads();
    high = red[0][0];
    for (int w = 1; w < warps; ++w)
        high = red[0][w] > high || red[0][w] != red[0][w] ? red[0][w] : high;
    const bool nan_row = bad != 0;
    const bool counted = nan_row || high != -INFINITY;
    // the sum of a row's exponentials: each thread's in order, then lanes, then warps
    float sum = 0.0f, weighted = 0.0f;
    int own = 0;
    if (counted) {
        for (int i = tid; i < p.top; i += threads) {
            if (words[i] != kNone) {
                const float d = logits[i] - high;
                const float e = exp2_fast(d * kLog2e);
                sum += e;
                weighted += e > 0.0f ? e * d : e;  // a share of 0 has no entropy; NaN stays
                ++own;
            }
        }
    }
    sum = butterfly_sum(sum, 32);
    weighted = butterfly_sum(weighted, 32);
    own = __reduce_add_sync(0xffffffffu, own);
    if (lane == 0) {
        red[1][warp] = sum;
        red[2][warp] = weighted;
        atomicAdd(&counted_entries, own);  // whole numbers: any order
    }
    __syncthreads();
    sum = red[1][0];
    weighted = red[2][0];
    for (int w = 1; w < warps; ++w) {
        sum += red[1][w];
        weighted += red[2][w];
    }
    const int entries = nan_row ? 1 : counted_entries;
    const float nan = __int_as_float(0x7FC00000);
    if (nan_row) {
        if (tid == 0) {
            ordered[0] = 0;
            shares[0] = nan;
        }
    } else if (counted) {
        for (int i = tid; i < p.top; i += threads) {
            const uint32_t word = words[i];
            if (word == kNone)
                continue;
            const int block = i >> 2;
            int place = 0;
            for (int j = 0; j < size >> 2; ++j) {
                const uint4 w = reinterpret_cast<const uint4*>(words)[j];
                const uint32_t below = word + (j < block);  // the same word at an earlier place comes first
                place += (w.x < below) + (w.y < below) + (w.z < below) + (w.w < below);
            }
            for (int j = block << 2; j < i; ++j)
                place += words[j] == word;
            ordered[place] = word;
            shares[place] = exp2_fast((logits[i] - high) * kLog2e) / sum;
        }
    }
    __syncthreads();
    for (int i = tid; i < p.top; i += threads) {
        const bool in = i < entries;
        p.entries[row * p.top + i] = {in ? static_cast<int>(ordered[i]) : INT_MAX, in ? shares[i] : 0.0f};
    }
    if (p.entropy && tid == 0)
        p.entropy[row] = nan_row ? make_float2(nan, 1.0f) : make_float2(counted ? weighted / sum : 0.0f, sum);
    // the first entry at or behind each part's first column
    for (int g = tid; g < p.parts; g += threads) {
        const uint32_t from = static_cast<uint32_t>(g) * kHalfCols;
        int at = 0, hi = entries;
        while (at < hi) {
            const int mid = (at + hi) >> 1;
            if (ordered[mid] < from)
                at = mid + 1;
            else
                hi = mid;
        }
        p.first[row * p.parts + g] = static_cast<uint16_t>(at);
    }
}

cudaError_t launch_teacher(const TeacherParams& p, cudaStream_t stream)
{
    const int size = (p.top + 3) & ~3, threads = (p.top + 31) & ~31;
    return launch(teacher_kernel, p.rows, threads < kTeacherMost ? threads : kTeacherMost,
                  static_cast<size_t>(size) * 16, false, stream, p, size);
}

// --------------------------------------------- logits from partial sums
// A warp takes a row's part of 128 columns, a lane four neighbours.
template <bool GRAD, class P>
__global__ void __launch_bounds__(256) logits_kernel(const LogitParts l, const P p, uint16_t* out, int64_t stride,
                                                     int bf16)
{
    wait_prior_grids();
    allow_next_grid();
    const int lane = threadIdx.x & 31, part = blockIdx.x;
    const int row = blockIdx.y * 8 + (threadIdx.x >> 5);
    if (row >= p.rows)
        return;
    const int col = part * kHalfCols + lane * 4;
    const int n = p.vocab - col;  // of the lane's columns
    float v[4] = {};
    if (n > 0) {
        const float* from = l.partials + row * l.pitch + col;
        for (int s = 0; s < l.splits; ++s) {
            const float4 f = *reinterpret_cast<const float4*>(from + s * (l.pitch * p.rows));
            v[0] += f.x;
            v[1] += f.y;
            v[2] += f.z;
            v[3] += f.w;
        }
    }
    const Entry* entry = p.entries + static_cast<int64_t>(row) * p.top;
    const int first = p.top ? p.first[static_cast<int64_t>(row) * p.parts + part] : 0;
    if constexpr (!GRAD) {
        const auto value = [&](int at) {  // of a column of the part, in every lane
            const float x = (at & 3) == 0 ? v[0] : (at & 3) == 1 ? v[1] : (at & 3) == 2 ? v[2] : v[3];
            return __shfl_sync(0xffffffffu, x, at >> 2);
        };
        float picked = 0.0f;
        if (p.top == 0) {
            const int64_t at = p.target[row] - part * kHalfCols;
            if (at >= 0 && at < kHalfCols) {
                picked = value(static_cast<int>(at));
                if (lane == 0)
                    p.picked[row] = picked;
            }
        } else {
            for (int i = first; i < p.top; ++i) {
                const int at = entry[i].word - part * kHalfCols;
                if (at >= kHalfCols)
                    break;
                picked = fmaf(entry[i].share, value(at), picked);
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
            v[j] = j < n ? v[j] : -INFINITY;
        const float high = warp_max(fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3]))) * p.scale;
        const float shift = high == -INFINITY ? 0.0f : high;
        float s[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            s[j] = exp2_fast(fmaf(v[j], p.scale, -shift));
        const float sum = butterfly_sum((s[0] + s[1]) + (s[2] + s[3]), 32);
        if (lane == 0) {
            const int64_t at = static_cast<int64_t>(part) * p.rows + row;
            p.part[at] = make_float2(high, sum);
            if (p.top != 0)
                p.picked[at] = picked;
        }
    } else {
        const float lse2 = p.lse[row] * kLog2e;
        const float2 coef = p.coef[row];
        const bool live = coef.x != 0.0f || coef.y != 0.0f;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            v[j] = coef.x * exp2_fast(fmaf(v[j], p.scale, -lse2));
        const auto take = [&](int64_t at, float less) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                v[j] = at == lane * 4 + j ? v[j] - less : v[j];
        };
        if (p.top == 0) {
            take(p.target[row] - part * kHalfCols, coef.y);
        } else {
            for (int i = first; i < p.top; ++i) {
                const int at = entry[i].word - part * kHalfCols;
                if (at >= kHalfCols)
                    break;
                take(at, coef.y * entry[i].share);
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
            v[j] = live && j < n ? v[j] : 0.0f;
        *reinterpret_cast<uint2*>(out + row * stride + col) =
            bf16 ? make_uint2(pack_rne(v[0], v[1]), pack_rne(v[2], v[3]))
                 : make_uint2(Elem<kElemF16>::pack2(v[0], v[1]), Elem<kElemF16>::pack2(v[2], v[3]));
    }
}

template <bool GRAD, class P>
cudaError_t launch_logits(const LogitParts& l, const P& p, uint16_t* out, int64_t stride, int bf16, int parts,
                          cudaStream_t stream)
{
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(parts), static_cast<unsigned>((p.rows + 7) / 8));
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, logits_kernel<GRAD, P>, l, p, out, stride, bf16);
}

cudaError_t launch_stats(const LogitParts& l, const StatsParams& p, cudaStream_t stream)
{
    return launch_logits<false>(l, p, nullptr, 0, 0, p.parts, stream);
}

cudaError_t launch_slope(const LogitParts& l, const SlopeParams& p, void* out, int64_t stride, int bf16,
                         cudaStream_t stream)
{
    return launch_logits<true>(l, p, static_cast<uint16_t*>(out), stride, bf16, (p.vocab + kHalfCols - 1) / kHalfCols,
                               stream);
}

// --------------------------------------------------------- joined statistics
// A CTA takes 16 rows, a lane each of half warps that take every slices-th
// part; as many half warps, up to 64, as leave four parts each.
__global__ void __launch_bounds__(1024) loss_kernel(const LossParams p)
{
    __shared__ float highs[64][17], sums[64][17], picks[64][17];
    allow_next_grid();
    wait_prior_grids();
    const int lane = threadIdx.x & 15, warp = threadIdx.x >> 4, slices = static_cast<int>(blockDim.x) >> 4;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * 16 + lane;
    const bool teacher = p.top != 0;
    float high = -INFINITY, sum = 0.0f, picked = 0.0f;
    if (row < p.rows) {
        for (int g = warp; g < p.parts; g += 4 * slices) {
            float2 v[4];
            float k[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int64_t at = static_cast<int64_t>(g + slices * j) * p.rows + row;
                const bool in = g + slices * j < p.parts;
                v[j] = in ? p.part[at] : make_float2(-INFINITY, 0.0f);
                k[j] = in && teacher ? p.picked[at] : 0.0f;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float now = fmaxf(high, v[j].x), shift = now == -INFINITY ? 0.0f : now;
                sum = sum * exp2_fast(high - shift) + v[j].y * exp2_fast(v[j].x - shift);
                high = now;
                picked += k[j];
            }
        }
    }
    highs[warp][lane] = high;
    sums[warp][lane] = sum;
    picks[warp][lane] = picked;
    __syncthreads();
    if (warp != 0 || row >= p.rows)
        return;
    high = -INFINITY;
#pragma unroll 8
    for (int w = 0; w < slices; ++w)
        high = fmaxf(high, highs[w][lane]);
    const float shift = high == -INFINITY ? 0.0f : high;
    sum = 0.0f;
    picked = 0.0f;
#pragma unroll 8
    for (int w = 0; w < slices; ++w) {
        sum += sums[w][lane] * exp2_fast(highs[w][lane] - shift);
        picked += picks[w][lane];
    }
    p.lse[row] = (high + log2f(sum)) * kLn2;
    // A loss may be a small difference of large numbers: the highest logit
    // and the picked one are subtracted from one another, the product's
    // rounding with them, before anything else is added; and one logarithm
    // stands for the student's and the teacher's.
    const bool counted = teacher ? p.entries[row * p.top].word != INT_MAX : p.target[row] != p.ignore_index;
    if (!teacher && counted) {
        const int64_t target = p.target[row];
        picked = target >= 0 && target < p.vocab ? p.picked[row] : __int_as_float(0x7FC00000);
    }
    const float at = picked * p.scale, off = fmaf(picked, p.scale, -at);
    const float2 h = teacher ? p.entropy[row] : make_float2(0.0f, 1.0f);
    const float loss = h.x + kLn2 * ((high - at) + (log2f(sum / h.y) - off));
    p.loss[row] = counted ? loss : 0.0f;
}

cudaError_t launch_loss(const LossParams& p, cudaStream_t stream)
{
    int slices = 8;
    while (slices < 64 && 4 * slices < p.parts)
        slices *= 2;
    return launch(loss_kernel, (p.rows + 15) / 16, 16 * slices, 0, false, stream, p);
}

// -------------------------------------------------------------- row factors
__device__ __forceinline__ void row_factors(const CoefParams& p, int64_t row, float& loss, float& both)
{
    bool counted, valid = true;
    if (p.top == 0) {
        const int64_t target = p.target[row];
        counted = target != p.ignore_index;
        valid = target >= 0 && target < p.vocab;
    } else {
        counted = p.entries[row * p.top].word != INT_MAX;
    }
    loss = counted ? p.dloss[row * p.dloss_stride] : 0.0f;
    if (counted && !valid)
        loss = __int_as_float(0x7FC00000);
    both = loss + (p.dlse ? p.dlse[row * p.dlse_stride] : 0.0f);
}

// What dz is multiplied by before it is rounded to fp16, whose smallest
// numbers a mean over many tokens would fall below: the power of two that
// takes the largest factor of a row to between 2^13 and 2^14.  By a whole CTA,
// every thread gets it.
__device__ __forceinline__ int factor_exponent(const CoefParams& p, float* red)
{
    float most = 0.0f;
    for (int64_t r = threadIdx.x; r < p.rows; r += blockDim.x) {
        float loss, both;
        row_factors(p, r, loss, both);
        const float m = (fabsf(loss) + fabsf(both)) * p.inv_temperature;
        most = m < INFINITY ? fmaxf(most, m) : most;
    }
    most = warp_max(most);
    if ((threadIdx.x & 31) == 0)
        red[threadIdx.x >> 5] = most;
    __syncthreads();
    most = red[0];
    for (int w = 1; w < static_cast<int>(blockDim.x) >> 5; ++w)
        most = fmaxf(most, red[w]);
    int e = 0;
    if (most > 0.0f) {
        frexpf(most, &e);
        e = max(-100, min(100, 14 - e));
    }
    return e;
}

// Up to this many rows every CTA of coef_kernel finds the factor for itself,
// which costs less than a grid in front of it: gradients of 128, 511 and 1000
// tokens of 512 over 4000 words 22.5, 24.9 and 27.3 us, with that grid 24.6,
// 26.6 and 29.9.
constexpr int kFactorRows = 1024;

__global__ void __launch_bounds__(1024) factor_kernel(const CoefParams p)
{
    __shared__ float red[32];
    wait_prior_grids();
    allow_next_grid();
    const int e = factor_exponent(p, red);
    if (threadIdx.x == 0) {
        p.factor[0] = ldexpf(1.0f, e);
        p.factor[1] = ldexpf(1.0f, -e);
    }
}

// A warp a row.
__global__ void __launch_bounds__(256) coef_kernel(const CoefParams p)
{
    __shared__ float red[8];
    wait_prior_grids();
    allow_next_grid();
    float factor = 1.0f;
    if (p.factor && p.rows <= kFactorRows) {
        const int e = factor_exponent(p, red);
        factor = ldexpf(1.0f, e);
        if (blockIdx.x == 0 && threadIdx.x == 0) {
            p.factor[0] = factor;
            p.factor[1] = ldexpf(1.0f, -e);
        }
    } else if (p.factor) {
        factor = p.factor[0];
    }
    const int lane = threadIdx.x & 31;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    if (row >= p.rows)
        return;
    float loss, both;
    row_factors(p, row, loss, both);
    const float scale = factor * p.inv_temperature;
    loss *= scale;
    both *= scale;
    if (lane == 0)
        p.coef[row] = make_float2(both, loss);
    if (!p.x_live)
        return;
    const bool live = both != 0.0f || loss != 0.0f;
    const uint4* from = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.x) + row * p.x_stride);
    uint4* to = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.x_live) + row * p.inner);
    for (int i = lane; i < p.inner >> 3; i += 128) {
        uint4 v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            v[j] = live && i + 32 * j < p.inner >> 3 ? from[i + 32 * j] : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (i + 32 * j < p.inner >> 3)
                to[i + 32 * j] = v[j];
    }
}

cudaError_t launch_coef(const CoefParams& p, cudaStream_t stream)
{
    if (p.factor && p.rows > kFactorRows) {
        const cudaError_t e = launch(factor_kernel, 1, 1024, 0, false, stream, p);
        if (e != cudaSuccess)
            return e;
    }
    return launch(coef_kernel, (p.rows + 7) / 8, 256, 0, false, stream, p);
}

}  // namespace dradd
