// dradd_linear_abi.cu -- the C entry points of include/dradd_linear.h:
// argument checks, how a call is tiled and split, and its launches.  Every
// check is made before any GPU work.
#include <atomic>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "dradd_linear.h"

#include "dradd_host.h"
#include "dradd_internal.h"
#include "dradd_linear_internal.h"
#include "dradd_train_internal.h"

namespace dradd {

bool make_map(CUtensorMap* map, const void* base, int64_t rows, int64_t cols, int64_t stride, int box_rows)
{
    using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
    static std::atomic<void*> entry{nullptr};
    void* fn = entry.load(std::memory_order_acquire);
    if (!fn) {
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &found) !=
                cudaSuccess ||
            found != cudaDriverEntryPointSuccess || !fn)
            return false;
        entry.store(fn, std::memory_order_release);
    }
    const cuuint64_t sizes[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(stride) * 2};
    const cuuint32_t box[2] = {64, static_cast<cuuint32_t>(box_rows)};
    const cuuint32_t steps[2] = {1, 1};
    return reinterpret_cast<Encode>(fn)(map, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, const_cast<void*>(base), sizes, strides,
                                        box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

namespace {

constexpr int64_t kMaxInner = 1 << 24;
constexpr int64_t kMaxVocab = 1 << 30;
constexpr int64_t kMaxRows = 0x7FFFFFFF - 4095;  // a last tile's rows are still counted in 32 bits
constexpr int64_t kMaxTiles = 1 << 30;
constexpr int64_t kMaxTop = 1024;
// What plans count on, whatever device the call runs on: they decide the
// order of sums.
constexpr int kPlanSms = 152;

int64_t up(int64_t n, int64_t to) { return (n + to - 1) / to * to; }
int64_t parts_of(int64_t n, int64_t each) { return (n + each - 1) / each; }

// ------------------------------------------------------------------- plans
// A product of m x n with k summed: its tiles, pairs of CTAs from more than
// 128 rows on, and the parts that k is split into.
struct Plan {
    int group, tiles_m, tiles_n, k_blocks, splits;
    int64_t tiles() const { return static_cast<int64_t>(tiles_m) * tiles_n; }
    int64_t units() const { return tiles() * k_blocks; }
    void split(int64_t most_blocks, int most_splits)
    {
        int64_t s = parts_of(k_blocks, most_blocks < 1 ? 1 : most_blocks);
        s = s < most_splits ? s : most_splits;
        splits = static_cast<int>(parts_of(k_blocks, parts_of(k_blocks, s)));  // none empty
    }
};

Plan plan_of(int64_t m, int64_t n, int64_t k, int group)
{
    Plan p;
    p.group = group;
    p.tiles_m = static_cast<int>(parts_of(m, kTileRows * group));
    p.tiles_n = static_cast<int>(parts_of(n, kTileCols));
    p.k_blocks = static_cast<int>(parts_of(k, kTileDepth));
    p.splits = 1;
    return p;
}

int group_for(int64_t m) { return m <= kTileRows ? 1 : 2; }

constexpr int kLeastBlocks = 8;
constexpr int kMostSplits = 32;

// What a plan is thought to cost, in steps of one tile (256 x 256 x 64 by a
// pair or 128 x 256 x 64 by one CTA: 512 cycles): the steps of the busiest
// worker, kTileSteps more a tile, and for split sums the pass that finishes
// them, kFinishSteps and the time that its bytes take.
constexpr int64_t kTileSteps = 2;
constexpr int64_t kFinishSteps = 16;
int64_t finish_cost(const Plan& p, int64_t m, int64_t n)
{
    return p.splits > 1 ? kFinishSteps + p.splits * m * n * 8 / (3 << 20) : 0;
}

// The split of one product that runs alone.
void split_alone(Plan* p, int64_t m, int64_t n)
{
    const int64_t workers = kPlanSms / p->group;
    if (p->tiles() * 2 > workers)
        return;
    int64_t best = 0;
    Plan found = *p;
    for (int64_t s = 1; s <= workers / p->tiles() && s <= kMostSplits; ++s) {
        Plan t = *p;
        t.split(parts_of(t.k_blocks, s), kMostSplits);
        const int64_t each = parts_of(t.k_blocks, t.splits);
        if (s > 1 && each < kLeastBlocks)
            break;
        const int64_t cost = parts_of(t.tiles() * t.splits, workers) * (each + kTileSteps) + finish_cost(t, m, n);
        if (s == 1 || cost < best) {
            best = cost;
            found = t;
        }
    }
    *p = found;
}

// How tiles of the second of two products are worth those of the first, and
// the steps of the busiest worker, as tile_of deals them out.
int64_t worth_of(int64_t len0, int64_t len1) { return (len0 + len1 / 2) / len1; }

int64_t busiest(int64_t n0, int64_t len0, int64_t n1, int64_t len1, int64_t workers)
{
    const int64_t odd = n0 % workers, rest = odd ? workers - odd : 0, worth = n1 ? worth_of(len0, len1) : 0;
    int64_t most = 0;
    for (int64_t w = 0; w < workers; ++w) {
        const int64_t own = n0 / workers + (w < odd);
        int64_t more = 0;
        if (odd && w >= odd && n1 > w - odd) {
            const int64_t first = parts_of(n1 - (w - odd), rest);
            more = first < worth ? first : worth;
        }
        const int64_t left = n1 - rest * worth - w;
        more += left > 0 ? parts_of(left, workers) : 0;
        const int64_t steps = own * (len0 + kTileSteps) + more * (len1 + kTileSteps);
        most = steps > most ? steps : most;
    }
    return most;
}

// Two products m x n x k in one launch (either may be absent: no rows): by
// pairs of CTAs or by single ones, which cost a sixteenth more, and with how
// long tiles at most.
struct Size {
    int64_t m, n, k;
};
void plan_pair(const Size& a, const Size& b, bool split_b, Plan* p, Plan* q)
{
    int64_t best = -1;
    for (int group = 2; group >= 1; --group) {
        const int64_t workers = kPlanSms / group;
        const Plan p0 = plan_of(a.m, a.n, a.k, group), q0 = plan_of(b.m, b.n, b.k, group);
        const int64_t all = p0.units() + q0.units();
        int64_t before = 0;
        for (int part = 0; part <= 4; part = part ? part * 2 : 1) {
            Plan s = p0, t = q0;
            int64_t most = part ? all / (part * workers) : 1 << 30;
            most = most < kLeastBlocks ? kLeastBlocks : most;
            if (most == before)
                break;
            before = most;
            s.split(most, kMostSplits);
            if (split_b)
                t.split(most, kMostSplits);
            int64_t n0 = s.tiles() * s.splits, n1 = t.tiles() * t.splits;
            int64_t l0 = parts_of(s.k_blocks, s.splits), l1 = parts_of(t.k_blocks, t.splits);
            if (n0 == 0 || (n1 != 0 && l1 > l0)) {
                const int64_t x = n0, y = l0;
                n0 = n1, l0 = l1, n1 = x, l1 = y;
            }
            int64_t cost = busiest(n0, l0, n1, l1, workers);
            cost += group == 1 ? cost / 16 : 0;
            cost += finish_cost(s, a.m, a.n) + finish_cost(t, b.m, b.n);
            if (best < 0 || cost < best) {
                best = cost;
                *p = s;
                *q = t;
            }
        }
    }
}

int64_t partial_bytes(const Plan& p, int64_t m, int64_t n) { return p.splits > 1 ? p.splits * m * n * 4 : 0; }

// Parts of a call's workspace, each on 256 bytes.
struct Carver {
    char* base;
    int64_t used = 0;
    explicit Carver(void* p) : base(static_cast<char*>(p)) {}
    template <class T = void>
    T* take(int64_t bytes)
    {
        char* at = base ? base + used : nullptr;
        used += up(bytes, 256);
        return bytes ? reinterpret_cast<T*>(at) : nullptr;
    }
};

// ------------------------------------------------------------------ checks
bool dtype_ok(int dtype) { return dtype == DRADD_BF16 || dtype == DRADD_F16; }

View matrix_view(const void* p, int64_t rows, int64_t cols, int64_t stride, int64_t elem)
{
    View v;
    v.base = reinterpret_cast<uintptr_t>(p);
    v.elem = elem;
    v.add(rows, stride);
    v.add(cols, 1);
    return v;
}
View flat(const void* p, int64_t n, int64_t elem) { return matrix_view(p, 1, n, n, elem); }

struct Checks {
    View outs[4], ins[8];
    int n_out = 0, n_in = 0;
    bool exact_ok[8] = {};  // in: an output may be exactly this
    dradd_status st = DRADD_OK;

    void fail(dradd_status s)
    {
        if (st == DRADD_OK)
            st = s;
    }
    // A 16-bit matrix.
    void matrix(const dradd_matrix* m, int64_t rows, int64_t cols, bool out, bool exact = false)
    {
        if (!m || !m->data)
            return fail(DRADD_ERR_NULL_PTR);
        if (!aligned(m->data, 16) || (rows > 1 && m->stride % 8 != 0))
            return fail(DRADD_ERR_MISALIGNED);
        if (rows > 1 && m->stride < cols)
            return fail(DRADD_ERR_BAD_SHAPE);
        add(matrix_view(m->data, rows, cols, m->stride, 2), out, exact);
    }
    void buffer(const void* p, int64_t n, int64_t elem, int64_t align, bool out)
    {
        if (!p)
            return fail(DRADD_ERR_NULL_PTR);
        if (!aligned(p, align))
            return fail(DRADD_ERR_MISALIGNED);
        add(flat(p, n, elem), out, false);
    }
    void add(const View& v, bool out, bool exact)
    {
        if (!view_fits(v))
            return fail(DRADD_ERR_BAD_SHAPE);
        if (out) {
            outs[n_out++] = v;
        } else {
            exact_ok[n_in] = exact;
            ins[n_in++] = v;
        }
    }
    void workspace(void* p, size_t have, size_t need)
    {
        if (need == 0)
            return;
        if (!p || have < need)
            return fail(DRADD_ERR_WORKSPACE);
        buffer(p, static_cast<int64_t>(need), 1, 16, true);
    }
    dradd_status done()
    {
        if (st != DRADD_OK)
            return st;
        for (int i = 0; i < n_out; ++i) {
            for (int j = i + 1; j < n_out; ++j)
                if (views_may_overlap(outs[i], outs[j]))
                    return DRADD_ERR_ALIAS;
            for (int j = 0; j < n_in; ++j)
                if (!(exact_ok[j] && i == 0 && outs[i].same(ins[j])) && views_may_overlap(outs[i], ins[j]))
                    return DRADD_ERR_ALIAS;
        }
        return DRADD_OK;
    }
};

dradd_status inner_ok(int64_t n)
{
    if (n <= 0)
        return DRADD_ERR_BAD_SHAPE;
    return n % 8 != 0 || n >= kMaxInner ? DRADD_ERR_UNSUPPORTED_HIDDEN : DRADD_OK;
}

dradd_status from_cuda(cudaError_t e) { return e == cudaSuccess ? DRADD_OK : DRADD_ERR_CUDA; }

#define DRADD_TRY(call)            \
    do {                           \
        const dradd_status tried = (call); \
        if (tried != DRADD_OK)         \
            return tried;              \
    } while (0)

// ---------------------------------------------------------------- products
struct Side {  // an operand: a matrix in memory, its rows along k or not
    const void* data;
    int64_t rows, cols, stride;
    bool mn;
};

// A row stride for a matrix of one row, which a map wants to be a whole and
// sufficient number of bytes all the same.
int64_t map_stride(const Side& s) { return s.rows > 1 ? s.stride : up(s.cols, 8); }

// Tile rows in a band.  The first operand's rows of a band are read for every
// column of tiles, the second operand once a band; 8 rows make what 76 pairs
// share in one round smallest.  Where only statistics are written, a band of
// as many rows as L2 keeps (48 of its 126 MB) reads the second operand less
// often, and what DRAM need not bring leaves power to the products: 4096 x
// 4096 by 128000 words take 2475 us in bands of 8 rows and 2378 in one of 16
// (33 MB).  Products that write much gain nothing from it: 8192 x 16384 by
// 4096 683 us and 698, the gradients of 2048 tokens over 65536 words 2022 us
// in bands of 8 and 2107 in bands of 46.
constexpr int kBand = 8;
int wide_band(const Plan& p)
{
    const int64_t row_bytes = static_cast<int64_t>(p.k_blocks) * kTileDepth * 2 * kTileRows * p.group;
    const int64_t fit = (48ll << 20) / row_bytes;
    return static_cast<int>(fit < kBand ? kBand : fit < p.tiles_m ? fit : p.tiles_m);
}

dradd_status set_shape(ProductShape* s, const Plan& p, const Side& a, const Side& b, int band)
{
    s->a_mn = a.mn;
    s->b_mn = b.mn;
    s->tiles_m = p.tiles_m;
    s->tiles_n = p.tiles_n;
    s->k_blocks = p.k_blocks;
    s->splits = p.splits;
    s->band = band < p.tiles_m ? band : p.tiles_m;
    s->per_split = Divisor::of(p.tiles_m * p.tiles_n);
    s->per_band = Divisor::of(s->band * p.tiles_n);
    s->in_band = Divisor::of(s->band);
    s->in_last = Divisor::of(p.tiles_m % s->band ? p.tiles_m % s->band : s->band);
    s->k_each = static_cast<int>(parts_of(p.k_blocks, p.splits));
    const bool ok = make_map(&s->a, a.data, a.rows, a.cols, map_stride(a), a.mn ? 64 : kTileRows) &&
                    make_map(&s->b, b.data, b.rows, b.cols, map_stride(b), b.mn ? 64 : kTileCols / p.group);
    return ok ? DRADD_OK : DRADD_ERR_CUDA;
}

// The map that an epilogue's boxes of 32 rows and 64 columns leave through,
// or come in.
dradd_status staging_map(CUtensorMap* map, const void* p, int64_t rows, int64_t cols, int64_t stride)
{
    return make_map(map, p, rows, cols, rows > 1 ? stride : up(cols, 8), 32) ? DRADD_OK : DRADD_ERR_CUDA;
}

template <class K>
dradd_status start(ProductArgs<K>* a, int dtype, int* sms)
{
    DeviceLimits L;
    DRADD_TRY(query_limits(&L));
    *sms = L.sm_count;
    a->bf16 = dtype == DRADD_BF16;
    a->wait_limit_ns = kDefaultWaitLimitNs;
    return from_cuda(device_status_ptr(&a->status));
}

// A product may be `early`, its operands read while the grid in front of it
// runs, in two cases.  The operands are the caller's, which no grid of the call
// writes, and some grid of this call waited for every grid before itself
// before it let its successor start (the teacher's, the row factors'): all
// that come behind that one start when the caller's tensors are complete,
// whatever the grid directly in front does.  Or the grid directly in front did
// so, and what wrote the operands came before it (the bias's, behind dz).
// Products themselves let their successor start before they wait.
template <class K>
dradd_status run_product(const Plan& p, const Side& a, const Side& b, const typename K::Params& epi, bool early,
                         int dtype, cudaStream_t stream)
{
    static_assert(sizeof(ProductArgs<K>) <= 4096, "kernel parameters");
    ProductArgs<K> args = {};
    int sms = 0;
    DRADD_TRY(start(&args, dtype, &sms));
    DRADD_TRY(set_shape(&args.shape[0], p, a, b, std::is_same<K, StatsProduct>::value ? wide_band(p) : kBand));
    args.epi[0] = epi;
    args.early = early;
    args.prefetch = p.tiles_m == 1 && !b.mn;
    const int64_t tiles = p.tiles() * p.splits;
    args.tiles0 = args.tiles = static_cast<int>(tiles);
    return from_cuda(launch_product<K>(args, p.group, sms, stream));
}

// Two products whose results are gradients, the longer tiles first.
struct GradProduct {
    Plan plan;
    Side a, b;
    GradParams epi;
    bool on;
};

dradd_status grad_params(GradParams* p, void* out, float* partials, const float* factor, int64_t rows, int64_t cols,
                         bool add)
{
    *p = {};
    p->to_out = out != nullptr;
    p->partials = partials;
    p->factor = factor;
    p->rows = static_cast<int>(rows);
    p->cols = static_cast<int>(cols);
    p->add = add;
    return out ? staging_map(&p->out_map, out, rows, cols, cols) : DRADD_OK;
}

dradd_status run_gradients(GradProduct p, GradProduct q, bool early, int dtype, cudaStream_t stream)
{
    if (!p.on && !q.on)
        return DRADD_OK;
    const auto blocks = [](const GradProduct& g) { return parts_of(g.plan.k_blocks, g.plan.splits); };
    if (!p.on || (q.on && blocks(q) > blocks(p))) {
        const GradProduct t = p;
        p = q;
        q = t;
    }
    ProductArgs<GradProducts> args = {};
    int sms = 0;
    DRADD_TRY(start(&args, dtype, &sms));
    DRADD_TRY(set_shape(&args.shape[0], p.plan, p.a, p.b, kBand));
    args.epi[0] = p.epi;
    args.early = early;
    args.tiles0 = args.tiles = static_cast<int>(p.plan.tiles() * p.plan.splits);
    if (q.on) {
        DRADD_TRY(set_shape(&args.shape[1], q.plan, q.a, q.b, kBand));
        args.epi[1] = q.epi;
        args.tiles += static_cast<int>(q.plan.tiles() * q.plan.splits);
        args.worth = static_cast<int>(worth_of(blocks(p), blocks(q)));
    }
    return from_cuda(launch_product<GradProducts>(args, p.plan.group, sms, stream));
}

dradd_status finish_sums(const float* partials, int splits, int64_t rows, int64_t cols, void* out, const float* factor,
                         int dtype, cudaStream_t stream)
{
    FinishParams f = {};
    f.partials = partials;
    f.splits = splits;
    f.factor = factor;
    f.act.out = out;
    f.act.out_stride = cols;
    f.act.rows = static_cast<int>(rows);
    f.act.cols = static_cast<int>(cols);
    f.act.act = -1;
    f.bf16 = dtype == DRADD_BF16;
    return from_cuda(launch_finish(f, stream));
}

// ------------------------------------------------------- linear_act_add
Plan forward_plan(int64_t rows, int64_t inner, int64_t cols)
{
    Plan p = plan_of(rows, cols, inner, group_for(rows));
    split_alone(&p, rows, cols);
    return p;
}

// Whether the few rows' own kernel takes a product.  A CTA of it has 8 columns
// (from 9 rows on 16), three (two) of them share an SM, and a wave of them
// takes 2 us however short the rows of W are, from 9 rows on 2.5 us for every
// 1024 of them.  Times in us, that kernel's and the tiles':
//   up to 8 rows, as many columns as 16 times the inner dimension pay off,
//   from 1024 of it on, where tiles are split, 24 times (256 -> 4096 4.3 and
//   6.0, -> 8192 6.4 and 6.0; 512 -> 8192 6.4 and 7.4, -> 16384 10.9 and 8.2;
//   1024 -> 22000 14.6 and 18.9; 1136 -> 22000 19.2 and 21.9, -> 29528 25.0 and
//   22.2), rows of W up to 8192 (8192 -> 6144 20.4 and 23.0, 10240 -> 4096
//   23.7 and 20.4 for 8 rows), and some 50 million weights (7168 -> 7168 21.0
//   and 24.1 for 8 rows, 8192 -> 8192 30.1 and 27.5);
//   9 to 16 rows, while the waves are short together (4096 -> 4096 10.7 and
//   11.3, -> 5120 in two waves 19.5 and 16.2; 5120 -> 4096 12.8 and 15.5;
//   1024 -> 14592 10.6 and 13.0; 8192 -> 2048 20.4 and 13.6) and few (512 ->
//   14592 in three 8.1 and 8.1, -> 32768 in seven 18.3 and 10.9).
bool few(int64_t rows, int64_t inner, int64_t cols)
{
    if (rows <= 8)
        return (cols <= (inner < 1024 ? 16 : 24) * inner || cols <= 3 * kPlanSms * 8) && inner <= 8192 &&
               inner * cols <= 13 << 22;
    const int64_t waves = parts_of(cols, 2 * kPlanSms * 16);
    return rows <= kFewRows && waves <= 3 && waves * inner <= 5120;
}

dradd_status linear_shape(int64_t rows, int64_t inner, int64_t cols)
{
    if (rows < 0 || rows > kMaxRows)
        return DRADD_ERR_BAD_SHAPE;
    DRADD_TRY(inner_ok(inner));
    DRADD_TRY(inner_ok(cols));
    // tiles of every product below are counted in 32 bits
    const int64_t most = parts_of(inner > cols ? inner : cols, kTileCols);
    return parts_of(rows > cols ? rows : cols, kTileRows) * most * kMostSplits > kMaxTiles ? DRADD_ERR_BAD_SHAPE
                                                                                          : DRADD_OK;
}

struct LinearGradPlan {
    Plan z, dx, dw;
    bool sums;
    int chunks;
    int64_t dz, partial_z, partial_dx, partial_dw, partial_db;
    int64_t bytes;
};

LinearGradPlan linear_grad_plan(int64_t rows, int64_t inner, int64_t cols, int act, bool want_dx, bool want_dw,
                                bool want_db)
{
    LinearGradPlan g = {};
    g.z = forward_plan(rows, inner, cols);
    plan_pair({want_dx ? rows : 0, inner, cols}, {want_dw ? cols : 0, inner, rows}, true, &g.dx, &g.dw);
    const int64_t c = parts_of(rows, 64);
    // with an activation and whole sums dz's product adds its columns up itself
    g.sums = act != DRADD_ACT_NONE && g.z.splits == 1;
    g.chunks = static_cast<int>(g.sums ? parts_of(rows, 32) : c < 64 ? c : 64);
    g.dz = act == DRADD_ACT_NONE ? 0 : rows * cols * 2;
    g.partial_z = act == DRADD_ACT_NONE ? 0 : partial_bytes(g.z, rows, cols);
    g.partial_dx = want_dx ? partial_bytes(g.dx, rows, inner) : 0;
    g.partial_dw = want_dw ? partial_bytes(g.dw, cols, inner) : 0;
    g.partial_db = want_db ? static_cast<int64_t>(g.chunks) * cols * 4 : 0;
    Carver c0(nullptr);
    for (const int64_t n : {g.dz, g.partial_z, g.partial_dx, g.partial_dw, g.partial_db})
        c0.take(n);
    g.bytes = c0.used;
    return g;
}

ActParams act_params(void* out, int64_t out_stride, const void* bias, const void* other, int64_t other_stride,
                     int64_t rows, int64_t cols, int act)
{
    return {out, out_stride, bias, other, other_stride, static_cast<int>(rows), static_cast<int>(cols), act,
            nullptr};
}

// out = residual + act(x W^T + bias), or with `grad` dz; by one product, or
// by split ones and their finish.
dradd_status run_linear(const Plan& p, const dradd_matrix& x, const dradd_matrix& w, const ActParams& act, bool grad,
                        int64_t inner, float* partials, int dtype, cudaStream_t stream)
{
    const Side a = {x.data, act.rows, inner, x.stride, false}, b = {w.data, act.cols, inner, w.stride, false};
    if (p.splits == 1) {
        ActProductParams e = {};
        e.act = act;
        DRADD_TRY(staging_map(&e.out_map, act.out, act.rows, act.cols, act.out_stride));
        if (act.other)
            DRADD_TRY(staging_map(&e.other_map, act.other, act.rows, act.cols, act.other_stride));
        return grad ? run_product<ActGradProduct>(p, a, b, e, false, dtype, stream)
                    : run_product<ActProduct>(p, a, b, e, false, dtype, stream);
    }
    const SplitParams s = {partials, act.rows, act.cols};
    DRADD_TRY(run_product<SplitProduct>(p, a, b, s, false, dtype, stream));
    FinishParams f = {partials, p.splits, nullptr, act, grad, dtype == DRADD_BF16};
    return from_cuda(launch_finish(f, stream));
}

// --------------------------------------------------------------- the losses
// A loss's words: a target a row, or a teacher's entries.
struct LossCall {
    const int64_t* target;
    int64_t ignore_index;
    const dradd_teacher* teacher;
    int64_t rows, hidden, vocab;
    int64_t top() const { return teacher ? teacher->top : 0; }
    float inv_temperature() const { return teacher ? 1.0f / teacher->temperature : 1.0f; }
};

dradd_status loss_shape(const LossCall& c, int dtype)
{
    if (!dtype_ok(dtype))
        return DRADD_ERR_BAD_ARG;
    if (c.teacher) {
        const dradd_teacher& t = *c.teacher;
        if (t.logits_dtype != DRADD_BF16 && t.logits_dtype != DRADD_F16 && t.logits_dtype != DRADD_F32)
            return DRADD_ERR_BAD_ARG;
        if (!std::isfinite(t.temperature) || !(t.temperature > 0.0f) || !std::isfinite(1.0f / t.temperature))
            return DRADD_ERR_BAD_ARG;
        if (t.top < 1 || t.top > kMaxTop)
            return DRADD_ERR_BAD_SHAPE;
    }
    if (c.rows < 0 || c.rows > kMaxRows || c.vocab < 1 || c.vocab > kMaxVocab)
        return DRADD_ERR_BAD_SHAPE;
    DRADD_TRY(inner_ok(c.hidden));
    const int64_t tr = parts_of(c.rows, kTileRows), tv = parts_of(c.vocab, kTileRows),
                  th = parts_of(c.hidden, kTileCols);
    if (tr * parts_of(c.vocab, kTileCols) > kMaxTiles || (tr + tv) * th * kMostSplits > kMaxTiles)
        return DRADD_ERR_BAD_SHAPE;
    return DRADD_OK;
}

void loss_inputs(Checks* k, const LossCall& c, const dradd_matrix* x, const dradd_matrix* w)
{
    k->matrix(x, c.rows, c.hidden, false);
    k->matrix(w, c.vocab, c.hidden, false);
    if (c.teacher) {
        const int64_t eb = c.teacher->logits_dtype == DRADD_F32 ? 4 : 2;
        k->buffer(c.teacher->index, c.rows * c.teacher->top, 8, 8, false);
        k->buffer(c.teacher->logits, c.rows * c.teacher->top, eb, eb, false);
    } else {
        k->buffer(c.target, c.rows, 8, 8, false);
    }
}

// The workspace of a teacher's entries.
struct TeacherSpace {
    Entry* entries;
    float2* entropy;
    uint16_t* first;
    int parts;

    TeacherSpace(Carver* w, int64_t rows, int64_t vocab, int64_t top, bool with_entropy)
    {
        parts = static_cast<int>(2 * parts_of(vocab, kTileCols));
        entries = w->take<Entry>(rows * top * 8);
        entropy = w->take<float2>(top && with_entropy ? rows * 8 : 0);
        first = w->take<uint16_t>(top ? rows * parts * 2 : 0);
    }
    cudaError_t run(const LossCall& c, cudaStream_t stream) const
    {
        TeacherParams p = {};
        p.index = c.teacher->index;
        p.logits = c.teacher->logits;
        p.logits_type = c.teacher->logits_dtype;
        p.entries = entries;
        p.entropy = entropy;
        p.first = first;
        p.rows = static_cast<int>(c.rows);
        p.top = static_cast<int>(c.teacher->top);
        p.vocab = static_cast<int>(c.vocab);
        p.parts = parts;
        p.inv_temperature = c.inv_temperature();
        return launch_teacher(p, stream);
    }
};

// The product that makes a loss's logits: where its tiles do not fill the
// device it is split, and the logits of these few rows or few words are
// summed up in the workspace.
Plan logit_plan(int64_t rows, int64_t hidden, int64_t words)
{
    Plan p = plan_of(rows, words, hidden, group_for(rows));
    split_alone(&p, rows, words);
    return p;
}

int64_t logit_bytes(const Plan& p, int64_t rows, int64_t words) { return partial_bytes(p, rows, up(words, 8)); }

struct LossForwardSpace {
    TeacherSpace teacher;
    float2* part;
    float* picked;
    float* partials;

    LossForwardSpace(Carver* w, int64_t rows, int64_t hidden, int64_t vocab, int64_t top)
        : teacher(w, rows, vocab, top, true)
    {
        partials = w->take<float>(logit_bytes(logit_plan(rows, hidden, vocab), rows, vocab));
        part = w->take<float2>(teacher.parts * rows * 8);
        picked = w->take<float>((top ? teacher.parts : 1) * rows * 4);
    }
};

float logit_scale(float inv_temperature) { return static_cast<float>(1.4426950408889634 * inv_temperature); }

dradd_status run_logits(const Plan& p, const Side& x, const Side& w, float* partials, bool early, int dtype,
                        cudaStream_t stream)
{
    const SplitParams e = {partials, static_cast<int>(x.rows), static_cast<int>(up(w.rows, 8))};
    return run_product<LogitSplitProduct>(p, x, w, e, early, dtype, stream);
}

size_t loss_fwd_bytes(int64_t rows, int64_t hidden, int64_t vocab, int64_t top)
{
    Carver w(nullptr);
    LossForwardSpace s(&w, rows, hidden, vocab, top);
    return static_cast<size_t>(w.used);
}

dradd_status loss_fwd(float* loss, float* lse, const dradd_matrix* x, const dradd_matrix* weight, const LossCall& c,
                      int dtype, void* workspace, size_t workspace_bytes, cudaStream_t stream)
{
    DRADD_TRY(loss_shape(c, dtype));
    if (c.rows == 0)
        return DRADD_OK;
    Checks k;
    k.buffer(loss, c.rows, 4, 4, true);
    k.buffer(lse, c.rows, 4, 4, true);
    loss_inputs(&k, c, x, weight);
    k.workspace(workspace, workspace_bytes, loss_fwd_bytes(c.rows, c.hidden, c.vocab, c.top()));
    DRADD_TRY(k.done());
    Carver w(workspace);
    const LossForwardSpace s(&w, c.rows, c.hidden, c.vocab, c.top());
    const Plan p = logit_plan(c.rows, c.hidden, c.vocab);
    const Side sx = {x->data, c.rows, c.hidden, x->stride, false},
               sw = {weight->data, c.vocab, c.hidden, weight->stride, false};
    if (c.teacher)
        DRADD_TRY(from_cuda(s.teacher.run(c, stream)));
    StatsParams e = {};
    e.part = s.part;
    e.picked = s.picked;
    e.target = c.target;
    e.entries = s.teacher.entries;
    e.first = s.teacher.first;
    e.parts = s.teacher.parts;
    e.rows = static_cast<int>(c.rows);
    e.vocab = static_cast<int>(c.vocab);
    e.top = static_cast<int>(c.top());
    e.scale = logit_scale(c.inv_temperature());
    if (p.splits == 1) {
        DRADD_TRY(run_product<StatsProduct>(p, sx, sw, e, c.teacher != nullptr, dtype, stream));
    } else {
        DRADD_TRY(run_logits(p, sx, sw, s.partials, c.teacher != nullptr, dtype, stream));
        DRADD_TRY(from_cuda(launch_stats({s.partials, p.splits, up(c.vocab, 8)}, e, stream)));
    }
    LossParams l = {};
    l.loss = loss;
    l.lse = lse;
    l.part = s.part;
    l.picked = s.picked;
    l.target = c.target;
    l.ignore_index = c.ignore_index;
    l.entries = s.teacher.entries;
    l.entropy = s.teacher.entropy;
    l.rows = e.rows;
    l.vocab = e.vocab;
    l.top = e.top;
    l.parts = s.teacher.parts;
    l.scale = e.scale;
    return from_cuda(launch_loss(l, stream));
}

// The gradients take the vocabulary in pieces whose dz fills at most
// kPieceBytes (and at least one column of tiles).
constexpr int64_t kPieceBytes = 256ll << 20;

struct LossGradPlan {
    int64_t piece, pieces;
    Plan z, dx, dw;  // of a whole piece; the last may be smaller
};

LossGradPlan loss_grad_plan(int64_t rows, int64_t hidden, int64_t vocab)
{
    LossGradPlan g = {};
    const int64_t whole = up(vocab, kTileCols);
    int64_t most = kPieceBytes / (2 * rows) / kTileCols * kTileCols;
    most = most < kTileCols ? kTileCols : most;
    g.pieces = parts_of(whole, most);
    g.piece = up(parts_of(whole, g.pieces), kTileCols);  // of about one size
    g.pieces = parts_of(whole, g.piece);
    const int64_t width = g.pieces == 1 ? vocab : g.piece;
    g.z = g.pieces == 1 ? logit_plan(rows, hidden, width) : plan_of(rows, width, hidden, group_for(rows));
    plan_pair({rows, hidden, width}, {width, hidden, rows}, false, &g.dx, &g.dw);
    return g;
}

struct LossBackwardSpace {
    TeacherSpace teacher;
    float2* coef;
    float* factor;
    void* x_live;
    void* dz;
    float* logits;    // partial sums of z
    float* partials;  // of dx

    LossBackwardSpace(Carver* w, const LossGradPlan& g, int64_t rows, int64_t hidden, int64_t vocab, int64_t top)
        : teacher(w, rows, vocab, top, false)
    {
        coef = w->take<float2>(rows * 8);
        factor = w->take<float>(8);
        x_live = w->take(rows * hidden * 2);
        dz = w->take(rows * g.piece * 2);
        logits = w->take<float>(logit_bytes(g.z, rows, vocab));
        partials = w->take<float>(g.dx.splits > 1 || g.pieces > 1 ? g.dx.splits * rows * hidden * 4 : 0);
    }
};

size_t loss_bwd_bytes(int64_t rows, int64_t hidden, int64_t vocab, int64_t top)
{
    Carver w(nullptr);
    LossBackwardSpace s(&w, loss_grad_plan(rows, hidden, vocab), rows, hidden, vocab, top);
    return static_cast<size_t>(w.used);
}

dradd_status loss_bwd(void* dx, void* dweight, const float* dloss, int64_t dloss_stride, const float* dlse,
                      int64_t dlse_stride, const dradd_matrix* x, const dradd_matrix* weight, const LossCall& c,
                      const float* lse, int dtype, void* workspace, size_t workspace_bytes, cudaStream_t stream)
{
    DRADD_TRY(loss_shape(c, dtype));
    if (dloss_stride < 0 || dloss_stride > 1 || dlse_stride < 0 || dlse_stride > 1)
        return DRADD_ERR_BAD_SHAPE;
    if (dweight && !aligned(dweight, 16))
        return DRADD_ERR_MISALIGNED;
    if (c.rows == 0)
        return dweight ? from_cuda(cudaMemsetAsync(dweight, 0, c.vocab * c.hidden * 2, stream)) : DRADD_OK;
    if (!dx && !dweight)
        return DRADD_OK;
    Checks k;
    const int64_t r = c.rows, h = c.hidden, v = c.vocab;
    const dradd_matrix mx = {dx, h}, mw = {dweight, h};
    if (dx)
        k.matrix(&mx, r, h, true);
    if (dweight)
        k.matrix(&mw, v, h, true);
    loss_inputs(&k, c, x, weight);
    k.buffer(dloss, dloss_stride ? r : 1, 4, 4, false);
    if (dlse)
        k.buffer(dlse, dlse_stride ? r : 1, 4, 4, false);
    k.buffer(lse, r, 4, 4, false);
    k.workspace(workspace, workspace_bytes, loss_bwd_bytes(r, h, v, c.top()));
    DRADD_TRY(k.done());
    const LossGradPlan g = loss_grad_plan(r, h, v);
    Carver w(workspace);
    const LossBackwardSpace s(&w, g, r, h, v, c.top());
    if (c.teacher)
        DRADD_TRY(from_cuda(s.teacher.run(c, stream)));
    CoefParams f = {};
    f.dloss = dloss;
    f.dloss_stride = dloss_stride;
    f.dlse = dlse;
    f.dlse_stride = dlse_stride;
    f.target = c.target;
    f.ignore_index = c.ignore_index;
    f.entries = s.teacher.entries;
    f.x = x->data;
    f.x_stride = x->stride;
    f.x_live = dweight ? s.x_live : nullptr;
    f.coef = s.coef;
    f.factor = dtype == DRADD_F16 ? s.factor : nullptr;
    f.rows = static_cast<int>(r);
    f.inner = static_cast<int>(h);
    f.vocab = static_cast<int>(v);
    f.top = static_cast<int>(c.top());
    f.inv_temperature = c.inv_temperature();
    DRADD_TRY(from_cuda(launch_coef(f, stream)));
    const float* factor = f.factor ? f.factor + 1 : nullptr;
    for (int64_t i = 0; i < g.pieces; ++i) {
        const int64_t col0 = i * g.piece, width = v - col0 < g.piece ? v - col0 : g.piece;
        const char* w0 = static_cast<const char*>(weight->data) + col0 * weight->stride * 2;
        SlopeParams e = {};
        DRADD_TRY(staging_map(&e.out_map, s.dz, r, g.piece, g.piece));
        e.lse = lse;
        e.coef = s.coef;
        e.target = c.target;
        e.entries = s.teacher.entries;
        e.first = s.teacher.first;
        e.parts = s.teacher.parts;
        e.rows = f.rows;
        e.vocab = static_cast<int>(width);
        e.top = f.top;
        e.col0 = static_cast<int>(col0);
        e.scale = logit_scale(c.inv_temperature());
        const Side sx = {x->data, r, h, x->stride, false}, sw = {w0, width, h, weight->stride, false};
        if (g.z.splits == 1) {
            DRADD_TRY(run_product<SlopeProduct>(plan_of(r, width, h, g.z.group), sx, sw, e, true, dtype, stream));
        } else {
            DRADD_TRY(run_logits(g.z, sx, sw, s.logits, true, dtype, stream));
            DRADD_TRY(from_cuda(launch_slope({s.logits, g.z.splits, up(width, 8)}, e, s.dz, g.piece,
                                             dtype == DRADD_BF16, stream)));
        }
        GradProduct px = {}, pw = {};
        const bool last = i + 1 == g.pieces;
        px.on = dx != nullptr;
        px.plan = plan_of(r, h, width, g.dx.group);
        // the same parts of every piece; of a smaller last one perhaps fewer,
        // whose other partial sums then stay as they are
        px.plan.split(parts_of(g.dx.k_blocks, g.dx.splits), kMostSplits);
        px.a = {s.dz, r, width, g.piece, false};
        px.b = {w0, width, h, weight->stride, true};
        DRADD_TRY(
            grad_params(&px.epi, last && g.dx.splits == 1 ? dx : nullptr, s.partials, factor, r, h, i > 0));
        pw.on = dweight != nullptr;
        pw.plan = plan_of(width, h, r, g.dw.group);
        pw.a = {s.dz, r, width, g.piece, true};
        pw.b = {s.x_live, r, h, h, true};
        DRADD_TRY(grad_params(&pw.epi, dweight ? static_cast<char*>(dweight) + col0 * h * 2 : nullptr, nullptr, factor,
                              width, h, false));
        DRADD_TRY(run_gradients(px, pw, false, dtype, stream));
    }
    if (dx && g.dx.splits > 1)
        return finish_sums(s.partials, g.dx.splits, r, h, dx, factor, dtype, stream);
    return DRADD_OK;
}

LossCall target_call(const int64_t* target, int64_t ignore_index, int64_t rows, int64_t hidden, int64_t vocab)
{
    return {target, ignore_index, nullptr, rows, hidden, vocab};
}

LossCall teacher_call(const dradd_teacher* t, int64_t rows, int64_t hidden, int64_t vocab)
{
    return {nullptr, 0, t, rows, hidden, vocab};
}

bool loss_size_ok(int64_t rows, int64_t hidden, int64_t vocab, int64_t top)
{
    dradd_teacher t = {nullptr, nullptr, DRADD_F32, top, 1.0f};
    return rows > 0 && loss_shape(top ? teacher_call(&t, rows, hidden, vocab)
                                      : target_call(nullptr, 0, rows, hidden, vocab),
                                  DRADD_BF16) == DRADD_OK;
}

}  // namespace
}  // namespace dradd

using namespace dradd;

extern "C" {

size_t linear_act_add_fwd_workspace_bytes(int64_t rows, int64_t inner, int64_t cols)
{
    if (rows <= 0 || linear_shape(rows, inner, cols) != DRADD_OK || few(rows, inner, cols))
        return 0;
    return static_cast<size_t>(partial_bytes(forward_plan(rows, inner, cols), rows, cols));
}

dradd_status linear_act_add_fwd(const dradd_matrix* out, const dradd_matrix* x, const dradd_matrix* weight,
                                const void* bias, const dradd_matrix* residual, int act, int64_t rows,
                                int64_t inner, int64_t cols, int dtype, void* workspace, size_t workspace_bytes,
                                cudaStream_t stream)
{
    if (!dtype_ok(dtype) || act < DRADD_ACT_NONE || act > DRADD_ACT_SILU)
        return DRADD_ERR_BAD_ARG;
    DRADD_TRY(linear_shape(rows, inner, cols));
    if (rows == 0)
        return DRADD_OK;
    const bool has_residual = residual && residual->data;
    Checks k;
    k.matrix(out, rows, cols, true);
    k.matrix(x, rows, inner, false);
    k.matrix(weight, cols, inner, false);
    if (bias)
        k.buffer(bias, cols, 2, 16, false);
    if (has_residual)
        k.matrix(residual, rows, cols, false, true);
    const Plan p = forward_plan(rows, inner, cols);
    k.workspace(workspace, workspace_bytes, few(rows, inner, cols) ? 0 : partial_bytes(p, rows, cols));
    DRADD_TRY(k.done());
    const ActParams a = act_params(out->data, out->stride, bias, has_residual ? residual->data : nullptr,
                                   has_residual ? residual->stride : 0, rows, cols, act);
    if (few(rows, inner, cols)) {
        FewParams f = {x->data, x->stride, weight->data, weight->stride, static_cast<int>(inner), a,
                       dtype == DRADD_BF16, nullptr, kDefaultWaitLimitNs};
        DRADD_TRY(from_cuda(device_status_ptr(&f.status)));
        return from_cuda(launch_few(f, stream));
    }
    return run_linear(p, *x, *weight, a, false, inner, static_cast<float*>(workspace), dtype, stream);
}

size_t linear_act_add_bwd_workspace_bytes(int64_t rows, int64_t inner, int64_t cols, int act, int want_dx,
                                          int want_dweight, int want_dbias)
{
    if (rows <= 0 || linear_shape(rows, inner, cols) != DRADD_OK || act < DRADD_ACT_NONE || act > DRADD_ACT_SILU)
        return 0;
    return static_cast<size_t>(
        linear_grad_plan(rows, inner, cols, act, want_dx != 0, want_dweight != 0, want_dbias != 0).bytes);
}

dradd_status linear_act_add_bwd(void* dx, void* dweight, void* dbias, const dradd_matrix* dout,
                                const dradd_matrix* x, const dradd_matrix* weight, const void* bias, int act,
                                int64_t rows, int64_t inner, int64_t cols, int dtype, void* workspace,
                                size_t workspace_bytes, cudaStream_t stream)
{
    if (!dtype_ok(dtype) || act < DRADD_ACT_NONE || act > DRADD_ACT_SILU)
        return DRADD_ERR_BAD_ARG;
    DRADD_TRY(linear_shape(rows, inner, cols));
    if (!aligned(dweight, 16) || !aligned(dbias, 16))
        return DRADD_ERR_MISALIGNED;
    if (rows == 0) {
        if (dweight)
            DRADD_TRY(from_cuda(cudaMemsetAsync(dweight, 0, cols * inner * 2, stream)));
        return dbias ? from_cuda(cudaMemsetAsync(dbias, 0, cols * 2, stream)) : DRADD_OK;
    }
    if (!dx && !dweight && !dbias)
        return DRADD_OK;
    const LinearGradPlan g = linear_grad_plan(rows, inner, cols, act, dx, dweight, dbias);
    Checks k;
    const dradd_matrix mx = {dx, inner}, mw = {dweight, inner};
    if (dx)
        k.matrix(&mx, rows, inner, true);
    if (dweight)
        k.matrix(&mw, cols, inner, true);
    if (dbias)
        k.buffer(dbias, cols, 2, 16, true);
    k.matrix(dout, rows, cols, false);
    k.matrix(x, rows, inner, false);
    k.matrix(weight, cols, inner, false);
    if (bias)
        k.buffer(bias, cols, 2, 16, false);
    k.workspace(workspace, workspace_bytes, static_cast<size_t>(g.bytes));
    DRADD_TRY(k.done());
    Carver w(workspace);
    void* dz_space = w.take(g.dz);
    float* partial_z = w.take<float>(g.partial_z);
    float* partial_dx = w.take<float>(g.partial_dx);
    float* partial_dw = w.take<float>(g.partial_dw);
    float* partial_db = w.take<float>(g.partial_db);
    const void* dz = dout->data;
    int64_t dz_stride = dout->stride;
    if (act != DRADD_ACT_NONE) {
        ActParams a = act_params(dz_space, cols, bias, dout->data, dout->stride, rows, cols, act);
        a.col_sums = dbias && g.sums ? partial_db : nullptr;
        DRADD_TRY(run_linear(g.z, *x, *weight, a, true, inner, partial_z, dtype, stream));
        dz = dz_space;
        dz_stride = cols;
    }
    if (dbias) {
        const bool once = !g.sums && g.chunks == 1;
        if (!g.sums)
            DRADD_TRY(from_cuda(launch_row_sums(dz, dz_stride, static_cast<int>(rows), static_cast<int>(cols),
                                                dtype == DRADD_BF16, g.chunks, partial_db, once ? dbias : nullptr,
                                                stream)));
        if (!once)
            DRADD_TRY(from_cuda(
                launch_bias(partial_db, g.chunks, static_cast<int>(cols), dbias, dtype == DRADD_BF16, stream)));
    }
    GradProduct px = {}, pw = {};
    px.on = dx != nullptr;
    px.plan = g.dx;
    px.a = {dz, rows, cols, dz_stride, false};
    px.b = {weight->data, cols, inner, weight->stride, true};
    DRADD_TRY(grad_params(&px.epi, g.dx.splits == 1 ? dx : nullptr, partial_dx, nullptr, rows, inner, false));
    pw.on = dweight != nullptr;
    pw.plan = g.dw;
    pw.a = {dz, rows, cols, dz_stride, true};
    pw.b = {x->data, rows, inner, x->stride, true};
    DRADD_TRY(grad_params(&pw.epi, g.dw.splits == 1 ? dweight : nullptr, partial_dw, nullptr, cols, inner, false));
    // the bias's kernel starts its successor when dz is complete
    DRADD_TRY(run_gradients(px, pw, dbias != nullptr, dtype, stream));
    if (dx && g.dx.splits > 1)
        DRADD_TRY(finish_sums(partial_dx, g.dx.splits, rows, inner, dx, nullptr, dtype, stream));
    if (dweight && g.dw.splits > 1)
        DRADD_TRY(finish_sums(partial_dw, g.dw.splits, cols, inner, dweight, nullptr, dtype, stream));
    return DRADD_OK;
}

size_t linear_cross_entropy_fwd_workspace_bytes(int64_t rows, int64_t hidden, int64_t vocab)
{
    return loss_size_ok(rows, hidden, vocab, 0) ? loss_fwd_bytes(rows, hidden, vocab, 0) : 0;
}

dradd_status linear_cross_entropy_fwd(float* loss, float* lse, const dradd_matrix* x, const dradd_matrix* weight,
                                      const int64_t* target, int64_t ignore_index, int64_t rows, int64_t hidden,
                                      int64_t vocab, int dtype, void* workspace, size_t workspace_bytes,
                                      cudaStream_t stream)
{
    return loss_fwd(loss, lse, x, weight, target_call(target, ignore_index, rows, hidden, vocab), dtype, workspace,
                    workspace_bytes, stream);
}

size_t linear_cross_entropy_bwd_workspace_bytes(int64_t rows, int64_t hidden, int64_t vocab)
{
    return loss_size_ok(rows, hidden, vocab, 0) ? loss_bwd_bytes(rows, hidden, vocab, 0) : 0;
}

dradd_status linear_cross_entropy_bwd(void* dx, void* dweight, const float* dloss, int64_t dloss_stride,
                                      const float* dlse, int64_t dlse_stride, const dradd_matrix* x,
                                      const dradd_matrix* weight, const int64_t* target, int64_t ignore_index,
                                      const float* lse, int64_t rows, int64_t hidden, int64_t vocab, int dtype,
                                      void* workspace, size_t workspace_bytes, cudaStream_t stream)
{
    return loss_bwd(dx, dweight, dloss, dloss_stride, dlse, dlse_stride, x, weight,
                    target_call(target, ignore_index, rows, hidden, vocab), lse, dtype, workspace, workspace_bytes,
                    stream);
}

size_t linear_distill_fwd_workspace_bytes(int64_t rows, int64_t hidden, int64_t vocab, int64_t top)
{
    return top > 0 && loss_size_ok(rows, hidden, vocab, top) ? loss_fwd_bytes(rows, hidden, vocab, top) : 0;
}

dradd_status linear_distill_fwd(float* loss, float* lse, const dradd_matrix* x, const dradd_matrix* weight,
                                const dradd_teacher* teacher, int64_t rows, int64_t hidden, int64_t vocab,
                                int dtype, void* workspace, size_t workspace_bytes, cudaStream_t stream)
{
    if (!teacher)
        return DRADD_ERR_NULL_PTR;
    return loss_fwd(loss, lse, x, weight, teacher_call(teacher, rows, hidden, vocab), dtype, workspace,
                    workspace_bytes, stream);
}

size_t linear_distill_bwd_workspace_bytes(int64_t rows, int64_t hidden, int64_t vocab, int64_t top)
{
    return top > 0 && loss_size_ok(rows, hidden, vocab, top) ? loss_bwd_bytes(rows, hidden, vocab, top) : 0;
}

dradd_status linear_distill_bwd(void* dx, void* dweight, const float* dloss, int64_t dloss_stride,
                                const float* dlse, int64_t dlse_stride, const dradd_matrix* x,
                                const dradd_matrix* weight, const dradd_teacher* teacher, const float* lse,
                                int64_t rows, int64_t hidden, int64_t vocab, int dtype, void* workspace,
                                size_t workspace_bytes, cudaStream_t stream)
{
    if (!teacher)
        return DRADD_ERR_NULL_PTR;
    return loss_bwd(dx, dweight, dloss, dloss_stride, dlse, dlse_stride, x, weight,
                    teacher_call(teacher, rows, hidden, vocab), lse, dtype, workspace, workspace_bytes, stream);
}

}  // extern "C"
