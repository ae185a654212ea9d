// dradd_train_abi.cu -- the C entry points of include/dradd_train.h:
// argument checks and dispatch.  Every check is made before any GPU work.
#include <cmath>
#include <cstdint>

#include "dradd_train.h"

#include "dradd_host.h"
#include "dradd_internal.h"
#include "dradd_train_internal.h"

namespace {

using namespace dradd;

bool dtype_ok(int dtype) { return dtype == DRADD_BF16 || dtype == DRADD_F16 || dtype == DRADD_F32; }
int64_t elem_bytes(int dtype) { return dtype == DRADD_F32 ? 4 : 2; }

float inverse_if_pow2(int64_t n) { return (n & (n - 1)) == 0 ? 1.0f / static_cast<float>(n) : 0.0f; }

// ------------------------------------------------------------------ dropout
dradd_status drop_params(const dradd_dropout* d, DropParams* out)
{
    if (!d)
        return DRADD_ERR_NULL_PTR;
    if (!(d->p >= 0.0f && d->p <= 1.0f))
        return DRADD_ERR_BAD_ARG;
    if (d->step && !aligned(d->step, 8))
        return DRADD_ERR_MISALIGNED;
    const uint32_t t = static_cast<uint32_t>(std::nearbyint(static_cast<double>(d->p) * 65536.0));
    *out = make_drop_params(d->seed, d->offset, d->step, t,
                            t < 65536 ? static_cast<float>(65536.0 / (65536.0 - t)) : 0.0f);
    return DRADD_OK;
}

View rows_view(const void* p, int64_t n_rows, int64_t cols, int64_t stride, int64_t elem)
{
    View v;
    v.base = reinterpret_cast<uintptr_t>(p);
    v.elem = elem;
    v.add(n_rows, stride);
    v.add(cols, 1);
    return v;
}

View flat_view(const void* p, int64_t n, int64_t elem) { return rows_view(p, 1, n, n, elem); }

dradd_status run_dropout(void* out, int64_t out_stride, const void* x, int64_t x_stride, const void* residual,
                         int64_t residual_stride, bool add, int64_t n_rows, int64_t hidden,
                         const dradd_dropout* drop, int dtype, cudaStream_t stream)
{
    DropoutArgs a = {};
    if (!dtype_ok(dtype))
        return DRADD_ERR_BAD_ARG;
    dradd_status st = drop_params(drop, &a.drop);
    if (st != DRADD_OK)
        return st;
    if (n_rows < 0 || n_rows > 0x7FFFFFFFll || hidden <= 0 || hidden > 0x7FFFFFFFll)
        return DRADD_ERR_BAD_SHAPE;
    if (n_rows == 0)
        return DRADD_OK;
    if (n_rows > 1 && (out_stride < hidden || x_stride < hidden || (add && residual_stride < hidden)))
        return DRADD_ERR_BAD_SHAPE;
    if (!out || !x || (add && !residual))
        return DRADD_ERR_NULL_PTR;
    const int64_t eb = elem_bytes(dtype);
    if (!aligned(out, eb) || !aligned(x, eb) || (add && !aligned(residual, eb)))
        return DRADD_ERR_MISALIGNED;
    const View vo = rows_view(out, n_rows, hidden, out_stride, eb);
    const View vx = rows_view(x, n_rows, hidden, x_stride, eb);
    const View vr = rows_view(residual, n_rows, hidden, residual_stride, eb);
    if (!view_fits(vo) || !view_fits(vx) || (add && !view_fits(vr)))
        return DRADD_ERR_BAD_SHAPE;
    if ((!vo.same(vx) && views_may_overlap(vo, vx)) || (add && !vo.same(vr) && views_may_overlap(vo, vr)))
        return DRADD_ERR_ALIAS;
    if (a.drop.step && views_may_overlap(vo, flat_view(a.drop.step, 1, 8)))
        return DRADD_ERR_ALIAS;
    DeviceLimits L;
    st = query_limits(&L);
    if (st != DRADD_OK)
        return st;
    a.out = out;
    a.x = x;
    a.residual = add ? residual : nullptr;
    a.out_stride = out_stride;
    a.x_stride = x_stride;
    a.residual_stride = residual_stride;
    a.n_rows = n_rows;
    a.hidden = hidden;
    auto rows_aligned = [&](const void* p, int64_t stride) {
        return aligned(p, 16) && (n_rows == 1 || stride * eb % 16 == 0);
    };
    const bool blocks = hidden % 8 == 0 && rows_aligned(out, out_stride) && rows_aligned(x, x_stride) &&
                        (!add || rows_aligned(residual, residual_stride));
    auto one_run = [&](const void* p, int64_t stride) {
        return aligned(p, 16) && (n_rows == 1 || stride == hidden);
    };
    const bool flat = hidden >= kFlatHidden && one_run(out, out_stride) && one_run(x, x_stride) &&
                      (!add || one_run(residual, residual_stride));
    const DropoutLayout layout = blocks ? kDropoutBlocks : flat ? kDropoutFlat : kDropoutRagged;
    return launch_dropout(a, dtype, layout, L.sm_count, stream) == cudaSuccess ? DRADD_OK : DRADD_ERR_CUDA;
}

// ------------------------------------- dropout + residual add + RMSNorm
dradd_status norm_shape(int64_t n_rows, int64_t hidden)
{
    if (n_rows < 0 || n_rows > 0x7FFFFFFFll || hidden <= 0)
        return DRADD_ERR_BAD_SHAPE;
    if (hidden % 8 != 0 || hidden > DRADD_MAX_HIDDEN)
        return DRADD_ERR_UNSUPPORTED_HIDDEN;
    return DRADD_OK;
}

bool eps_ok(float eps) { return std::isfinite(eps) && eps >= 0.0f; }

// Each output disjoint from the others, and from every input but those it
// may be exactly.
struct Checked {
    View view;
    bool in_place;  // input: an output may be exactly this
};

dradd_status check_views(const View* outs, int n_out, const Checked* ins, int n_in)
{
    for (int i = 0; i < n_out; ++i) {
        for (int j = i + 1; j < n_out; ++j)
            if (views_may_overlap(outs[i], outs[j]))
                return DRADD_ERR_ALIAS;
        for (int j = 0; j < n_in; ++j)
            if (!(ins[j].in_place && outs[i].same(ins[j].view)) && views_may_overlap(outs[i], ins[j].view))
                return DRADD_ERR_ALIAS;
    }
    return DRADD_OK;
}

dradd_status fill_status(DropNormArgs* a)
{
    a->wait_limit_ns = kDefaultWaitLimitNs;
    return device_status_ptr(&a->status) == cudaSuccess ? DRADD_OK : DRADD_ERR_CUDA;
}

dradd_status run_norm_bwd(void* dx, void* dresidual, float* dweight, const void* dout, const void* dresidual_out,
                          const void* h, const void* weight, float eps, int64_t n_rows, int64_t hidden,
                          const dradd_dropout* drop, int dtype, void* workspace, size_t workspace_bytes,
                          cudaStream_t stream)
{
    DropNormArgs a = {};
    if (!dtype_ok(dtype))
        return DRADD_ERR_BAD_ARG;
    dradd_status st = drop_params(drop, &a.drop);
    if (st != DRADD_OK)
        return st;
    st = norm_shape(n_rows, hidden);
    if (st != DRADD_OK)
        return st;
    if (!eps_ok(eps))
        return DRADD_ERR_BAD_EPS;
    if (dweight && !aligned(dweight, 4))
        return DRADD_ERR_MISALIGNED;
    if (n_rows == 0) {
        if (dweight && cudaMemsetAsync(dweight, 0, hidden * 4, stream) != cudaSuccess)
            return DRADD_ERR_CUDA;
        return DRADD_OK;
    }
    if (!dresidual || !dout || !h || !weight)
        return DRADD_ERR_NULL_PTR;
    if (!aligned(dx, 16) || !aligned(dresidual, 16) || !aligned(dout, 16) || !aligned(dresidual_out, 16) ||
        !aligned(h, 16) || !aligned(weight, 16) || (dweight && !aligned(workspace, 16)))
        return DRADD_ERR_MISALIGNED;
    const size_t need = rmsnorm_bwd_workspace_bytes(n_rows, hidden, dtype);
    if (dweight && (!workspace || workspace_bytes < need))
        return DRADD_ERR_WORKSPACE;
    const int64_t eb = elem_bytes(dtype), n = n_rows * hidden;
    View outs[4];
    Checked ins[5];
    int n_out = 0, n_in = 0;
    outs[n_out++] = flat_view(dresidual, n, eb);
    if (dx)
        outs[n_out++] = flat_view(dx, n, eb);
    if (dweight) {
        outs[n_out++] = flat_view(dweight, hidden, 4);
        outs[n_out++] = flat_view(workspace, static_cast<int64_t>(need / 4), 4);
    }
    ins[n_in++] = {flat_view(dout, n, eb), true};
    if (dresidual_out)
        ins[n_in++] = {flat_view(dresidual_out, n, eb), true};
    ins[n_in++] = {flat_view(h, n, eb), true};
    ins[n_in++] = {flat_view(weight, hidden, eb), false};
    if (a.drop.step)
        ins[n_in++] = {flat_view(a.drop.step, 1, 8), false};
    st = check_views(outs, n_out, ins, n_in);
    if (st == DRADD_OK)
        st = fill_status(&a);
    if (st != DRADD_OK)
        return st;
    a.weight = weight;
    a.dx = dx;
    a.dresidual = dresidual;
    a.partials = dweight ? static_cast<float*>(workspace) : nullptr;
    a.dout = dout;
    a.dresidual_out = dresidual_out;
    a.h = h;
    a.n_rows = n_rows;
    a.hidden = static_cast<int>(hidden);
    a.inv_hidden = inverse_if_pow2(hidden);
    a.eps = eps;
    const bool device = all_device_memory({dx, dresidual, dout, dresidual_out, h, weight});
    const DropNormPlan p = drop_norm_plan(n_rows, a.hidden, dtype, true, device);
    a.stages = p.stages;
    if (launch_drop_norm_bwd(a, p, dtype, stream) != cudaSuccess)
        return DRADD_ERR_CUDA;
    if (dweight && launch_column_sums(a.partials, p.grid, a.hidden, dweight, a.hidden, nullptr, stream) != cudaSuccess)
        return DRADD_ERR_CUDA;
    return DRADD_OK;
}

// ------------------------------------------------------------------- rotary
// A checked side of a rotary call.
View heads_view(const dradd_heads& t, const dradd_rope& r, int64_t heads, int64_t elem)
{
    View v;
    v.base = reinterpret_cast<uintptr_t>(t.data);
    v.elem = elem;
    v.add(r.batch, t.batch_stride);
    v.add(r.seq, t.seq_stride);
    v.add(heads, t.head_stride);
    v.add(r.head_dim, 1);
    return v;
}

// Shape and layout; the plan of the call goes to `a` and `grid`.
dradd_status rope_shape(const dradd_rope* r, int dtype, RopeArgs* a, bool backward, int* grid)
{
    if (!r)
        return DRADD_ERR_NULL_PTR;
    if (!dtype_ok(dtype) || (r->interleaved != 0 && r->interleaved != 1) || !std::isfinite(r->scale))
        return DRADD_ERR_BAD_ARG;
    if (r->batch < 0 || r->seq < 0 || r->q_heads < 1 || r->k_heads < 0 || r->head_dim < 1)
        return DRADD_ERR_BAD_SHAPE;
    if (r->rot_dim < 2 || r->rot_dim % 2 != 0 || r->rot_dim > r->head_dim)
        return DRADD_ERR_BAD_SHAPE;
    if (r->head_dim > kRopeMaxDim || (r->rot_dim + 15) / 16 + (r->head_dim - r->rot_dim + 15) / 16 > 32)
        return DRADD_ERR_UNSUPPORTED_HIDDEN;
    if (r->q_heads > 65536 || r->k_heads > 65536 ||
        (r->seq > 0 && r->batch > 0x7FFFFFFFll / r->seq))
        return DRADD_ERR_BAD_SHAPE;
    a->tokens = r->batch * r->seq;
    a->seq = r->seq;
    a->dim = static_cast<int>(r->head_dim);
    a->rot = static_cast<int>(r->rot_dim);
    a->inv_dim = 1.0f / static_cast<float>(r->head_dim);
    a->q.heads = static_cast<int>(r->q_heads);
    a->k.heads = static_cast<int>(r->k_heads);
    a->inv_freq = r->inv_freq;
    a->positions = r->positions;
    a->position0 = r->position0;
    a->scale = r->scale;
    if (a->tokens > 0)
        rope_plan(a, dtype, backward, grid);
    return DRADD_OK;
}

// Pointers, strides and overlaps of one call's views: out[i] may be exactly
// in[i] or grad[i].  *blocks: every head moves as aligned blocks of 8.
struct RopeSideArgs {
    const dradd_heads *out, *in, *grad;  // grad: the norm's backward only
    const void* weight;                  // the norm only
};

dradd_status rope_check(const dradd_rope& r, const RopeSideArgs (&sides)[2], bool norm, bool has_grad, int64_t eb,
                        const void* extra_out0, int64_t extra_bytes0, const void* extra_out1, int64_t extra_bytes1,
                        const void* extra_out2, int64_t extra_bytes2, bool* blocks)
{
    const int n_sides = r.k_heads > 0 ? 2 : 1;
    const int64_t heads[2] = {r.q_heads, r.k_heads};
    View outs[5];
    Checked ins[8];
    int n_out = 0, n_in = 0;
    if (!r.inv_freq)
        return DRADD_ERR_NULL_PTR;
    if (!aligned(r.inv_freq, 8) || !aligned(r.positions, 8))
        return DRADD_ERR_MISALIGNED;
    bool vec = r.head_dim % 8 == 0 && (r.interleaved || r.rot_dim % 16 == 0);
    for (int s = 0; s < n_sides; ++s) {
        const dradd_heads* t[3] = {sides[s].out, sides[s].in, sides[s].grad};
        for (int i = 0; i < 3; ++i) {
            if (i == 2 && !has_grad)
                continue;
            if (!t[i] || !t[i]->data)
                return DRADD_ERR_NULL_PTR;
            if (!aligned(t[i]->data, eb))
                return DRADD_ERR_MISALIGNED;
            const View v = heads_view(*t[i], r, heads[s], eb);
            if (!view_fits(v))
                return DRADD_ERR_BAD_SHAPE;
            const auto whole = [&](int64_t n, int64_t stride) { return n == 1 || stride * eb % 16 == 0; };
            vec = vec && aligned(t[i]->data, 16) && whole(r.batch, t[i]->batch_stride) &&
                  whole(r.seq, t[i]->seq_stride) && whole(heads[s], t[i]->head_stride);
            if (i == 0)
                outs[n_out++] = v;
            else
                ins[n_in++] = {v, true};
        }
        if (norm) {
            if (!sides[s].weight)
                return DRADD_ERR_NULL_PTR;
            if (!aligned(sides[s].weight, eb))
                return DRADD_ERR_MISALIGNED;
            ins[n_in++] = {flat_view(sides[s].weight, r.head_dim, eb), false};
        }
    }
    ins[n_in++] = {flat_view(r.inv_freq, r.rot_dim / 2, 8), false};
    if (r.positions)
        ins[n_in++] = {flat_view(r.positions, r.batch * r.seq, 8), false};
    for (int i = 0; i < n_out; ++i)
        if (view_overlaps_itself(outs[i]))
            return DRADD_ERR_ALIAS;
    // an output may be exactly its own side's input, not the other's
    for (int i = 0; i < n_out; ++i) {
        for (int s = 0; s < n_sides; ++s) {
            if (s == i)
                continue;
            const dradd_heads* t[2] = {sides[s].in, sides[s].grad};
            for (const dradd_heads* other : t)
                if (other && views_may_overlap(outs[i], heads_view(*other, r, heads[s], eb)))
                    return DRADD_ERR_ALIAS;
        }
    }
    if (extra_out0)
        outs[n_out++] = flat_view(extra_out0, extra_bytes0, 1);
    if (extra_out1)
        outs[n_out++] = flat_view(extra_out1, extra_bytes1, 1);
    if (extra_out2)
        outs[n_out++] = flat_view(extra_out2, extra_bytes2, 1);
    *blocks = vec;
    return check_views(outs, n_out, ins, n_in);
}

HeadsView heads_bytes(const dradd_heads& t, int64_t eb, int per_step)
{
    return {static_cast<char*>(t.data), t.batch_stride * eb, t.seq_stride * eb, t.head_stride * eb,
            t.head_stride * eb * per_step};
}

void fill_side(RopeSide* s, const RopeSideArgs& t, float eps, int64_t eb, int per_step)
{
    s->t[kRopeIn] = heads_bytes(*t.in, eb, per_step);
    s->t[kRopeOut] = heads_bytes(*t.out, eb, per_step);
    if (t.grad)
        s->t[kRopeGrad] = heads_bytes(*t.grad, eb, per_step);
    s->weight = t.weight;
    s->eps = eps;
}

dradd_status run_rope(const dradd_heads* q_out, const dradd_heads* k_out, const dradd_heads* q, const dradd_heads* k,
                      const void* q_weight, const void* k_weight, float q_eps, float k_eps, bool norm, float sign,
                      const dradd_rope* r, int dtype, cudaStream_t stream)
{
    RopeArgs a = {};
    int grid = 0;
    dradd_status st = rope_shape(r, dtype, &a, false, &grid);
    if (st != DRADD_OK)
        return st;
    if (norm && (!eps_ok(q_eps) || (r->k_heads > 0 && !eps_ok(k_eps))))
        return DRADD_ERR_BAD_EPS;
    if (a.tokens == 0)
        return DRADD_OK;
    const RopeSideArgs sides[2] = {{q_out, q, nullptr, q_weight}, {k_out, k, nullptr, k_weight}};
    bool blocks = false;
    st = rope_check(*r, sides, norm, false, elem_bytes(dtype), nullptr, 0, nullptr, 0, nullptr, 0, &blocks);
    if (st != DRADD_OK)
        return st;
    a.sign = sign;
    fill_side(&a.q, sides[0], q_eps, elem_bytes(dtype), a.heads_per_step);
    if (r->k_heads > 0)
        fill_side(&a.k, sides[1], k_eps, elem_bytes(dtype), a.heads_per_step);
    if (!norm) {
        a.q.skip_rest = a.q.t[kRopeOut].data == a.q.t[kRopeIn].data;
        a.k.skip_rest = a.k.t[kRopeOut].data == a.k.t[kRopeIn].data;
    }
    return launch_rope(a, norm ? kRopeNorm : kRopePlain, dtype, r->interleaved != 0, blocks, grid, stream) ==
                   cudaSuccess
               ? DRADD_OK
               : DRADD_ERR_CUDA;
}

}  // namespace

extern "C" {

dradd_status dropout_fwd(void* out, int64_t out_stride, const void* x, int64_t x_stride, int64_t n_rows,
                         int64_t hidden, const dradd_dropout* drop, int dtype, cudaStream_t stream)
{
    return run_dropout(out, out_stride, x, x_stride, nullptr, 0, false, n_rows, hidden, drop, dtype, stream);
}

dradd_status dropout_add_fwd(void* residual_out, int64_t out_stride, const void* x, int64_t x_stride,
                             const void* residual, int64_t residual_stride, int64_t n_rows, int64_t hidden,
                             const dradd_dropout* drop, int dtype, cudaStream_t stream)
{
    return run_dropout(residual_out, out_stride, x, x_stride, residual, residual_stride, true, n_rows, hidden, drop,
                       dtype, stream);
}

dradd_status dropout_add_rmsnorm_fwd(void* out, void* residual_out, const void* x, const void* residual,
                                     const void* weight, float eps, int64_t n_rows, int64_t hidden,
                                     const dradd_dropout* drop, int dtype, cudaStream_t stream)
{
    DropNormArgs a = {};
    if (!dtype_ok(dtype))
        return DRADD_ERR_BAD_ARG;
    dradd_status st = drop_params(drop, &a.drop);
    if (st == DRADD_OK)
        st = norm_shape(n_rows, hidden);
    if (st != DRADD_OK)
        return st;
    if (!eps_ok(eps))
        return DRADD_ERR_BAD_EPS;
    if (n_rows == 0)
        return DRADD_OK;
    if (!out || !residual_out || !x || !residual || !weight)
        return DRADD_ERR_NULL_PTR;
    if (!aligned(out, 16) || !aligned(residual_out, 16) || !aligned(x, 16) || !aligned(residual, 16) ||
        !aligned(weight, 16))
        return DRADD_ERR_MISALIGNED;
    const int64_t eb = elem_bytes(dtype), n = n_rows * hidden;
    const View outs[2] = {flat_view(out, n, eb), flat_view(residual_out, n, eb)};
    const Checked ins[4] = {{flat_view(x, n, eb), true},
                            {flat_view(residual, n, eb), true},
                            {flat_view(weight, hidden, eb), false},
                            {flat_view(a.drop.step, 1, 8), false}};
    st = check_views(outs, 2, ins, a.drop.step ? 4 : 3);
    if (st == DRADD_OK)
        st = fill_status(&a);
    if (st != DRADD_OK)
        return st;
    a.out = out;
    a.residual_out = residual_out;
    a.x = x;
    a.residual = residual;
    a.weight = weight;
    a.n_rows = n_rows;
    a.hidden = static_cast<int>(hidden);
    a.inv_hidden = inverse_if_pow2(hidden);
    a.eps = eps;
    const bool device = all_device_memory({out, residual_out, x, residual, weight});
    const DropNormPlan p = drop_norm_plan(n_rows, a.hidden, dtype, false, device);
    a.stages = p.stages;
    return launch_drop_norm_fwd(a, p, dtype, stream) == cudaSuccess ? DRADD_OK : DRADD_ERR_CUDA;
}

dradd_status dropout_add_rmsnorm_bwd(void* dx, void* dresidual, float* dweight, const void* dout,
                                     const void* dresidual_out, const void* h, const void* weight, float eps,
                                     int64_t n_rows, int64_t hidden, const dradd_dropout* drop, int dtype,
                                     void* workspace, size_t workspace_bytes, cudaStream_t stream)
{
    return run_norm_bwd(dx, dresidual, dweight, dout, dresidual_out, h, weight, eps, n_rows, hidden, drop, dtype,
                        workspace, workspace_bytes, stream);
}

dradd_status add_rmsnorm_bwd(void* dh, float* dweight, const void* dout, const void* dresidual_out, const void* h,
                             const void* weight, float eps, int64_t n_rows, int64_t hidden, int dtype,
                             void* workspace, size_t workspace_bytes, cudaStream_t stream)
{
    const dradd_dropout none = {0.0f, 0, 0, nullptr};
    return run_norm_bwd(nullptr, dh, dweight, dout, dresidual_out, h, weight, eps, n_rows, hidden, &none, dtype,
                        workspace, workspace_bytes, stream);
}

size_t rmsnorm_bwd_workspace_bytes(int64_t n_rows, int64_t hidden, int dtype)
{
    if (!dtype_ok(dtype) || norm_shape(n_rows, hidden) != DRADD_OK || n_rows == 0)
        return 0;
    const DropNormPlan p = drop_norm_plan(n_rows, static_cast<int>(hidden), dtype, true, true);
    return static_cast<size_t>(p.grid) * static_cast<size_t>(hidden) * sizeof(float);
}

dradd_status rope_fwd(const dradd_heads* q_out, const dradd_heads* k_out, const dradd_heads* q,
                      const dradd_heads* k, const dradd_rope* rope, int dtype, cudaStream_t stream)
{
    return run_rope(q_out, k_out, q, k, nullptr, nullptr, 0.0f, 0.0f, false, 1.0f, rope, dtype, stream);
}

dradd_status rope_bwd(const dradd_heads* dq, const dradd_heads* dk, const dradd_heads* dq_out,
                      const dradd_heads* dk_out, const dradd_rope* rope, int dtype, cudaStream_t stream)
{
    return run_rope(dq, dk, dq_out, dk_out, nullptr, nullptr, 0.0f, 0.0f, false, -1.0f, rope, dtype, stream);
}

dradd_status qk_rmsnorm_rope_fwd(const dradd_heads* q_out, const dradd_heads* k_out, const dradd_heads* q,
                                 const dradd_heads* k, const void* q_weight, const void* k_weight, float q_eps,
                                 float k_eps, const dradd_rope* rope, int dtype, cudaStream_t stream)
{
    return run_rope(q_out, k_out, q, k, q_weight, k_weight, q_eps, k_eps, true, 1.0f, rope, dtype, stream);
}

dradd_status qk_rmsnorm_rope_bwd(const dradd_heads* dq, const dradd_heads* dk, float* dq_weight, float* dk_weight,
                                 const dradd_heads* dq_out, const dradd_heads* dk_out, const dradd_heads* q,
                                 const dradd_heads* k, const void* q_weight, const void* k_weight, float q_eps, float k_eps,
                                 const dradd_rope* rope, int dtype, void* workspace, size_t workspace_bytes,
                                 cudaStream_t stream)
{
    RopeArgs a = {};
    int grid = 0;
    dradd_status st = rope_shape(rope, dtype, &a, true, &grid);
    if (st != DRADD_OK)
        return st;
    const bool has_k = rope->k_heads > 0;
    if (!eps_ok(q_eps) || (has_k && !eps_ok(k_eps)))
        return DRADD_ERR_BAD_EPS;
    float* const dk_sums = has_k ? dk_weight : nullptr;  // a sum over no heads is zeros, below
    const bool sums = dq_weight || dk_sums;
    if (!aligned(dq_weight, 4) || !aligned(dk_weight, 4))
        return DRADD_ERR_MISALIGNED;
    if (a.tokens == 0) {
        for (float* w : {dq_weight, dk_weight})
            if (w && cudaMemsetAsync(w, 0, static_cast<size_t>(a.dim) * 4, stream) != cudaSuccess)
                return DRADD_ERR_CUDA;
        return DRADD_OK;
    }
    const size_t need = static_cast<size_t>(grid) * 2 * static_cast<size_t>(a.dim) * sizeof(float);
    if (sums && !aligned(workspace, 16))
        return DRADD_ERR_MISALIGNED;
    if (sums && (!workspace || workspace_bytes < need))
        return DRADD_ERR_WORKSPACE;
    const RopeSideArgs sides[2] = {{dq, q, dq_out, q_weight}, {dk, k, dk_out, k_weight}};
    bool blocks = false;
    st = rope_check(*rope, sides, true, true, elem_bytes(dtype), dq_weight, a.dim * 4, dk_weight, a.dim * 4,
                    sums ? workspace : nullptr, static_cast<int64_t>(need), &blocks);
    if (st != DRADD_OK)
        return st;
    a.sign = -1.0f;
    fill_side(&a.q, sides[0], q_eps, elem_bytes(dtype), a.heads_per_step);
    if (has_k)
        fill_side(&a.k, sides[1], k_eps, elem_bytes(dtype), a.heads_per_step);
    a.partials = sums ? static_cast<float*>(workspace) : nullptr;
    if (launch_rope(a, kRopeNormBwd, dtype, rope->interleaved != 0, blocks, grid, stream) != cudaSuccess)
        return DRADD_ERR_CUDA;
    if (sums && launch_column_sums(a.partials, grid, 2 * a.dim, dq_weight, a.dim, dk_sums, stream) != cudaSuccess)
        return DRADD_ERR_CUDA;
    if (dk_weight && !has_k && cudaMemsetAsync(dk_weight, 0, static_cast<size_t>(a.dim) * 4, stream) != cudaSuccess)
        return DRADD_ERR_CUDA;
    return DRADD_OK;
}

size_t qk_rmsnorm_rope_bwd_workspace_bytes(const dradd_rope* rope, int dtype)
{
    RopeArgs a = {};
    int grid = 0;
    if (rope_shape(rope, dtype, &a, true, &grid) != DRADD_OK || a.tokens == 0)
        return 0;
    return static_cast<size_t>(grid) * 2 * static_cast<size_t>(a.dim) * sizeof(float);
}

dradd_status rope_frequencies(double* out, int64_t rot_dim, double base, int scaling, double factor,
                              double original_length, double low, double high)
{
    if (!out)
        return DRADD_ERR_NULL_PTR;
    if (rot_dim < 2 || rot_dim % 2 != 0 || rot_dim > kRopeMaxDim)
        return DRADD_ERR_BAD_SHAPE;
    if (!std::isfinite(base) || base <= 0.0 || scaling < DRADD_ROPE_PLAIN || scaling > DRADD_ROPE_BY_PARTS)
        return DRADD_ERR_BAD_ARG;
    if (scaling != DRADD_ROPE_PLAIN && (!std::isfinite(factor) || factor < 1.0))
        return DRADD_ERR_BAD_ARG;
    if (scaling == DRADD_ROPE_BY_PARTS && (!std::isfinite(original_length) || original_length <= 0.0 ||
                                           !std::isfinite(low) || !std::isfinite(high) || low >= high))
        return DRADD_ERR_BAD_ARG;
    if (scaling == DRADD_ROPE_BASE && rot_dim == 2)
        return DRADD_ERR_BAD_ARG;
    const double d = static_cast<double>(rot_dim);
    if (scaling == DRADD_ROPE_BASE)
        base *= std::pow(factor, d / (d - 2.0));
    for (int64_t i = 0; i < rot_dim / 2; ++i) {
        double f = std::pow(base, -2.0 * static_cast<double>(i) / d);
        if (scaling == DRADD_ROPE_LINEAR) {
            f /= factor;
        } else if (scaling == DRADD_ROPE_BY_PARTS) {
            const double turns = original_length * f / 6.283185307179586476925;
            double r = (turns - low) / (high - low);
            r = r < 0.0 ? 0.0 : r > 1.0 ? 1.0 : r;
            f *= r + (1.0 - r) / factor;
        }
        out[i] = f;
    }
    return DRADD_OK;
}

}  // extern "C"
