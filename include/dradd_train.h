/*
 * dradd_train.h -- what libdradd adds around the residual-add + RMSNorm of
 * dradd.h for training a pre-norm block and for its attention inputs:
 *   - dropout whose mask is a function of (seed, offset, row, column) and is
 *     never stored, alone, with the residual add, and fused in front of
 *     residual-add + RMSNorm;
 *   - the gradients of (dropout +) residual-add + RMSNorm;
 *   - rotary positions of q and k, plain or behind their RMSNorm, and the
 *     gradients of both.
 *
 * The conventions of dradd.h hold (pointers the device can reach, caller's
 * buffers, asynchronous on `stream`, argument errors before any GPU work,
 * results that do not depend on the launch), with these additions:
 *   - dtype: DRADD_BF16, DRADD_F16 or DRADD_F32, the type of every tensor
 *     argument declared void*.  Arithmetic is fp32; each stored element is
 *     rounded once, to nearest even.
 *   - A call makes one launch, or two where it sums weight gradients: each
 *     CTA adds its rows in order into one partial sum per column, in the
 *     caller's workspace, and a second kernel adds those in a fixed order.
 *     How many partial sums there are depends on the shape and the dtype
 *     alone, so the bits do too.
 *   - workspace: device memory, 16-byte aligned, of the size its query
 *     states; contents need no preparation and are left undefined.  Calls
 *     that may run at the same time need workspaces of their own.
 *   - "may be exactly": the same address, sizes and strides.  Any other
 *     overlap of an output with another buffer is DRADD_ERR_ALIAS.
 */
#ifndef DRADD_TRAIN_H
#define DRADD_TRAIN_H

#include <stddef.h>

#include "dradd.h"

#ifdef __cplusplus
extern "C" {
#endif

enum { DRADD_BF16 = 0, DRADD_F16 = 1, DRADD_F32 = 2 };

/*
 * The dropout mask of a call.
 *   p       probability of dropping, 0 <= p <= 1, applied as t / 65536 with
 *           t = p * 65536 rounded to nearest even
 *   seed, offset   which mask: calls with another seed or another offset
 *           draw independent ones.  Forward and backward of one dropout take
 *           the same pair.
 *   step    NULL, or a device int64 added to offset (mod 2^64) when the
 *           kernel runs, so a captured graph draws a new mask at every
 *           replay if the program changes the value in between (8-byte
 *           aligned).  Calls of equal offset + step have one mask: where
 *           layers take the offsets 0 .. L - 1, let the value advance by L
 *           a replay, or space the offsets 2^32 apart; advancing by one
 *           would give a layer the mask its neighbour just had.
 * The element in (row, column) is kept when
 *     u >= t,  u = 16 bits (column % 8) of Philox4x32-7 with the counter
 *     (column / 8, row, offset low, offset high) and the key seed,
 * low halves first, and is then multiplied by RN(65536 / (65536 - t)), so
 * that the expectation is the input.  A dropped element counts as +0,
 * whatever it holds.
 */
typedef struct dradd_dropout {
    float p;
    uint64_t seed;
    uint64_t offset;
    const int64_t* step;
} dradd_dropout;

/*
 * dropout_fwd -- out = dropout(x), n_rows x hidden with row strides in
 * elements (unit column stride).  It is its own gradient: dx = dropout(dy)
 * with the same mask.
 *   1 <= hidden < 2^31 (a multiple of 8 or not), n_rows < 2^31, strides >=
 *   hidden, pointers aligned to the element.  Rows of whole 16-byte vectors
 *   (hidden % 8 == 0, 16-byte aligned rows) take the fast path.
 *   out may be exactly x.
 */
dradd_status dropout_fwd(void* out, int64_t out_stride, const void* x, int64_t x_stride, int64_t n_rows,
                         int64_t hidden, const dradd_dropout* drop, int dtype, cudaStream_t stream);

/*
 * dropout_add_fwd -- residual_out = residual + dropout(x) (one fp32 addition
 * of the scaled, unrounded x).  Its gradients: dresidual = dy, dx =
 * dropout(dy).  residual_out may be exactly x or residual.
 */
dradd_status dropout_add_fwd(void* residual_out, int64_t out_stride, const void* x, int64_t x_stride,
                             const void* residual, int64_t residual_stride, int64_t n_rows, int64_t hidden,
                             const dradd_dropout* drop, int dtype, cudaStream_t stream);

/*
 * dropout_add_rmsnorm_fwd -- add_rmsnorm_fwd with dropout on x:
 *     acc          = fp32(residual) + dropout(fp32(x))
 *     residual_out = rne(acc)
 *     out          = rne((acc * inv) * fp32(weight)),  inv as in dradd.h
 * With p = 0 and bf16 the results are add_rmsnorm_fwd's, bit for bit.
 * Tensors are contiguous, hidden a multiple of 8 up to DRADD_MAX_HIDDEN,
 * pointers 16-byte aligned, n_rows < 2^31.  out and residual_out may each be
 * exactly x or residual.
 */
dradd_status dropout_add_rmsnorm_fwd(void* out, void* residual_out, const void* x, const void* residual,
                                     const void* weight, float eps, int64_t n_rows, int64_t hidden,
                                     const dradd_dropout* drop, int dtype, cudaStream_t stream);

/*
 * dropout_add_rmsnorm_bwd -- gradients of dropout_add_rmsnorm_fwd.
 *   h              the forward's residual_out (inv is computed from it again)
 *   dout           gradient of out
 *   dresidual_out  gradient of residual_out from later layers; NULL: zero
 * With xh = h * inv and g = dout * weight:
 *   dresidual = dresidual_out + inv * (g - xh * mean(g * xh))
 *   dx        = dropout(the unrounded dresidual); NULL: not written
 *   dweight   = sum over rows of dout * xh, [hidden] fp32; NULL: not
 *               computed, and no workspace is needed
 * dx and dresidual may each be exactly dout, dresidual_out or h.  Shapes as
 * in the forward; dweight 4-byte aligned; n_rows == 0 writes zeros to
 * dweight.
 */
dradd_status dropout_add_rmsnorm_bwd(void* dx, void* dresidual, float* dweight, const void* dout,
                                     const void* dresidual_out, const void* h, const void* weight, float eps,
                                     int64_t n_rows, int64_t hidden, const dradd_dropout* drop, int dtype,
                                     void* workspace, size_t workspace_bytes, cudaStream_t stream);

/*
 * add_rmsnorm_bwd -- gradients of add_rmsnorm_fwd: the same without dropout,
 * where x and residual share one gradient, dh.  With dresidual_out NULL and
 * h = x it is the gradient of rmsnorm_fwd.
 */
dradd_status add_rmsnorm_bwd(void* dh, float* dweight, const void* dout, const void* dresidual_out, const void* h,
                             const void* weight, float eps, int64_t n_rows, int64_t hidden, int dtype,
                             void* workspace, size_t workspace_bytes, cudaStream_t stream);

/* Bytes of workspace the two calls above need for a dweight (0 for an
 * invalid shape). */
size_t rmsnorm_bwd_workspace_bytes(int64_t n_rows, int64_t hidden, int dtype);

/*
 * Rotary positions.
 *
 * A tensor of heads: element (b, s, head, i) at
 * data[b * batch_stride + s * seq_stride + head * head_stride + i], so q and
 * k may be slices of one packed projection, and heads may come before or
 * after the sequence.
 */
typedef struct dradd_heads {
    void* data;
    int64_t batch_stride, seq_stride, head_stride; /* elements, >= 0 */
} dradd_heads;

/*
 * How q and k turn.  With theta = position * inv_freq[i], i < rot_dim / 2,
 * the pair (a, b) becomes scale * (a cos theta - b sin theta,
 * a sin theta + b cos theta); it is columns (i, i + rot_dim / 2) of a head,
 * or (2 i, 2 i + 1) when interleaved.  Columns from rot_dim on pass (a NaN as
 * some NaN).
 *   batch, seq, q_heads, k_heads, head_dim  k_heads may be 0: no k, whose
 *                tensors and weight are then not looked at
 *                (batch * seq < 2^31, at most 65536 heads a side)
 *   rot_dim      even, 2 <= rot_dim <= head_dim
 *   inv_freq     device double[rot_dim / 2], radians per position, finite
 *                (rope_frequencies makes the usual ones)
 *   positions    device int64[batch * seq], any values; NULL: the position
 *                of (b, s) is position0 + s
 *   scale        finite
 * head_dim <= 512, and ceil(rot_dim / 16) + ceil((head_dim - rot_dim) / 16)
 * <= 32 (every head_dim <= 496).
 * An angle, reduced to half a turn either way, is off by at most |position| *
 * 2^-53 turns (where |inv_freq| <= 1) plus 2^-32, and is then rounded to fp32
 * (2^-26 turns at most).  The first two are absolute: the sine of an angle
 * next to zero does not have fp32's relative precision.
 * Heads of whole 16-byte vectors (8 divides head_dim, the strides and, in the
 * halves layout, rot_dim / 2; 16-byte aligned tensors) take the fast path.
 */
typedef struct dradd_rope {
    int64_t batch, seq, q_heads, k_heads, head_dim, rot_dim;
    int interleaved;
    const double* inv_freq;
    const int64_t* positions;
    int64_t position0;
    float scale;
} dradd_rope;

/*
 * rope_fwd -- q_out = turned q, k_out = turned k.  rope_bwd turns by -theta:
 * the gradient of rope_fwd, given the gradients of q_out and k_out (and its
 * inverse when scale is 1).  An output may be exactly its own input; then
 * the columns from rot_dim on are not written (interleaved: those from the
 * next multiple of 16 on; between, they are written with what they hold).  An
 * output must not overlap itself (a stride of 0 with more than one element).
 */
dradd_status rope_fwd(const dradd_heads* q_out, const dradd_heads* k_out, const dradd_heads* q,
                      const dradd_heads* k, const dradd_rope* rope, int dtype, cudaStream_t stream);
dradd_status rope_bwd(const dradd_heads* dq, const dradd_heads* dk, const dradd_heads* dq_out,
                      const dradd_heads* dk_out, const dradd_rope* rope, int dtype, cudaStream_t stream);

/*
 * qk_rmsnorm_rope_fwd -- RMSNorm of every head of q and k (weights
 * [head_dim], shared by the heads of one side), then the rotation, in one
 * pass with one rounding: z = (x * inv) * weight in fp32, out = turned z.
 * inv = 1 / sqrt(mean(x^2) + eps) over the head_dim columns, within a few
 * fp32 roundings (not the correctly rounded one of dradd.h's rows).
 */
dradd_status qk_rmsnorm_rope_fwd(const dradd_heads* q_out, const dradd_heads* k_out, const dradd_heads* q,
                                 const dradd_heads* k, const void* q_weight, const void* k_weight, float q_eps,
                                 float k_eps, const dradd_rope* rope, int dtype, cudaStream_t stream);

/*
 * qk_rmsnorm_rope_bwd -- its gradients from dq_out and dk_out: with
 * g = dq_out turned by -theta, xh = q * inv:
 *   dq        = inv * (g * w - xh * mean(g * w * xh))
 *   dq_weight = sum over tokens and heads of g * xh, [head_dim] fp32
 * and the same for k.  dq may be exactly q or dq_out, dk exactly k or
 * dk_out.  dq_weight and dk_weight both NULL: not computed, no workspace.
 * With k_heads == 0 a dk_weight is set to zeros.
 */
dradd_status qk_rmsnorm_rope_bwd(const dradd_heads* dq, const dradd_heads* dk, float* dq_weight, float* dk_weight,
                                 const dradd_heads* dq_out, const dradd_heads* dk_out, const dradd_heads* q,
                                 const dradd_heads* k,
                                 const void* q_weight, const void* k_weight, float q_eps, float k_eps,
                                 const dradd_rope* rope, int dtype, void* workspace, size_t workspace_bytes,
                                 cudaStream_t stream);

/* Bytes of workspace qk_rmsnorm_rope_bwd needs for its weight gradients (0
 * for an invalid shape). */
size_t qk_rmsnorm_rope_bwd_workspace_bytes(const dradd_rope* rope, int dtype);

/*
 * rope_frequencies -- inv_freq on the host, out[i] for i < rot_dim / 2, with
 * f_i = base^(-2 i / rot_dim):
 *   DRADD_ROPE_PLAIN     f_i
 *   DRADD_ROPE_LINEAR    f_i / factor (positions interpolated)
 *   DRADD_ROPE_BASE      the base enlarged to base * factor^(d / (d - 2)),
 *                        d = rot_dim > 2: the slowest pair is stretched by
 *                        factor, the fastest not at all
 *   DRADD_ROPE_BY_PARTS  f_i * (r + (1 - r) / factor), r = clamp((n_i - low)
 *                        / (high - low), 0, 1), n_i = original_length * f_i
 *                        / (2 pi) the turns pair i makes within the original
 *                        length: pairs of more than `high` turns stay, those
 *                        of fewer than `low` are interpolated
 * base > 0, factor >= 1, original_length > 0 and low < high where used, all
 * finite; else DRADD_ERR_BAD_ARG.
 */
enum { DRADD_ROPE_PLAIN = 0, DRADD_ROPE_LINEAR = 1, DRADD_ROPE_BASE = 2, DRADD_ROPE_BY_PARTS = 3 };
dradd_status rope_frequencies(double* out, int64_t rot_dim, double base, int scaling, double factor,
                              double original_length, double low, double high);

#ifdef __cplusplus
}
#endif

#endif /* DRADD_TRAIN_H */
