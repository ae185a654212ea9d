/*
 * dradd_linear.h -- matrix products with what stands next to them in a model
 * fused behind them:
 *   - a layer's product with bias, activation and the residual add, which
 *     makes the rows that residual-add + RMSNorm (dradd.h) takes, and its
 *     gradients;
 *   - softmax cross entropy of a token's logits x W^T, which are never kept,
 *     and its gradients;
 *   - the divergence of those logits' softmax from a teacher's top logits,
 *     and its gradients.
 *
 * The conventions of dradd.h and dradd_train.h hold (caller's buffers,
 * asynchronous on `stream`, argument errors before any GPU work, workspaces),
 * with these additions:
 *   - dtype: DRADD_BF16 or DRADD_F16, the type of every tensor declared
 *     void*.  Products are summed in fp32 by the tensor cores, which cut off
 *     what does not fit instead of rounding it: a sum of k terms is off by at
 *     most (k / 16 + 32) 2^-23 of the sum of their magnitudes, and comes out
 *     nearer to 0 by about 1e-9 k of its size.  The logits of the losses
 *     and of their gradients are taken out after every 512 terms and joined by
 *     rounded additions.  Each stored element is rounded once.  The gradients pass
 *     through dz, the gradient of the product's output, which is rounded to
 *     dtype before it is multiplied again (the losses' in fp16 at a power of
 *     two that puts the largest factor of a row between 2^13 and 2^14).  Calls
 *     whose tiles (128 x 256) would be more than 2^30 are DRADD_ERR_BAD_SHAPE.
 *   - Tensors are device memory, 16-byte aligned; rows have unit column
 *     stride and a row stride that is a multiple of 8 elements.  Inner
 *     dimensions (and the columns of linear_act_add) are multiples of 8.
 *   - No output may overlap an input, another output or the workspace,
 *     except that `out` of linear_act_add_fwd may be exactly `residual`.
 *   - How a call is tiled and its sums are split depends on its shape alone:
 *     equal calls give equal bits.  A row's bits may depend on the number of
 *     rows.
 */
#ifndef DRADD_LINEAR_H
#define DRADD_LINEAR_H

#include <stddef.h>

#include "dradd_train.h"

#ifdef __cplusplus
extern "C" {
#endif

enum {
    DRADD_ACT_NONE = 0,
    DRADD_ACT_RELU = 1,
    DRADD_ACT_GELU = 2,      /* z Phi(z)                                             */
    DRADD_ACT_GELU_TANH = 3, /* z / (1 + e^(-2 u)), u = sqrt(2 / pi) (z + 0.044715 z^3) */
    DRADD_ACT_SILU = 4       /* z / (1 + e^-z)                                       */
};

/* A matrix: element (i, j) at data[i * stride + j]. */
typedef struct dradd_matrix {
    void* data;
    int64_t stride;
} dradd_matrix;

/*
 * linear_act_add_fwd -- out = residual + act(x W^T + bias), one rounding.
 *   x         [rows, inner]
 *   weight    [cols, inner]
 *   bias      [cols] or NULL
 *   residual  [rows, cols], its data NULL or the pointer NULL: none
 *   rows <= 2^31 - 4096, 8 <= inner, cols < 2^24, both multiples of 8
 * Workspace: linear_act_add_fwd_workspace_bytes (may be 0).
 */
dradd_status linear_act_add_fwd(const dradd_matrix* out, const dradd_matrix* x, const dradd_matrix* weight,
                                const void* bias, const dradd_matrix* residual, int act, int64_t rows,
                                int64_t inner, int64_t cols, int dtype, void* workspace, size_t workspace_bytes,
                                cudaStream_t stream);
size_t linear_act_add_fwd_workspace_bytes(int64_t rows, int64_t inner, int64_t cols);

/*
 * linear_act_add_bwd -- its gradients from dout (the residual's is dout):
 *   dz      = dout * act'(x W^T + bias), the product computed again (not for
 *             DRADD_ACT_NONE, where dz is dout)
 *   dx      = dz W           [rows, inner], or NULL
 *   dweight = dz^T x         [cols, inner], contiguous, or NULL
 *   dbias   = sum over rows of dz, [cols], or NULL
 * dx contiguous.  relu's derivative at 0 is 0.  rows == 0 sets dweight and
 * dbias to zeros.
 */
dradd_status linear_act_add_bwd(void* dx, void* dweight, void* dbias, const dradd_matrix* dout,
                                const dradd_matrix* x, const dradd_matrix* weight, const void* bias, int act,
                                int64_t rows, int64_t inner, int64_t cols, int dtype, void* workspace,
                                size_t workspace_bytes, cudaStream_t stream);
size_t linear_act_add_bwd_workspace_bytes(int64_t rows, int64_t inner, int64_t cols, int act, int want_dx,
                                          int want_dweight, int want_dbias);

/*
 * linear_cross_entropy_fwd -- with z = x W^T, W [vocab, hidden]:
 *   lse[t]  = log sum over v of exp(z[t, v])
 *   loss[t] = lse[t] - z[t, target[t]]; 0 where target[t] is ignore_index;
 *             NaN where it is neither that nor a word
 * both fp32 [rows]; target int64 [rows].  Logits that are not finite make
 * their own row's results infinite or NaN.
 *   rows <= 2^31 - 4096, 8 <= hidden < 2^24 a multiple of 8, 1 <= vocab <= 2^30
 */
dradd_status linear_cross_entropy_fwd(float* loss, float* lse, const dradd_matrix* x, const dradd_matrix* weight,
                                      const int64_t* target, int64_t ignore_index, int64_t rows, int64_t hidden,
                                      int64_t vocab, int dtype, void* workspace, size_t workspace_bytes,
                                      cudaStream_t stream);
size_t linear_cross_entropy_fwd_workspace_bytes(int64_t rows, int64_t hidden, int64_t vocab);

/*
 * linear_cross_entropy_bwd -- its gradients, from those of loss and lse and
 * from the forward's lse:
 *   dz[t, v] = (dloss[t] + dlse[t]) exp(z[t, v] - lse[t]) - dloss[t] [v = target[t]]
 * with dloss[t] = 0 where the target is ignored;
 *   dx      = dz W    [rows, hidden] contiguous, or NULL
 *   dweight = dz^T x  [vocab, hidden] contiguous, or NULL
 * dloss_stride and dlse_stride are 0 (one value for all rows) or 1; dlse
 * NULL: zero.  The vocabulary is taken in pieces, whose dz are held in the
 * workspace one at a time: at most 256 MB, and 256 words at least.  dx's sums
 * are read and written for every piece, so from some 65536 rows on several
 * calls are faster.  A row whose two factors are 0 (an ignored token
 * without dlse, a loss masked by its dloss) adds nothing to dweight and has
 * a zero dx, whatever its x and lse hold.
 */
dradd_status linear_cross_entropy_bwd(void* dx, void* dweight, const float* dloss, int64_t dloss_stride,
                                      const float* dlse, int64_t dlse_stride, const dradd_matrix* x,
                                      const dradd_matrix* weight, const int64_t* target, int64_t ignore_index,
                                      const float* lse, int64_t rows, int64_t hidden, int64_t vocab, int dtype,
                                      void* workspace, size_t workspace_bytes, cudaStream_t stream);
size_t linear_cross_entropy_bwd_workspace_bytes(int64_t rows, int64_t hidden, int64_t vocab);

/*
 * A teacher's likeliest words: index int64 [rows, top], logits [rows, top] of
 * logits_dtype (any of the three), both contiguous, 1 <= top <= 1024.  An
 * entry with a negative index is empty; a row of empty entries (or of logits
 * -infinity alone) is not counted; an index of vocab or more makes the row
 * NaN.  A word may be listed more than once.  temperature: finite, > 0.
 */
typedef struct dradd_teacher {
    const int64_t* index;
    const void* logits;
    int logits_dtype;
    int64_t top;
    float temperature;
} dradd_teacher;

/*
 * linear_distill_fwd -- with z = x W^T / temperature, and q the softmax of a
 * row's teacher logits / temperature over its entries:
 *   lse[t]  = log sum over v of exp(z[t, v])
 *   loss[t] = sum over k of q[t, k] (log q[t, k] - z[t, index[t, k]] + lse[t]),
 *             the divergence of the student's softmax from q; 0 in rows that
 *             are not counted
 * (no factor temperature^2).
 */
dradd_status linear_distill_fwd(float* loss, float* lse, const dradd_matrix* x, const dradd_matrix* weight,
                                const dradd_teacher* teacher, int64_t rows, int64_t hidden, int64_t vocab,
                                int dtype, void* workspace, size_t workspace_bytes, cudaStream_t stream);
size_t linear_distill_fwd_workspace_bytes(int64_t rows, int64_t hidden, int64_t vocab, int64_t top);

/*
 * linear_distill_bwd -- its gradients with respect to x and weight:
 *   dz[t, v] = ((dloss[t] + dlse[t]) exp(z[t, v] - lse[t])
 *               - dloss[t] sum over k of q[t, k] [index[t, k] = v]) / temperature
 * with the rest as in linear_cross_entropy_bwd.
 */
dradd_status linear_distill_bwd(void* dx, void* dweight, const float* dloss, int64_t dloss_stride,
                                const float* dlse, int64_t dlse_stride, const dradd_matrix* x,
                                const dradd_matrix* weight, const dradd_teacher* teacher, const float* lse,
                                int64_t rows, int64_t hidden, int64_t vocab, int dtype, void* workspace,
                                size_t workspace_bytes, cudaStream_t stream);
size_t linear_distill_bwd_workspace_bytes(int64_t rows, int64_t hidden, int64_t vocab, int64_t top);

#ifdef __cplusplus
}
#endif

#endif /* DRADD_LINEAR_H */
