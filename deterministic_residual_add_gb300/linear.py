"""Binding of include/dradd_linear.h: matrix products with bias, activation
and residual, and the losses of logits that are never kept.

As in train.py these functions only name their arguments; checks, allocations
and calls are one compiled function each (csrc/dradd_binding.cpp).  Tensors
are bf16 or fp16, one type per call: rows with unit column stride, contiguous
or 2-D with a row stride that is a multiple of 8, on 16-byte boundaries.
What a call allocates (outputs not given, its workspace) it allocates on the
stream it launches on; a workspace of one's own has the size that the C ABI's
query states, and serves one call at a time.

Results carry no autograd graph, whatever their inputs require: a program's
own torch.autograd.Function calls a forward and its gradient.
"""
from __future__ import annotations

from . import train

ACTIVATIONS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}


def _act(activation) -> int:
    try:
        return ACTIVATIONS[activation]
    except (KeyError, TypeError):
        raise ValueError(f"activation must be one of {sorted(ACTIVATIONS)} (got {activation!r})") from None


# ------------------------------------------- bias, activation and residual
def linear_act_add_fwd(x, weight, bias=None, residual=None, *, activation: str = "none", out=None, workspace=None,
                       stream=None):
    """out = residual + activation(x weight^T + bias), summed in fp32 and
    rounded once.

    x: [..., inner], weight: [cols, inner], bias: [cols], residual and out:
    [..., cols]; inner and cols multiples of 8.  out may be residual.
    activation: one of ACTIVATIONS ("gelu" by the error function, "gelu_tanh"
    its usual approximation)."""
    if stream is not None:
        with train._on(x, stream):
            return linear_act_add_fwd(x, weight, bias, residual, activation=activation, out=out, workspace=workspace)
    return (train._C or train._load()).linear_fwd(x, weight, bias, residual, _act(activation), out, workspace)


def linear_act_add_bwd(dout, x, weight, bias=None, *, activation: str = "none", dx=None, dweight=None, dbias=None,
                       input_grad: bool = True, weight_grad: bool = True, workspace=None, stream=None):
    """(dx, dweight, dbias): gradients of linear_act_add_fwd; the residual's
    is dout.

    x weight^T + bias is computed again where the activation's derivative
    needs it.  dbias is None without a bias; dx is None with input_grad=False,
    dweight and dbias with weight_grad=False.  The gradient of x weight^T +
    bias is rounded to the tensors' type before it is multiplied again."""
    if stream is not None:
        with train._on(x, stream):
            return linear_act_add_bwd(dout, x, weight, bias, activation=activation, dx=dx, dweight=dweight,
                                      dbias=dbias, input_grad=input_grad, weight_grad=weight_grad,
                                      workspace=workspace)
    return (train._C or train._load()).linear_bwd(dout, x, weight, bias, _act(activation), dx, dweight, dbias,
                                                  input_grad, weight_grad, workspace)


# ------------------------------------------------------------ cross entropy
def linear_cross_entropy_fwd(x, weight, target, *, ignore_index: int = -100, loss=None, lse=None, workspace=None,
                             stream=None):
    """(loss, lse) of the logits z = x weight^T, which are not kept: lse =
    logsumexp(z), loss = lse - z[target], fp32, one of each for a row of x.

    x: [..., hidden], weight: [vocab, hidden], target: int64 [...].  The loss
    is 0 where the target is ignore_index, NaN where it is no word."""
    if stream is not None:
        with train._on(x, stream):
            return linear_cross_entropy_fwd(x, weight, target, ignore_index=ignore_index, loss=loss, lse=lse,
                                            workspace=workspace)
    return (train._C or train._load()).loss_fwd(x, weight, target, None, ignore_index, 1.0, loss, lse, workspace)


def linear_cross_entropy_bwd(dloss, dlse, x, weight, target, lse, *, ignore_index: int = -100, dx=None, dweight=None,
                             input_grad: bool = True, weight_grad: bool = True, workspace=None, stream=None):
    """(dx, dweight): gradients of linear_cross_entropy_fwd from those of
    loss and lse (dlse None: zero) and its lse.

    dloss, dlse: fp32 [...], contiguous or one value for all rows (an expanded
    or a 0-dimensional tensor).  The logits are computed again, a piece of the
    vocabulary at a time; from some 65536 rows on, calls over parts of them
    (and the sum of their dweights) are faster.  Rows whose dloss (0 where ignored) and dloss + dlse
    are both 0 count for nothing, whatever x and lse hold there."""
    if stream is not None:
        with train._on(x, stream):
            return linear_cross_entropy_bwd(dloss, dlse, x, weight, target, lse, ignore_index=ignore_index, dx=dx,
                                            dweight=dweight, input_grad=input_grad, weight_grad=weight_grad,
                                            workspace=workspace)
    return (train._C or train._load()).loss_bwd(dloss, dlse, x, weight, target, None, ignore_index, 1.0, lse, dx,
                                                dweight, input_grad, weight_grad, workspace)


# ------------------------------------------------------------- distillation
def _needs_logits(teacher_logits):
    if teacher_logits is None:
        raise TypeError("teacher_logits must be a tensor (got None)")


def linear_distill_fwd(x, weight, teacher_index, teacher_logits, *, temperature: float = 1.0, loss=None, lse=None,
                       workspace=None, stream=None):
    """(loss, lse) of z = x weight^T / temperature, which is not kept: lse =
    logsumexp(z), and loss = sum of q (log q - z[index] + lse), the divergence
    of softmax(z) from q = softmax(teacher_logits / temperature) over the
    teacher's entries (no factor temperature^2).

    teacher_index: int64 [..., top], teacher_logits: bf16, fp16 or fp32 [...,
    top], top <= 1024.  An entry with a negative index is empty; a row without
    entries has loss 0.  An index that is no word makes its row NaN."""
    if stream is not None:
        with train._on(x, stream):
            return linear_distill_fwd(x, weight, teacher_index, teacher_logits, temperature=temperature, loss=loss,
                                      lse=lse, workspace=workspace)
    _needs_logits(teacher_logits)
    return (train._C or train._load()).loss_fwd(x, weight, teacher_index, teacher_logits, 0, temperature, loss, lse,
                                                workspace)


def linear_distill_bwd(dloss, dlse, x, weight, teacher_index, teacher_logits, lse, *, temperature: float = 1.0,
                       dx=None, dweight=None, input_grad: bool = True, weight_grad: bool = True, workspace=None,
                       stream=None):
    """(dx, dweight): gradients of linear_distill_fwd with respect to x and
    weight; arguments as in linear_cross_entropy_bwd."""
    if stream is not None:
        with train._on(x, stream):
            return linear_distill_bwd(dloss, dlse, x, weight, teacher_index, teacher_logits, lse,
                                      temperature=temperature, dx=dx, dweight=dweight, input_grad=input_grad,
                                      weight_grad=weight_grad, workspace=workspace)
    _needs_logits(teacher_logits)
    return (train._C or train._load()).loss_bwd(dloss, dlse, x, weight, teacher_index, teacher_logits, 0, temperature,
                                                lse, dx, dweight, input_grad, weight_grad, workspace)
