"""Binding of include/dradd_train.h: dropout, the gradients of residual-add +
RMSNorm, and rotary positions with and without the q/k RMSNorm.

As in the package's other entry points these functions only check and
marshal arguments; the work is done by the kernels of libdradd.so.  Tensors
are bf16, fp16 or fp32, one type per call.  What a call allocates (outputs
not given, the workspace of weight gradients) it allocates on the stream it
launches on.

A dropout mask is a function of (seed, offset, row, column), row and column
those of the tensor seen as [rows, last dimension]; forward and backward
take the same seed and offset.  `step` is an optional device int64 that the
kernel adds to the offset, so that a captured graph draws a new mask at
every replay when the program advances it in between.  Calls of equal
offset + step have one mask, so with layers at the offsets 0 .. L - 1 it has
to advance by L a replay (or the offsets lie 2^32 apart).

Results carry no autograd graph, whatever their inputs require: a program's
own torch.autograd.Function calls a forward and its gradient.

Checks, allocations and calls are one compiled function each
(csrc/dradd_binding.cpp): a decode step's kernels take two or three
microseconds, less than the same in Python.
"""
from __future__ import annotations

import contextlib
import ctypes

ROPE_SCALINGS = {"none": 0, "linear": 1, "base": 2, "by_parts": 3}

_C = None  # the compiled part, loaded with the first call


def _load():
    global _C
    from . import lib
    lib()  # says how to build where nothing is built
    try:
        from . import _binding
    except ImportError as e:
        raise RuntimeError("the compiled binding does not load: build it with `python -m "
                           "deterministic_residual_add_gb300.build` (needs g++, Python's headers and a torch with "
                           f"CUDA): {e}") from e
    _C = _binding
    return _C


def _bind(L):
    """Argument types of the entry points called through ctypes."""
    f64 = ctypes.c_double
    L.rope_frequencies.argtypes = [ctypes.c_void_p, ctypes.c_int64, f64, ctypes.c_int, f64, f64, f64, f64]
    L.rope_frequencies.restype = ctypes.c_int
    L.rmsnorm_bwd_workspace_bytes.argtypes = [ctypes.c_int64, ctypes.c_int64, ctypes.c_int]
    L.rmsnorm_bwd_workspace_bytes.restype = ctypes.c_size_t
    L.qk_rmsnorm_rope_bwd_workspace_bytes.argtypes = [ctypes.c_void_p, ctypes.c_int]
    L.qk_rmsnorm_rope_bwd_workspace_bytes.restype = ctypes.c_size_t


@contextlib.contextmanager
def _on(x, stream):
    """The launch stream current; a call launches on the current stream of
    its tensors' device."""
    import torch  # here, as elsewhere in the package: the library and its build do without
    if not x.is_cuda:
        raise ValueError("tensors must be CUDA tensors")
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, x.device)
    if stream.device != x.device:
        raise ValueError(f"the stream is on {stream.device}, the tensors on {x.device}")
    with torch.cuda.stream(stream):
        yield


# ------------------------------------------------------------------ dropout
def dropout_fwd(x, p: float, *, seed: int, offset: int = 0, step=None, out=None, stream=None):
    """out = x where kept, times 1 / (1 - p) (p applied in steps of 2^-16),
    and 0 where dropped.  The gradient is the same call on the gradient.
    x: contiguous, or 2-D with any row stride; out may be x."""
    if stream is not None:
        with _on(x, stream):
            return dropout_fwd(x, p, seed=seed, offset=offset, step=step, out=out)
    return (_C or _load()).dropout(x, None, p, seed, offset, step, out)


def dropout_add_fwd(x, residual, p: float, *, seed: int, offset: int = 0, step=None, residual_out=None, stream=None):
    """residual_out = residual + dropout(x), rounded once.  Gradients:
    dresidual = dy, dx = dropout_fwd(dy) with the same p, seed and offset.
    residual_out may be x or residual."""
    if stream is not None:
        with _on(x, stream):
            return dropout_add_fwd(x, residual, p, seed=seed, offset=offset, step=step, residual_out=residual_out)
    if residual is None:
        raise TypeError("residual must be a tensor (got None)")
    return (_C or _load()).dropout(x, residual, p, seed, offset, step, residual_out)


# ------------------------------------- dropout + residual add + RMSNorm
def dropout_add_rmsnorm_fwd(x, residual, weight, p: float, eps: float = 1e-6, *, seed: int, offset: int = 0, step=None,
                            out=None, residual_out=None, stream=None):
    """(out, residual_out) of add_rmsnorm_fwd with dropout on x: acc =
    residual + dropout(x), residual_out = rne(acc), out = rne(acc / rms *
    weight).  With p = 0 the bits are add_rmsnorm_fwd's.  Contiguous
    [..., hidden] tensors, hidden a multiple of 8; out and residual_out may
    each be x or residual."""
    if stream is not None:
        with _on(x, stream):
            return dropout_add_rmsnorm_fwd(x, residual, weight, p, eps, seed=seed, offset=offset, step=step, out=out,
                                           residual_out=residual_out)
    return (_C or _load()).drop_norm_fwd(x, residual, weight, p, eps, seed, offset, step, out, residual_out)


def dropout_add_rmsnorm_bwd(dout, dresidual_out, residual_out, weight, p: float, eps: float = 1e-6, *, seed: int,
                            offset: int = 0, step=None, dx=None, dresidual=None, dweight=None, weight_grad: bool = True,
                            workspace=None, stream=None):
    """(dx, dresidual, dweight): gradients of dropout_add_rmsnorm_fwd from
    those of its two outputs (dresidual_out None: zero) and its residual_out.
    dweight is fp32, None with weight_grad=False.  dx and dresidual may each
    be dout, dresidual_out or residual_out.  workspace: a tensor of at least
    rmsnorm_bwd_workspace_bytes (C ABI); by default one is allocated."""
    if stream is not None:
        with _on(residual_out, stream):
            return dropout_add_rmsnorm_bwd(dout, dresidual_out, residual_out, weight, p, eps, seed=seed, offset=offset,
                                           step=step, dx=dx, dresidual=dresidual, dweight=dweight,
                                           weight_grad=weight_grad, workspace=workspace)
    return (_C or _load()).drop_norm_bwd(dout, dresidual_out, residual_out, weight, True, p, eps, seed, offset, step, dx,
                                         dresidual, dweight, weight_grad, workspace)


def add_rmsnorm_bwd(dout, dresidual_out, residual_out, weight, eps: float = 1e-6, *, dh=None, dweight=None,
                    weight_grad: bool = True, workspace=None, stream=None):
    """(dh, dweight): gradients of add_rmsnorm_fwd; dh is that of x and of
    residual.  Arguments as in dropout_add_rmsnorm_bwd."""
    if stream is not None:
        with _on(residual_out, stream):
            return add_rmsnorm_bwd(dout, dresidual_out, residual_out, weight, eps, dh=dh, dweight=dweight,
                                   weight_grad=weight_grad, workspace=workspace)
    return (_C or _load()).drop_norm_bwd(dout, dresidual_out, residual_out, weight, False, 0.0, eps, 0, 0, None, None,
                                         dh, dweight, weight_grad, workspace)[1:]


def rmsnorm_bwd(dout, x, weight, eps: float = 1e-6, **kw):
    """(dx, dweight): gradients of rmsnorm_fwd, and in fp16 and fp32, which
    that call does not take, of dropout_add_rmsnorm_fwd with p = 0 and a
    residual of zeros.  Keywords as in add_rmsnorm_bwd."""
    return add_rmsnorm_bwd(dout, None, x, weight, eps, **kw)


# ------------------------------------------------------------------- rotary
def rope_frequencies(rot_dim: int, base: float = 10000.0, *, scaling: str = "none", factor: float = 1.0,
                     original_length: float = 0.0, low: float = 1.0, high: float = 32.0, device=None):
    """Radians per position of the rot_dim / 2 pairs, float64:
    base^(-2 i / rot_dim), stretched for contexts `factor` times longer by
    scaling "linear" (all pairs / factor), "base" (an enlarged base) or
    "by_parts" (pairs that make more than `high` turns within
    original_length stay, those that make fewer than `low` are divided by
    factor, those between are blended)."""
    import torch
    from . import DraddError, lib
    if scaling not in ROPE_SCALINGS:
        raise ValueError(f"scaling must be one of {sorted(ROPE_SCALINGS)}")
    f = torch.empty(max(int(rot_dim) // 2, 1), dtype=torch.float64)
    st = lib().rope_frequencies(f.data_ptr(), int(rot_dim), float(base), ROPE_SCALINGS[scaling], float(factor),
                                float(original_length), float(low), float(high))
    if st:
        raise DraddError(st, "rope_frequencies")
    return f if device is None else f.to(device)


def rope_fwd(q, k, inv_freq, positions=None, *, position0: int = 0, interleaved: bool = False, scale: float = 1.0,
             q_out=None, k_out=None, stream=None):
    """(q_out, k_out): q and k turned by position * inv_freq.

    q, k: [batch, seq, heads, head_dim] with any strides but a unit last one
    (slices of a packed projection, or a transposed [batch, heads, seq,
    head_dim]); k may be None.  The first 2 * len(inv_freq) columns turn, in
    pairs (i, i + half) or, interleaved, (2 i, 2 i + 1).  inv_freq: float64
    (rope_frequencies).  positions: int64 [batch, seq], else position0 + s.
    Outputs are contiguous unless given; each may be its own input."""
    if stream is not None:
        with _on(q, stream):
            return rope_fwd(q, k, inv_freq, positions, position0=position0, interleaved=interleaved, scale=scale,
                            q_out=q_out, k_out=k_out)
    return (_C or _load()).rope(False, q, k, inv_freq, positions, position0, interleaved, scale, q_out, k_out)


def rope_bwd(dq_out, dk_out, inv_freq, positions=None, *, position0: int = 0, interleaved: bool = False,
             scale: float = 1.0, dq=None, dk=None, stream=None):
    """(dq, dk): the gradient of rope_fwd, a turn by the opposite angles."""
    if stream is not None:
        with _on(dq_out, stream):
            return rope_bwd(dq_out, dk_out, inv_freq, positions, position0=position0, interleaved=interleaved,
                            scale=scale, dq=dq, dk=dk)
    return (_C or _load()).rope(True, dq_out, dk_out, inv_freq, positions, position0, interleaved, scale, dq, dk)


def qk_rmsnorm_rope_fwd(q, k, q_weight, k_weight, inv_freq, q_eps: float = 1e-6, k_eps: float = 1e-6, *,
                        positions=None, position0: int = 0, interleaved: bool = False, scale: float = 1.0, q_out=None,
                        k_out=None, stream=None):
    """(q_out, k_out): RMSNorm of every head of q and k (weights [head_dim]),
    then rope_fwd, in one pass with one rounding.  k and k_weight may be
    None."""
    if stream is not None:
        with _on(q, stream):
            return qk_rmsnorm_rope_fwd(q, k, q_weight, k_weight, inv_freq, q_eps, k_eps, positions=positions,
                                       position0=position0, interleaved=interleaved, scale=scale, q_out=q_out,
                                       k_out=k_out)
    return (_C or _load()).norm_rope_fwd(q, k, q_weight, k_weight, q_eps, k_eps, inv_freq, positions, position0,
                                         interleaved, scale, q_out, k_out)


def qk_rmsnorm_rope_bwd(dq_out, dk_out, q, k, q_weight, k_weight, inv_freq, q_eps: float = 1e-6, k_eps: float = 1e-6,
                        *, positions=None, position0: int = 0, interleaved: bool = False, scale: float = 1.0, dq=None,
                        dk=None, dq_weight=None, dk_weight=None, weight_grad: bool = True, workspace=None,
                        stream=None):
    """(dq, dk, dq_weight, dk_weight): gradients of qk_rmsnorm_rope_fwd; the
    weights' are fp32, None with weight_grad=False.  dq may be q or dq_out,
    dk may be k or dk_out.  workspace: a tensor of at least
    qk_rmsnorm_rope_bwd_workspace_bytes (C ABI); by default one is
    allocated."""
    if stream is not None:
        with _on(q, stream):
            return qk_rmsnorm_rope_bwd(dq_out, dk_out, q, k, q_weight, k_weight, inv_freq, q_eps, k_eps,
                                       positions=positions, position0=position0, interleaved=interleaved, scale=scale,
                                       dq=dq, dk=dk, dq_weight=dq_weight, dk_weight=dk_weight, weight_grad=weight_grad,
                                       workspace=workspace)
    return (_C or _load()).norm_rope_bwd(dq_out, dk_out, q, k, q_weight, k_weight, q_eps, k_eps, inv_freq, positions,
                                         position0, interleaved, scale, dq, dk, dq_weight, dk_weight, weight_grad,
                                         workspace)
