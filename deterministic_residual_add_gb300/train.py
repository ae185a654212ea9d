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
every replay when the program advances it in between.

A decode step's kernels take a few microseconds, less than a call's host
side, so that side is kept short: one chain of tests per tensor, the C
structures packed as bytes, and stream and device switched (_switched) only
where they are not current already.
"""
from __future__ import annotations

import contextlib
import ctypes
import struct

import torch

ROPE_SCALINGS = {"none": 0, "linear": 1, "base": 2, "by_parts": 3}

_vp, _i64, _f32, _f64, _int, _size = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_float, ctypes.c_double, ctypes.c_int,
                                      ctypes.c_size_t)
_DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
_U64 = 0xFFFFFFFFFFFFFFFF

# dradd_dropout, dradd_heads and dradd_rope of the header, natively aligned
_pack_dropout = struct.Struct("fQQP").pack
_pack_heads = struct.Struct("Pqqq").pack
_pack_rope = struct.Struct("6qiPPqf0q").pack

_raw_stream = torch._C._cuda_getCurrentRawStream if hasattr(torch._C, "_cuda_getCurrentRawStream") else (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = torch.cuda.current_device

_L = None


def _bind(L):
    """Argument types of the entry points, set once when the library loads."""
    global _L
    for name, args in [
            ("dropout_fwd", [_vp, _i64, _vp, _i64, _i64, _i64, _vp, _int, _vp]),
            ("dropout_add_fwd", [_vp, _i64, _vp, _i64, _vp, _i64, _i64, _i64, _vp, _int, _vp]),
            ("dropout_add_rmsnorm_fwd", [_vp] * 5 + [_f32, _i64, _i64, _vp, _int, _vp]),
            ("dropout_add_rmsnorm_bwd", [_vp] * 7 + [_f32, _i64, _i64, _vp, _int, _vp, _size, _vp]),
            ("add_rmsnorm_bwd", [_vp] * 6 + [_f32, _i64, _i64, _int, _vp, _size, _vp]),
            ("rope_fwd", [_vp] * 5 + [_int, _vp]),
            ("rope_bwd", [_vp] * 5 + [_int, _vp]),
            ("qk_rmsnorm_rope_fwd", [_vp] * 6 + [_f32, _f32, _vp, _int, _vp]),
            ("qk_rmsnorm_rope_bwd", [_vp] * 10 + [_f32, _f32, _vp, _int, _vp, _size, _vp]),
            ("rope_frequencies", [_vp, _i64, _f64, _int, _f64, _f64, _f64, _f64])]:
        f = getattr(L, name)
        f.argtypes, f.restype = args, _int
    L.rmsnorm_bwd_workspace_bytes.argtypes, L.rmsnorm_bwd_workspace_bytes.restype = [_i64, _i64, _int], _size
    L.qk_rmsnorm_rope_bwd_workspace_bytes.argtypes = [_vp, _int]
    L.qk_rmsnorm_rope_bwd_workspace_bytes.restype = _size
    _L = L


def _lib():
    if _L is None:
        from . import lib
        lib()
    return _L


def _failed(status: int, where: str):
    from . import DraddError
    raise DraddError(status, where)


@contextlib.contextmanager
def _switched(x, stream):
    """x's device and the launch stream current; inside, a call without a
    stream takes the current one."""
    with torch.cuda.device(x.device):
        if stream is None:
            yield
            return
        if isinstance(stream, int):
            stream = torch.cuda.ExternalStream(stream, x.device)
        if stream.device != x.device:
            raise ValueError(f"the stream is on {stream.device}, the tensors on {x.device}")
        with torch.cuda.stream(stream):
            yield


# ------------------------------------------------------------------- checks
def _dtype(x, name: str) -> int:
    code = _DTYPES.get(x.dtype)
    if code is None:
        raise TypeError(f"{name} must be bfloat16, float16 or float32 (got {x.dtype})")
    if not x.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return code


def _refuse(t, name, dtype, device, shape, contiguous):
    if t.dtype is not dtype:
        raise TypeError(f"{name} must hold {dtype} (got {t.dtype})")
    if t.get_device() != device:
        raise ValueError(f"{name} is on {t.device}, expected cuda:{device}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    raise ValueError(f"{name} must have unit stride in its last dimension")


def _flat(t, name, dtype, device, shape) -> int:
    """data_ptr of a contiguous tensor of this type, device and shape."""
    if t.dtype is not dtype or t.get_device() != device or t.shape != shape or not t.is_contiguous():
        _refuse(t, name, dtype, device, shape, True)
    return t.data_ptr()


def _drop(p, seed, offset, step, device) -> bytes:
    if step is None:
        return _pack_dropout(p, seed & _U64, offset & _U64, 0)
    if step.numel() != 1:
        raise ValueError("step must hold one int64")
    return _pack_dropout(p, seed & _U64, offset & _U64, _flat(step, "step", torch.int64, device, step.shape))


# ------------------------------------------------------------------ dropout
def _rows(t, name, dtype, device, shape):
    """(data_ptr, rows, columns, row stride): a contiguous tensor as [rows,
    last dimension], or a 2-D tensor with unit column stride."""
    if t.dtype is not dtype or t.get_device() != device or t.shape != shape:
        _refuse(t, name, dtype, device, shape, False)
    if t.is_contiguous():
        cols = shape[-1] if shape else 1
        return t.data_ptr(), (t.numel() // cols if cols else 0), cols, cols
    if len(shape) != 2 or (shape[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"{name} must be contiguous, or 2-D with unit column stride")
    return t.data_ptr(), shape[0], shape[1], t.stride(0) if shape[0] > 1 else shape[1]


def dropout_fwd(x, p: float, *, seed: int, offset: int = 0, step=None, out=None, stream=None):
    """out = x where kept, times 1 / (1 - p) (p applied in steps of 2^-16),
    and 0 where dropped.  The gradient is the same call on the gradient.
    x: contiguous, or 2-D with any row stride; out may be x."""
    code, device = _dtype(x, "x"), x.get_device()
    if stream is not None or device != _current_device():
        with _switched(x, stream):
            return dropout_fwd(x, p, seed=seed, offset=offset, step=step, out=out)
    dtype, shape = x.dtype, x.shape
    xp, n, hidden, xs = _rows(x, "x", dtype, device, shape)
    if out is None:
        out = torch.empty_like(x, memory_format=torch.contiguous_format)
        op, os = out.data_ptr(), hidden
    else:
        op, _, _, os = _rows(out, "out", dtype, device, shape)
    if hidden:
        st = _lib().dropout_fwd(op, os, xp, xs, n, hidden, _drop(p, seed, offset, step, device), code,
                                _raw_stream(device))
        if st:
            _failed(st, "dropout_fwd")
    return out


def dropout_add_fwd(x, residual, p: float, *, seed: int, offset: int = 0, step=None, residual_out=None, stream=None):
    """residual_out = residual + dropout(x), rounded once.  Gradients:
    dresidual = dy, dx = dropout_fwd(dy) with the same p, seed and offset.
    residual_out may be x or residual."""
    code, device = _dtype(x, "x"), x.get_device()
    if stream is not None or device != _current_device():
        with _switched(x, stream):
            return dropout_add_fwd(x, residual, p, seed=seed, offset=offset, step=step, residual_out=residual_out)
    dtype, shape = x.dtype, x.shape
    xp, n, hidden, xs = _rows(x, "x", dtype, device, shape)
    rp, _, _, rs = _rows(residual, "residual", dtype, device, shape)
    if residual_out is None:
        residual_out = torch.empty_like(x, memory_format=torch.contiguous_format)
        op, os = residual_out.data_ptr(), hidden
    else:
        op, _, _, os = _rows(residual_out, "residual_out", dtype, device, shape)
    if hidden:
        st = _lib().dropout_add_fwd(op, os, xp, xs, rp, rs, n, hidden, _drop(p, seed, offset, step, device), code,
                                    _raw_stream(device))
        if st:
            _failed(st, "dropout_add_fwd")
    return residual_out


# ------------------------------------- dropout + residual add + RMSNorm
def _norm_shape(x):
    shape = x.shape
    if not shape or shape[-1] == 0:
        raise ValueError("the last dimension must not be empty")
    return shape, x.numel() // shape[-1], shape[-1]


def dropout_add_rmsnorm_fwd(x, residual, weight, p: float, eps: float = 1e-6, *, seed: int, offset: int = 0, step=None,
                            out=None, residual_out=None, stream=None):
    """(out, residual_out) of add_rmsnorm_fwd with dropout on x: acc =
    residual + dropout(x), residual_out = rne(acc), out = rne(acc / rms *
    weight).  With p = 0 the bits are add_rmsnorm_fwd's.  Contiguous
    [..., hidden] tensors, hidden a multiple of 8; out and residual_out may
    each be x or residual."""
    code, device = _dtype(x, "x"), x.get_device()
    if stream is not None or device != _current_device():
        with _switched(x, stream):
            return dropout_add_rmsnorm_fwd(x, residual, weight, p, eps, seed=seed, offset=offset, step=step, out=out,
                                           residual_out=residual_out)
    dtype = x.dtype
    shape, n, hidden = _norm_shape(x)
    xp = _flat(x, "x", dtype, device, shape)
    rp = _flat(residual, "residual", dtype, device, shape)
    wp = _flat(weight, "weight", dtype, device, shape[-1:])
    if out is None:
        out = torch.empty_like(x)
    if residual_out is None:
        residual_out = torch.empty_like(x)
    st = _lib().dropout_add_rmsnorm_fwd(
        _flat(out, "out", dtype, device, shape), _flat(residual_out, "residual_out", dtype, device, shape), xp, rp, wp,
        eps, n, hidden, _drop(p, seed, offset, step, device), code, _raw_stream(device))
    if st:
        _failed(st, "dropout_add_rmsnorm_fwd")
    return out, residual_out


def _workspace(given, need, device):
    """(tensor to keep alive, data_ptr, bytes)."""
    if given is None:
        given = torch.empty(need, dtype=torch.uint8, device=device)
        return given, given.data_ptr(), need
    if given.get_device() != device.index or not given.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {device}")
    return given, given.data_ptr(), given.numel() * given.element_size()


def _norm_bwd(where, drop, dx, want_dx, dresidual, dresidual_name, dweight, weight_grad, dout, dresidual_out, x, weight,
              eps, workspace, code, device):
    dtype = x.dtype
    shape, n, hidden = _norm_shape(x)
    hp = _flat(x, "residual_out", dtype, device, shape)
    gp = _flat(dout, "dout", dtype, device, shape)
    dp = None if dresidual_out is None else _flat(dresidual_out, "dresidual_out", dtype, device, shape)
    wp = _flat(weight, "weight", dtype, device, shape[-1:])
    if dresidual is None:
        dresidual = torch.empty_like(x)
    outs = [_flat(dresidual, dresidual_name, dtype, device, shape)]
    if want_dx:
        if dx is None:
            dx = torch.empty_like(x)
        outs.insert(0, _flat(dx, "dx", dtype, device, shape))
    L = _lib()
    dwp = wsp = None
    nbytes = 0
    if weight_grad:
        if dweight is None:
            dweight = torch.empty(hidden, dtype=torch.float32, device=x.device)
        dwp = _flat(dweight, "dweight", torch.float32, device, shape[-1:])
        workspace, wsp, nbytes = _workspace(workspace, L.rmsnorm_bwd_workspace_bytes(n, hidden, code), x.device)
    elif dweight is not None:
        raise ValueError("dweight is given but weight_grad is False")
    st = getattr(L, where)(*outs, dwp, gp, dp, hp, wp, eps, n, hidden, *drop, code, wsp, nbytes, _raw_stream(device))
    if st:
        _failed(st, where)
    return dx, dresidual, dweight


def dropout_add_rmsnorm_bwd(dout, dresidual_out, residual_out, weight, p: float, eps: float = 1e-6, *, seed: int,
                            offset: int = 0, step=None, dx=None, dresidual=None, dweight=None, weight_grad: bool = True,
                            workspace=None, stream=None):
    """(dx, dresidual, dweight): gradients of dropout_add_rmsnorm_fwd from
    those of its two outputs (dresidual_out None: zero) and its residual_out.
    dweight is fp32, None with weight_grad=False.  dx and dresidual may each
    be dout, dresidual_out or residual_out.  workspace: a tensor of at least
    rmsnorm_bwd_workspace_bytes (C ABI); by default one is allocated."""
    code, device = _dtype(residual_out, "residual_out"), residual_out.get_device()
    if stream is not None or device != _current_device():
        with _switched(residual_out, stream):
            return dropout_add_rmsnorm_bwd(dout, dresidual_out, residual_out, weight, p, eps, seed=seed, offset=offset,
                                           step=step, dx=dx, dresidual=dresidual, dweight=dweight,
                                           weight_grad=weight_grad, workspace=workspace)
    return _norm_bwd("dropout_add_rmsnorm_bwd", (_drop(p, seed, offset, step, device),), dx, True, dresidual,
                     "dresidual", dweight, weight_grad, dout, dresidual_out, residual_out, weight, eps, workspace, code,
                     device)


def add_rmsnorm_bwd(dout, dresidual_out, residual_out, weight, eps: float = 1e-6, *, dh=None, dweight=None,
                    weight_grad: bool = True, workspace=None, stream=None):
    """(dh, dweight): gradients of add_rmsnorm_fwd; dh is that of x and of
    residual.  Arguments as in dropout_add_rmsnorm_bwd."""
    code, device = _dtype(residual_out, "residual_out"), residual_out.get_device()
    if stream is not None or device != _current_device():
        with _switched(residual_out, stream):
            return add_rmsnorm_bwd(dout, dresidual_out, residual_out, weight, eps, dh=dh, dweight=dweight,
                                   weight_grad=weight_grad, workspace=workspace)
    return _norm_bwd("add_rmsnorm_bwd", (), None, False, dh, "dh", dweight, weight_grad, dout, dresidual_out,
                     residual_out, weight, eps, workspace, code, device)[1:]


def rmsnorm_bwd(dout, x, weight, eps: float = 1e-6, **kw):
    """(dx, dweight): gradients of rmsnorm_fwd.  Keywords as in
    add_rmsnorm_bwd."""
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
    if scaling not in ROPE_SCALINGS:
        raise ValueError(f"scaling must be one of {sorted(ROPE_SCALINGS)}")
    f = torch.empty(max(int(rot_dim) // 2, 1), dtype=torch.float64)
    st = _lib().rope_frequencies(f.data_ptr(), int(rot_dim), float(base), ROPE_SCALINGS[scaling], float(factor),
                                 float(original_length), float(low), float(high))
    if st:
        _failed(st, "rope_frequencies")
    return f if device is None else f.to(device)


def _heads(t, name, dtype, device, shape) -> bytes:
    if t.dtype is not dtype or t.get_device() != device or t.shape != shape:
        _refuse(t, name, dtype, device, shape, False)
    b, s, h, d = t.stride()
    if d != 1 and shape[3] > 1:
        _refuse(t, name, dtype, device, shape, False)
    return _pack_heads(t.data_ptr(), b, s, h)


def _new(x):
    return torch.empty_like(x, memory_format=torch.contiguous_format)


def _rope(q, k, inv_freq, positions, position0, interleaved, scale, device) -> bytes:
    shape = q.shape
    if len(shape) != 4:
        raise ValueError("q and k must be [batch, seq, heads, head_dim]")
    b, s, hq, d = shape
    hk = 0
    if k is not None:
        ks = k.shape
        if len(ks) != 4 or ks[0] != b or ks[1] != s or ks[3] != d:
            raise ValueError("q and k must be [batch, seq, heads, head_dim], alike but for their heads")
        hk = ks[2]
    if len(inv_freq.shape) != 1:
        raise ValueError("inv_freq must be 1-D: one frequency per pair")
    freq = _flat(inv_freq, "inv_freq", torch.float64, device, inv_freq.shape)
    pos = 0
    if positions is not None:
        if position0:
            raise ValueError("give positions or position0, not both")
        pos = _flat(positions, "positions", torch.int64, device, shape[:2])
    return _pack_rope(b, s, hq, hk, d, 2 * inv_freq.shape[0], 1 if interleaved else 0, freq, pos, position0, scale)


def _turn(where, q, k, inv_freq, positions, position0, interleaved, scale, q_out, k_out, stream):
    code, device = _dtype(q, "q"), q.get_device()
    if stream is not None or device != _current_device():
        with _switched(q, stream):
            return _turn(where, q, k, inv_freq, positions, position0, interleaved, scale, q_out, k_out, None)
    r = _rope(q, k, inv_freq, positions, position0, interleaved, scale, device)
    dtype = q.dtype
    if q_out is None:
        q_out = _new(q)
    ko = ki = None
    if k is not None:
        if k_out is None:
            k_out = _new(k)
        ko, ki = _heads(k_out, "k_out", dtype, device, k.shape), _heads(k, "k", dtype, device, k.shape)
    st = getattr(_lib(), where)(_heads(q_out, "q_out", dtype, device, q.shape), ko,
                                _heads(q, "q", dtype, device, q.shape), ki, r, code, _raw_stream(device))
    if st:
        _failed(st, where)
    return q_out, k_out


def rope_fwd(q, k, inv_freq, positions=None, *, position0: int = 0, interleaved: bool = False, scale: float = 1.0,
             q_out=None, k_out=None, stream=None):
    """(q_out, k_out): q and k turned by position * inv_freq.

    q, k: [batch, seq, heads, head_dim] with any strides but a unit last one
    (slices of a packed projection, or a transposed [batch, heads, seq,
    head_dim]); k may be None.  The first 2 * len(inv_freq) columns turn, in
    pairs (i, i + half) or, interleaved, (2 i, 2 i + 1).  inv_freq: float64
    (rope_frequencies).  positions: int64 [batch, seq], else position0 + s.
    Outputs are contiguous unless given; each may be its own input."""
    return _turn("rope_fwd", q, k, inv_freq, positions, position0, interleaved, scale, q_out, k_out, stream)


def rope_bwd(dq_out, dk_out, inv_freq, positions=None, *, position0: int = 0, interleaved: bool = False,
             scale: float = 1.0, dq=None, dk=None, stream=None):
    """(dq, dk): the gradient of rope_fwd, a turn by the opposite angles."""
    return _turn("rope_bwd", dq_out, dk_out, inv_freq, positions, position0, interleaved, scale, dq, dk, stream)


def qk_rmsnorm_rope_fwd(q, k, q_weight, k_weight, inv_freq, q_eps: float = 1e-6, k_eps: float = 1e-6, *,
                        positions=None, position0: int = 0, interleaved: bool = False, scale: float = 1.0, q_out=None,
                        k_out=None, stream=None):
    """(q_out, k_out): RMSNorm of every head of q and k (weights [head_dim]),
    then rope_fwd, in one pass with one rounding.  k and k_weight may be
    None."""
    code, device = _dtype(q, "q"), q.get_device()
    if stream is not None or device != _current_device():
        with _switched(q, stream):
            return qk_rmsnorm_rope_fwd(q, k, q_weight, k_weight, inv_freq, q_eps, k_eps, positions=positions,
                                       position0=position0, interleaved=interleaved, scale=scale, q_out=q_out,
                                       k_out=k_out)
    r = _rope(q, k, inv_freq, positions, position0, interleaved, scale, device)
    dtype, width = q.dtype, q.shape[3:]
    if q_out is None:
        q_out = _new(q)
    ko = ki = kw = None
    if k is not None:
        if k_out is None:
            k_out = _new(k)
        ko, ki = _heads(k_out, "k_out", dtype, device, k.shape), _heads(k, "k", dtype, device, k.shape)
        kw = _flat(k_weight, "k_weight", dtype, device, width)
    st = _lib().qk_rmsnorm_rope_fwd(
        _heads(q_out, "q_out", dtype, device, q.shape), ko, _heads(q, "q", dtype, device, q.shape), ki,
        _flat(q_weight, "q_weight", dtype, device, width), kw, q_eps, k_eps, r, code, _raw_stream(device))
    if st:
        _failed(st, "qk_rmsnorm_rope_fwd")
    return q_out, k_out


def qk_rmsnorm_rope_bwd(dq_out, dk_out, q, k, q_weight, k_weight, inv_freq, q_eps: float = 1e-6, k_eps: float = 1e-6,
                        *, positions=None, position0: int = 0, interleaved: bool = False, scale: float = 1.0, dq=None,
                        dk=None, dq_weight=None, dk_weight=None, weight_grad: bool = True, workspace=None,
                        stream=None):
    """(dq, dk, dq_weight, dk_weight): gradients of qk_rmsnorm_rope_fwd; the
    weights' are fp32, None with weight_grad=False.  dq may be q or dq_out,
    dk may be k or dk_out.  workspace: a tensor of at least
    qk_rmsnorm_rope_bwd_workspace_bytes (C ABI); by default one is
    allocated."""
    code, device = _dtype(q, "q"), q.get_device()
    if stream is not None or device != _current_device():
        with _switched(q, stream):
            return qk_rmsnorm_rope_bwd(dq_out, dk_out, q, k, q_weight, k_weight, inv_freq, q_eps, k_eps,
                                       positions=positions, position0=position0, interleaved=interleaved, scale=scale,
                                       dq=dq, dk=dk, dq_weight=dq_weight, dk_weight=dk_weight, weight_grad=weight_grad,
                                       workspace=workspace)
    if not weight_grad and (dq_weight is not None or dk_weight is not None):
        raise ValueError("a weight's gradient is given but weight_grad is False")
    r = _rope(q, k, inv_freq, positions, position0, interleaved, scale, device)
    dtype, width, L = q.dtype, q.shape[3:], _lib()
    if dq is None:
        dq = _new(q)
    dkh = dkoh = kh = kw = None
    if k is not None:
        if dk is None:
            dk = _new(k)
        dkh, dkoh, kh = (_heads(t, name, dtype, device, k.shape) for t, name in ((dk, "dk"), (dk_out, "dk_out"),
                                                                               (k, "k")))
        kw = _flat(k_weight, "k_weight", dtype, device, width)
    dqw = dkw = wsp = None
    nbytes = 0
    if weight_grad:
        if dq_weight is None:
            dq_weight = torch.empty(width, dtype=torch.float32, device=q.device)
        dqw = _flat(dq_weight, "dq_weight", torch.float32, device, width)
        if k is not None:
            if dk_weight is None:
                dk_weight = torch.empty(width, dtype=torch.float32, device=q.device)
            dkw = _flat(dk_weight, "dk_weight", torch.float32, device, width)
        workspace, wsp, nbytes = _workspace(workspace, L.qk_rmsnorm_rope_bwd_workspace_bytes(r, code), q.device)
    st = L.qk_rmsnorm_rope_bwd(
        _heads(dq, "dq", dtype, device, q.shape), dkh, dqw, dkw, _heads(dq_out, "dq_out", dtype, device, q.shape), dkoh,
        _heads(q, "q", dtype, device, q.shape), kh, _flat(q_weight, "q_weight", dtype, device, width), kw, q_eps, k_eps,
        r, code, wsp, nbytes, _raw_stream(device))
    if st:
        _failed(st, "qk_rmsnorm_rope_bwd")
    return dq, dk, dq_weight, dk_weight
