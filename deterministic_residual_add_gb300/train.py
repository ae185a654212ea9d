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
"""
from __future__ import annotations

import ctypes

import torch

ROPE_SCALINGS = {"none": 0, "linear": 1, "base": 2, "by_parts": 3}

_vp, _i64, _f32, _f64, _int, _size = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_float, ctypes.c_double, ctypes.c_int,
                                      ctypes.c_size_t)
_DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}


class _Dropout(ctypes.Structure):
    _fields_ = [("p", _f32), ("seed", ctypes.c_uint64), ("offset", ctypes.c_uint64), ("step", _vp)]


class _Heads(ctypes.Structure):
    _fields_ = [("data", _vp), ("batch_stride", _i64), ("seq_stride", _i64), ("head_stride", _i64)]


class _Rope(ctypes.Structure):
    _fields_ = [("batch", _i64), ("seq", _i64), ("q_heads", _i64), ("k_heads", _i64), ("head_dim", _i64),
                ("rot_dim", _i64), ("interleaved", _int), ("inv_freq", _vp), ("positions", _vp), ("position0", _i64),
                ("scale", _f32)]


_L = None


def _bind(L):
    """Argument types of the entry points, set once when the library loads."""
    global _L
    drop, rope, heads4 = ctypes.POINTER(_Dropout), ctypes.POINTER(_Rope), [_Heads] * 4
    for name, args in [
            ("dropout_fwd", [_vp, _i64, _vp, _i64, _i64, _i64, drop, _int, _vp]),
            ("dropout_add_fwd", [_vp, _i64, _vp, _i64, _vp, _i64, _i64, _i64, drop, _int, _vp]),
            ("dropout_add_rmsnorm_fwd", [_vp] * 5 + [_f32, _i64, _i64, drop, _int, _vp]),
            ("dropout_add_rmsnorm_bwd", [_vp] * 7 + [_f32, _i64, _i64, drop, _int, _vp, _size, _vp]),
            ("add_rmsnorm_bwd", [_vp] * 6 + [_f32, _i64, _i64, _int, _vp, _size, _vp]),
            ("rope_fwd", heads4 + [rope, _int, _vp]),
            ("rope_bwd", heads4 + [rope, _int, _vp]),
            ("qk_rmsnorm_rope_fwd", heads4 + [_vp, _vp, _f32, _f32, rope, _int, _vp]),
            ("qk_rmsnorm_rope_bwd", [_Heads, _Heads, _vp, _vp] + heads4 + [_vp, _vp, _f32, _f32, rope, _int, _vp,
                                                                           _size, _vp]),
            ("rope_frequencies", [_vp, _i64, _f64, _int, _f64, _f64, _f64, _f64])]:
        f = getattr(L, name)
        f.argtypes, f.restype = args, _int
    L.rmsnorm_bwd_workspace_bytes.argtypes, L.rmsnorm_bwd_workspace_bytes.restype = [_i64, _i64, _int], _size
    L.qk_rmsnorm_rope_bwd_workspace_bytes.argtypes = [rope, _int]
    L.qk_rmsnorm_rope_bwd_workspace_bytes.restype = _size
    _L = L


def _lib():
    if _L is None:
        from . import lib
        lib()
    return _L


class _On:
    """Makes `device` and the launch stream current for a call; .handle is
    the stream's.  Where both already are, nothing is switched."""

    __slots__ = ("handle", "contexts")

    def __init__(self, device, stream):
        self.contexts = ()
        if device.index != torch.cuda.current_device():
            self.contexts = (torch.cuda.device(device),)
        if stream is None:
            self.handle = torch.cuda.current_stream(device).cuda_stream
        else:
            if isinstance(stream, int):
                stream = torch.cuda.ExternalStream(stream, device)
            if stream.device != device:
                raise ValueError(f"the stream is on {stream.device}, the tensors on {device}")
            self.handle = stream.cuda_stream
            self.contexts += (torch.cuda.stream(stream),)

    def __enter__(self):
        for c in self.contexts:
            c.__enter__()
        return self.handle

    def __exit__(self, *a):
        for c in reversed(self.contexts):
            c.__exit__(*a)


def _done(status: int, where: str):
    if status != 0:
        from . import DraddError
        raise DraddError(status, where)


def _dtype(x, name: str) -> int:
    code = _DTYPES.get(x.dtype)
    if code is None:
        raise TypeError(f"{name} must be bfloat16, float16 or float32 (got {x.dtype})")
    if not x.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return code


def _like(t, x, name: str, shape=None, dtype=None):
    """Checks that t is of x's type (or dtype) and device, and of `shape`."""
    if t.dtype != (x.dtype if dtype is None else dtype):
        raise TypeError(f"{name} must hold {x.dtype if dtype is None else dtype} (got {t.dtype})")
    if t.device != x.device:
        raise ValueError(f"{name} is on {t.device}, expected {x.device}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _flat(t, x, name: str, shape=None, dtype=None) -> int:
    """data_ptr of a contiguous tensor checked by _like."""
    _like(t, x, name, shape, dtype)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _drop(p, seed, offset, step, x):
    if step is not None:
        if step.numel() != 1:
            raise ValueError("step must hold one int64")
        step = _flat(step, x, "step", dtype=torch.int64)
    return _Dropout(p, seed & 0xFFFFFFFFFFFFFFFF, offset & 0xFFFFFFFFFFFFFFFF, step)


# ------------------------------------------------------------------ dropout
def _rows(t, name: str):
    """(rows, columns, row stride): any contiguous tensor as [rows, last
    dimension], or a 2-D tensor with unit column stride."""
    if t.is_contiguous():
        cols = t.shape[-1] if t.dim() else 1
        return (t.numel() // cols if cols else 0), cols, cols
    if t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"{name} must be contiguous, or 2-D with unit column stride")
    return t.shape[0], t.shape[1], t.stride(0) if t.shape[0] > 1 else t.shape[1]


def dropout_fwd(x, p: float, *, seed: int, offset: int = 0, step=None, out=None, stream=None):
    """out = x where kept, times 1 / (1 - p) (p applied in steps of 2^-16),
    and 0 where dropped.  The gradient is the same call on the gradient.
    x: contiguous, or 2-D with any row stride; out may be x."""
    code = _dtype(x, "x")
    with _On(x.device, stream) as handle:
        if out is None:
            out = torch.empty_like(x, memory_format=torch.contiguous_format)
        _like(out, x, "out", x.shape)
        n, h, xs = _rows(x, "x")
        _, _, os = _rows(out, "out")
        if n == 0:
            return out
        d = _drop(p, seed, offset, step, x)
        _done(_lib().dropout_fwd(out.data_ptr(), os, x.data_ptr(), xs, n, h, ctypes.byref(d), code, handle),
              "dropout_fwd")
    return out


def dropout_add_fwd(x, residual, p: float, *, seed: int, offset: int = 0, step=None, residual_out=None, stream=None):
    """residual_out = residual + dropout(x), rounded once.  Gradients:
    dresidual = dy, dx = dropout_fwd(dy) with the same p, seed and offset.
    residual_out may be x or residual."""
    code = _dtype(x, "x")
    with _On(x.device, stream) as handle:
        if residual_out is None:
            residual_out = torch.empty_like(x, memory_format=torch.contiguous_format)
        _like(residual, x, "residual", x.shape)
        _like(residual_out, x, "residual_out", x.shape)
        n, h, xs = _rows(x, "x")
        _, _, rs = _rows(residual, "residual")
        _, _, os = _rows(residual_out, "residual_out")
        if n == 0:
            return residual_out
        d = _drop(p, seed, offset, step, x)
        _done(_lib().dropout_add_fwd(residual_out.data_ptr(), os, x.data_ptr(), xs, residual.data_ptr(), rs, n, h,
                                     ctypes.byref(d), code, handle), "dropout_add_fwd")
    return residual_out


# ------------------------------------- dropout + residual add + RMSNorm
def _norm_shape(x):
    if x.dim() == 0 or x.shape[-1] == 0:
        raise ValueError("the last dimension must not be empty")
    hidden = x.shape[-1]
    return x.numel() // hidden, hidden


def dropout_add_rmsnorm_fwd(x, residual, weight, p: float, eps: float = 1e-6, *, seed: int, offset: int = 0, step=None,
                            out=None, residual_out=None, stream=None):
    """(out, residual_out) of add_rmsnorm_fwd with dropout on x: acc =
    residual + dropout(x), residual_out = rne(acc), out = rne(acc / rms *
    weight).  With p = 0 the bits are add_rmsnorm_fwd's.  Contiguous
    [..., hidden] tensors, hidden a multiple of 8; out and residual_out may
    each be x or residual."""
    code = _dtype(x, "x")
    n, hidden = _norm_shape(x)
    shape = x.shape
    with _On(x.device, stream) as handle:
        if out is None:
            out = torch.empty_like(x)
        if residual_out is None:
            residual_out = torch.empty_like(x)
        d = _drop(p, seed, offset, step, x)
        _done(_lib().dropout_add_rmsnorm_fwd(
            _flat(out, x, "out", shape), _flat(residual_out, x, "residual_out", shape), _flat(x, x, "x"),
            _flat(residual, x, "residual", shape), _flat(weight, x, "weight", shape[-1:]), eps, n, hidden,
            ctypes.byref(d), code, handle), "dropout_add_rmsnorm_fwd")
    return out, residual_out


def _workspace(given, need: int, x):
    """A workspace of `need` bytes on the current stream, or the one given."""
    if given is None:
        return torch.empty(need, dtype=torch.uint8, device=x.device)
    if given.device != x.device or not given.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {x.device}")
    return given


def dropout_add_rmsnorm_bwd(dout, dresidual_out, residual_out, weight, p: float, eps: float = 1e-6, *, seed: int,
                            offset: int = 0, step=None, dx=None, dresidual=None, dweight=None, weight_grad: bool = True,
                            workspace=None, stream=None):
    """(dx, dresidual, dweight): gradients of dropout_add_rmsnorm_fwd from
    those of its two outputs (dresidual_out None: zero) and its residual_out.
    dweight is fp32, None with weight_grad=False.  dx and dresidual may each
    be dout, dresidual_out or residual_out.  workspace: a tensor of at least
    rmsnorm_bwd_workspace_bytes; by default one is allocated."""
    x = residual_out
    code = _dtype(x, "residual_out")
    n, hidden = _norm_shape(x)
    shape = x.shape
    with _On(x.device, stream) as handle:
        if dx is None:
            dx = torch.empty_like(x)
        if dresidual is None:
            dresidual = torch.empty_like(x)
        dweight, work, nbytes = _weight_sums(dweight, weight_grad, workspace, n, hidden, code, x)
        d = _drop(p, seed, offset, step, x)
        _done(_lib().dropout_add_rmsnorm_bwd(
            _flat(dx, x, "dx", shape), _flat(dresidual, x, "dresidual", shape),
            None if dweight is None else dweight.data_ptr(), _flat(dout, x, "dout", shape),
            None if dresidual_out is None else _flat(dresidual_out, x, "dresidual_out", shape),
            _flat(x, x, "residual_out"), _flat(weight, x, "weight", shape[-1:]), eps, n, hidden, ctypes.byref(d), code,
            None if work is None else work.data_ptr(), nbytes, handle), "dropout_add_rmsnorm_bwd")
    return dx, dresidual, dweight


def _weight_sums(dweight, wanted, workspace, n, hidden, code, x):
    if not wanted:
        if dweight is not None:
            raise ValueError("dweight is given but weight_grad is False")
        return None, None, 0
    if dweight is None:
        dweight = torch.empty(hidden, dtype=torch.float32, device=x.device)
    _flat(dweight, x, "dweight", torch.Size((hidden,)), torch.float32)
    work = _workspace(workspace, _lib().rmsnorm_bwd_workspace_bytes(n, hidden, code), x)
    return dweight, work, work.numel() * work.element_size()


def add_rmsnorm_bwd(dout, dresidual_out, residual_out, weight, eps: float = 1e-6, *, dh=None, dweight=None,
                    weight_grad: bool = True, workspace=None, stream=None):
    """(dh, dweight): gradients of add_rmsnorm_fwd; dh is that of x and of
    residual.  Arguments as in dropout_add_rmsnorm_bwd."""
    x = residual_out
    code = _dtype(x, "residual_out")
    n, hidden = _norm_shape(x)
    shape = x.shape
    with _On(x.device, stream) as handle:
        if dh is None:
            dh = torch.empty_like(x)
        dweight, work, nbytes = _weight_sums(dweight, weight_grad, workspace, n, hidden, code, x)
        _done(_lib().add_rmsnorm_bwd(
            _flat(dh, x, "dh", shape), None if dweight is None else dweight.data_ptr(), _flat(dout, x, "dout", shape),
            None if dresidual_out is None else _flat(dresidual_out, x, "dresidual_out", shape),
            _flat(x, x, "residual_out"), _flat(weight, x, "weight", shape[-1:]), eps, n, hidden, code,
            None if work is None else work.data_ptr(), nbytes, handle), "add_rmsnorm_bwd")
    return dh, dweight


def rmsnorm_bwd(dout, x, weight, eps: float = 1e-6, **kw):
    """(dx, dweight): gradients of rmsnorm_fwd."""
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
    f = torch.empty(max(int(rot_dim), 0) // 2, dtype=torch.float64)
    _done(_lib().rope_frequencies(f.data_ptr() if f.numel() else ctypes.addressof(_f64()), int(rot_dim), float(base),
                                  ROPE_SCALINGS[scaling], float(factor), float(original_length), float(low),
                                  float(high)), "rope_frequencies")
    return f if device is None else f.to(device)


_NO_HEADS = _Heads(None, 0, 0, 0)


def _heads(t, x, name: str, shape=None):
    _like(t, x, name, shape)
    if t.stride(-1) != 1 and t.shape[-1] > 1:
        raise ValueError(f"{name} must have unit stride in its last dimension")
    return _Heads(t.data_ptr(), t.stride(0), t.stride(1), t.stride(2))


def _rope(q, k, inv_freq, positions, position0, interleaved, scale):
    if q.dim() != 4 or (k is not None and (k.dim() != 4 or k.shape[:2] != q.shape[:2] or k.shape[3] != q.shape[3])):
        raise ValueError("q and k must be [batch, seq, heads, head_dim], alike but for their heads")
    b, s, hq, d = q.shape
    freq = _flat(inv_freq, q, "inv_freq", dtype=torch.float64)
    if inv_freq.dim() != 1:
        raise ValueError("inv_freq must be 1-D: one frequency per pair")
    if positions is not None:
        if position0:
            raise ValueError("give positions or position0, not both")
        if positions.numel() != b * s or (positions.dim() == 2 and positions.shape != q.shape[:2]):
            raise ValueError(f"positions must be [{b}, {s}]")
        positions = _flat(positions, q, "positions", dtype=torch.int64)
    return _Rope(b, s, hq, 0 if k is None else k.shape[2], d, 2 * inv_freq.shape[0], int(bool(interleaved)), freq,
                 positions, position0, scale)


def _out(t, like):
    return torch.empty(like.shape, dtype=like.dtype, device=like.device) if t is None else t


def _turn(where, q, k, inv_freq, positions, position0, interleaved, scale, q_out, k_out, stream):
    code = _dtype(q, "q")
    r = _rope(q, k, inv_freq, positions, position0, interleaved, scale)
    with _On(q.device, stream) as handle:
        q_out = _out(q_out, q)
        ko, ki = _NO_HEADS, _NO_HEADS
        if k is not None:
            k_out = _out(k_out, k)
            ko, ki = _heads(k_out, q, "k_out", k.shape), _heads(k, q, "k")
        _done(getattr(_lib(), where)(_heads(q_out, q, "q_out", q.shape), ko, _heads(q, q, "q"), ki, ctypes.byref(r),
                                     code, handle), where)
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
    code = _dtype(q, "q")
    r = _rope(q, k, inv_freq, positions, position0, interleaved, scale)
    with _On(q.device, stream) as handle:
        q_out = _out(q_out, q)
        ko, ki, kw = _NO_HEADS, _NO_HEADS, None
        if k is not None:
            k_out = _out(k_out, k)
            ko, ki = _heads(k_out, q, "k_out", k.shape), _heads(k, q, "k")
            kw = _flat(k_weight, q, "k_weight", q.shape[3:])
        _done(_lib().qk_rmsnorm_rope_fwd(
            _heads(q_out, q, "q_out", q.shape), ko, _heads(q, q, "q"), ki, _flat(q_weight, q, "q_weight", q.shape[3:]),
            kw, q_eps, k_eps, ctypes.byref(r), code, handle), "qk_rmsnorm_rope_fwd")
    return q_out, k_out


def qk_rmsnorm_rope_bwd(dq_out, dk_out, q, k, q_weight, k_weight, inv_freq, q_eps: float = 1e-6, k_eps: float = 1e-6,
                        *, positions=None, position0: int = 0, interleaved: bool = False, scale: float = 1.0, dq=None,
                        dk=None, dq_weight=None, dk_weight=None, weight_grad: bool = True, workspace=None,
                        stream=None):
    """(dq, dk, dq_weight, dk_weight): gradients of qk_rmsnorm_rope_fwd; the
    weights' are fp32, None with weight_grad=False.  dq may be q or dq_out,
    dk may be k or dk_out."""
    code = _dtype(q, "q")
    r = _rope(q, k, inv_freq, positions, position0, interleaved, scale)
    if not weight_grad and (dq_weight is not None or dk_weight is not None):
        raise ValueError("a weight's gradient is given but weight_grad is False")
    with _On(q.device, stream) as handle:
        dq = _out(dq, q)
        kh, kw, dkw = [_NO_HEADS] * 3, None, None
        if k is not None:
            dk = _out(dk, k)
            kh = [_heads(dk, q, "dk", k.shape), _heads(dk_out, q, "dk_out", k.shape), _heads(k, q, "k")]
            kw = _flat(k_weight, q, "k_weight", q.shape[3:])
        work, nbytes, dqw = None, 0, None
        if weight_grad:
            if dq_weight is None:
                dq_weight = torch.empty(q.shape[3], dtype=torch.float32, device=q.device)
            dqw = _flat(dq_weight, q, "dq_weight", q.shape[3:], torch.float32)
            if k is not None:
                if dk_weight is None:
                    dk_weight = torch.empty(q.shape[3], dtype=torch.float32, device=q.device)
                dkw = _flat(dk_weight, q, "dk_weight", q.shape[3:], torch.float32)
            work = _workspace(workspace, _lib().qk_rmsnorm_rope_bwd_workspace_bytes(ctypes.byref(r), code), q)
            nbytes, work = work.numel() * work.element_size(), work.data_ptr()
        _done(_lib().qk_rmsnorm_rope_bwd(
            _heads(dq, q, "dq", q.shape), kh[0], dqw, dkw, _heads(dq_out, q, "dq_out", q.shape), kh[1],
            _heads(q, q, "q"), kh[2], _flat(q_weight, q, "q_weight", q.shape[3:]), kw, q_eps, k_eps, ctypes.byref(r),
            code, work, nbytes, handle), "qk_rmsnorm_rope_bwd")
    return dq, dk, dq_weight, dk_weight
