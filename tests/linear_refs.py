"""Plain fp64 references of the matrix products and losses of
include/dradd_linear.h, with bounds on how far the kernels may be from them.

The tensor cores add the terms of a product 16 at a time to an fp32 sum and
cut off what does not fit: at most 2^-23 of the magnitudes added so far, a
step.  With a few roundings where parts are joined, a sum of k terms is off
by at most (k / 16 + 32) 2^-23 of the sum of their magnitudes."""
from __future__ import annotations

import ctypes
import math

import torch

from train_refs import HALF_STEP, TINY, assert_close  # noqa: F401

ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")
EPS32 = 2.0 ** -24


class CMatrix(ctypes.Structure):
    """dradd_matrix of include/dradd_linear.h."""
    _fields_ = [("data", ctypes.c_void_p), ("stride", ctypes.c_int64)]


class CTeacher(ctypes.Structure):
    """dradd_teacher."""
    _fields_ = [("index", ctypes.c_void_p), ("logits", ctypes.c_void_p), ("logits_dtype", ctypes.c_int),
                ("top", ctypes.c_int64), ("temperature", ctypes.c_float)]


def c_entry(L, name):
    vp, i64, i32, size = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
    f = getattr(L, name)
    f.argtypes = {
        "linear_act_add_fwd": [vp] * 5 + [i32, i64, i64, i64, i32, vp, size, vp],
        "linear_act_add_bwd": [vp] * 7 + [i32, i64, i64, i64, i32, vp, size, vp],
        "linear_cross_entropy_fwd": [vp] * 5 + [i64] * 4 + [i32, vp, size, vp],
        "linear_cross_entropy_bwd": [vp, vp, vp, i64, vp, i64, vp, vp, vp, i64, vp, i64, i64, i64, i32, vp, size, vp],
        "linear_distill_fwd": [vp] * 5 + [i64] * 3 + [i32, vp, size, vp],
        "linear_distill_bwd": [vp, vp, vp, i64, vp, i64, vp, vp, vp, vp, i64, i64, i64, i32, vp, size, vp],
        "linear_act_add_fwd_workspace_bytes": [i64] * 3,
        "linear_act_add_bwd_workspace_bytes": [i64] * 3 + [i32] * 4,
        "linear_cross_entropy_fwd_workspace_bytes": [i64] * 3,
        "linear_cross_entropy_bwd_workspace_bytes": [i64] * 3,
        "linear_distill_fwd_workspace_bytes": [i64] * 4,
        "linear_distill_bwd_workspace_bytes": [i64] * 4,
    }[name]
    f.restype = size if name.endswith("bytes") else i32
    return f


def sum_err(k):
    return (k / 16 + 32) * 2.0 ** -23


def act64(z, act):
    if act == "relu":
        return z.clamp(min=0)
    if act == "gelu":
        return z * 0.5 * torch.erfc(-z / math.sqrt(2))
    if act == "gelu_tanh":
        return z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
    return z * torch.sigmoid(z) if act == "silu" else z


def slope64(z, act):
    z = z.detach().clone().requires_grad_()
    with torch.enable_grad():
        return torch.autograd.grad(act64(z, act).sum(), z)[0] if act != "none" else torch.ones_like(z)


def product(x, w, b=None):
    """x w^T + b in fp64, and the bound of the kernel's error."""
    x, w = x.double(), w.double()
    z, size = x @ w.t(), x.abs() @ w.abs().t()
    if b is not None:
        z, size = z + b.double(), size + b.double().abs()
    return z, sum_err(x.shape[-1]) * size


def linear(x, w, b, r, act):
    z, err = product(x, w, b)
    y = act64(z, act)
    # no activation is steeper than 1.13; their own steps 2^-15 of |z| at most, and where y is small of y
    err = 1.13 * err + (0 if act in ("none", "relu") else 2.0 ** -15) * y.abs()
    if r is not None:
        y = y + r.double()
        err = err + 2.0 ** -23 * (y.abs() + r.double().abs())
    return y, err


def linear_grads(dout, x, w, b, act):
    """[(dx, its bound), (dweight, ...), (dbias, ...)]."""
    z, zerr = product(x, w, b)
    g = dout.double()
    dz = g * slope64(z, act)
    half = HALF_STEP[x.dtype]
    err = torch.zeros_like(dz)
    if act == "relu":
        err = torch.where(z.abs() <= zerr, g.abs(), err)  # which side of 0 is not known
    elif act != "none":
        # second derivatives are below 1.2, the slope's own steps below 2^-14
        err = g.abs() * (1.2 * zerr + 2.0 ** -14)
    rounding = 0 if act == "none" else half * (dz.abs() + err) + TINY[x.dtype]
    d = err + rounding
    x64, w64 = x.double(), w.double()
    rows, cols = dz.shape
    return [(dz @ w64, d @ w64.abs() + sum_err(cols) * (dz.abs() @ w64.abs())),
            (dz.t() @ x64, d.t() @ x64.abs() + sum_err(rows) * (dz.abs().t() @ x64.abs())),
            (dz.sum(0), d.sum(0) + (rows / 8 + 64) * 2.0 ** -24 * dz.abs().sum(0))]


def shares64(index, logits, temperature):
    """The teacher's distribution over its entries; zeros in rows without any."""
    t = (logits.double() / temperature).masked_fill(index < 0, -math.inf)
    high = t.amax(1, keepdim=True)
    e = torch.exp(t - torch.where(high == -math.inf, 0.0, high))
    return e / torch.where(high == -math.inf, 1.0, e.sum(1, keepdim=True))


def ce_shares(target, ignore_index):
    return torch.where(target == ignore_index, 0, target)[:, None], (target != ignore_index).double()[:, None]


def loss(x, w, index, share, temperature=1.0):
    """(loss, bound, lse, bound); rows without shares have loss 0."""
    z, err = product(x, w)
    z, err = z / temperature, err / temperature
    lse = torch.logsumexp(z, 1)
    worst = err.amax(1)
    # lse moves by at most the largest error of a logit; exponentials and
    # their sums: 2^-22, the exponents' rounding, a rounding per part joined
    parts = -(-w.shape[0] // 128)
    lse_err = worst + (parts + 96) * 2.0 ** -24 + 8 * 2.0 ** -24 * (lse.abs() + z.abs().amax(1))
    at = index.clamp(min=0)
    picked = (share * z.gather(1, at)).sum(1)
    logs = torch.where(share > 0, torch.log(share.clamp(min=1e-300)), 0.0)
    entropy = (share * logs).sum(1)
    out = entropy + share.sum(1) * lse - picked
    counted = share.sum(1) > 0
    out_err = lse_err + worst + (share.shape[1] / 32 + 64) * 2.0 ** -24 * (
        (share * (z.gather(1, at).abs() + logs.abs())).sum(1) + lse.abs() + 1)
    return torch.where(counted, out, 0.0), torch.where(counted, out_err, 0.0), lse, lse_err


def loss_grads(dloss, dlse, x, w, index, share, lse, temperature=1.0):
    """[(dx, bound), (dweight, bound)] from the lse given."""
    z, zerr = product(x, w)
    z, zerr = z / temperature, zerr / temperature
    p = torch.exp(z - lse.double()[:, None])
    g = dloss.double().expand(x.shape[0]) * (share.sum(1) > 0)
    both = g + (0 if dlse is None else dlse.double().expand(x.shape[0]))
    live = ((g != 0) | (both != 0))[:, None]
    p = torch.where(live, p, 0.0)
    spike = torch.zeros_like(z).scatter_add_(1, index.clamp(min=0), share * g[:, None])
    dz = (both[:, None] * p - spike) / temperature
    # p: its logit's error, the exponent's rounding and 2^-21; shares: their
    # exponentials and a rounding each
    perr = (both.abs()[:, None] * p * (zerr + 2.0 ** -20 + 2.0 ** -22 * (z.abs() + lse.double().abs()[:, None])) +
            2.0 ** -18 * spike.abs()) / temperature
    perr = torch.where(live, perr, 0.0)
    half = HALF_STEP[x.dtype]
    d = perr + half * (dz.abs() + perr)
    if x.dtype == torch.float16:  # rounded at a scale that takes the largest factor of a row past 2^13
        most = ((g.abs() + both.abs()) / temperature).amax()
        d = d + live * TINY[x.dtype] * float(most) * 2.0 ** -13
    x64, w64 = torch.where(live, x.double(), 0.0), w.double()
    return [(dz @ w64, d @ w64.abs() + sum_err(w.shape[0]) * (dz.abs() @ w64.abs())),
            (dz.t() @ x64, d.t() @ x64.abs() + sum_err(x.shape[0]) * (dz.abs().t() @ x64.abs()))]


def norm_off(got, exact):
    n = exact.norm()
    return float((got.double() - exact).norm() / n) if n > 0 else float(got.double().norm())
