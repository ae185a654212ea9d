"""Plain references of the dropout, RMSNorm gradient and rotary operators,
written from their definitions: the generator in numpy integers, the
forwards of dropout in fp32 operations rounded one by one (the kernels'
results, bit for bit), everything else in fp64 with bounds on how far the
fp32 kernels may be from it."""
from __future__ import annotations

import ctypes

import numpy as np
import torch


class CDropout(ctypes.Structure):
    """dradd_dropout of include/dradd_train.h."""
    _fields_ = [("p", ctypes.c_float), ("seed", ctypes.c_uint64), ("offset", ctypes.c_uint64),
                ("step", ctypes.c_void_p)]


class CHeads(ctypes.Structure):
    """dradd_heads."""
    _fields_ = [("data", ctypes.c_void_p), ("batch_stride", ctypes.c_int64), ("seq_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64)]


class CRope(ctypes.Structure):
    """dradd_rope."""
    _fields_ = [(n, ctypes.c_int64) for n in ("batch", "seq", "q_heads", "k_heads", "head_dim", "rot_dim")] + [
        ("interleaved", ctypes.c_int), ("inv_freq", ctypes.c_void_p), ("positions", ctypes.c_void_p),
        ("position0", ctypes.c_int64), ("scale", ctypes.c_float)]


def c_entry(L, name):
    """An entry point of dradd_train.h for the C structures above: pointers
    by ctypes.byref, the rest converted by these argument types."""
    vp, i64, f32, i32, size = ctypes.c_void_p, ctypes.c_int64, ctypes.c_float, ctypes.c_int, ctypes.c_size_t
    f = getattr(L, name)
    f.argtypes = {
        "dropout_fwd": [vp, i64, vp, i64, i64, i64, vp, i32, vp],
        "dropout_add_fwd": [vp, i64, vp, i64, vp, i64, i64, i64, vp, i32, vp],
        "dropout_add_rmsnorm_fwd": [vp] * 5 + [f32, i64, i64, vp, i32, vp],
        "dropout_add_rmsnorm_bwd": [vp] * 7 + [f32, i64, i64, vp, i32, vp, size, vp],
        "add_rmsnorm_bwd": [vp] * 6 + [f32, i64, i64, i32, vp, size, vp],
        "rope_fwd": [vp] * 5 + [i32, vp],
        "rope_bwd": [vp] * 5 + [i32, vp],
        "qk_rmsnorm_rope_fwd": [vp] * 6 + [f32, f32, vp, i32, vp],
        "qk_rmsnorm_rope_bwd": [vp] * 10 + [f32, f32, vp, i32, vp, size, vp],
    }[name]
    f.restype = i32
    return f


HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
# half the spacing of a type's smallest values: what a rounding may add there
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}
EPS32 = 2.0 ** -24


def philox4x32(counter, key, rounds=7):
    """counter: four uint32 arrays (or numbers), key: two numbers."""
    c = [np.asarray(v, dtype=np.uint64) for v in counter]
    k = [int(v) for v in key]
    low, s = np.uint64(0xFFFFFFFF), np.uint64(32)
    for _ in range(rounds):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> s) ^ c[1] ^ np.uint64(k[0]), b & low, (a >> s) ^ c[3] ^ np.uint64(k[1]), a & low]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return c


def threshold(p) -> int:
    return int(np.rint(np.float64(np.float32(p)) * 65536))


def scale32(p) -> np.float32:
    t = threshold(p)
    return np.float32(65536.0 / (65536 - t)) if t < 65536 else np.float32(0)


def keep_mask(rows: int, cols: int, p, seed: int, offset: int = 0) -> torch.Tensor:
    blocks = -(-cols // 8)
    b = np.broadcast_to(np.arange(blocks, dtype=np.uint64), (rows, blocks))
    r = np.broadcast_to(np.arange(rows, dtype=np.uint64)[:, None], (rows, blocks))
    seed, offset = seed & (2 ** 64 - 1), offset & (2 ** 64 - 1)
    words = philox4x32((b, r, offset & 0xFFFFFFFF, offset >> 32), (seed & 0xFFFFFFFF, seed >> 32))
    halves = np.stack([(np.broadcast_to(w, (rows, blocks)) >> np.uint64(sh)) & np.uint64(0xFFFF)
                       for w in words for sh in (0, 16)], axis=-1)
    return torch.from_numpy(halves.reshape(rows, -1)[:, :cols] >= threshold(p))


def dropped32(x, p, seed, offset=0):
    """fp32 dropout(x), each product rounded once."""
    m = keep_mask(x.numel() // x.shape[-1], x.shape[-1], p, seed, offset).reshape(x.shape)
    return torch.where(m, x.float() * float(scale32(p)), torch.zeros((), dtype=torch.float32))


def tree_sum32(sq: torch.Tensor) -> torch.Tensor:
    """The canonical pairwise sum of the last dimension, padded with zeros to
    a power of two: the sum of a block is the rounded sum of its halves."""
    n = sq.shape[-1]
    size = 1
    while size < n:
        size *= 2
    sq = torch.nn.functional.pad(sq, (0, size - n))
    while sq.shape[-1] > 1:
        sq = sq[..., 0::2] + sq[..., 1::2]
    return sq


def dropout_add_rmsnorm32(x, residual, weight, p, eps, seed, offset=0):
    """(out, residual_out), every fp32 operation rounded once."""
    acc = residual.float() + dropped32(x, p, seed, offset)
    mean = tree_sum32(acc * acc) / np.float32(x.shape[-1]).item()
    v = (mean + torch.tensor(eps, dtype=torch.float32)).numpy()
    inv = torch.from_numpy(np.float32(1) / np.sqrt(v))
    return ((acc * inv) * weight.float()).to(x.dtype), acc.to(x.dtype)


def rmsnorm_bwd64(dout, dres, h, weight, eps):
    """d, dweight in fp64, with the bounds of the fp32 kernels' errors."""
    g64, h64, w64 = dout.double(), h.double(), weight.double()
    inv = 1 / torch.sqrt(h64.square().mean(-1, keepdim=True) + float(np.float32(eps)))
    xh, g = h64 * inv, g64 * w64
    t = inv * (g - xh * (g * xh).mean(-1, keepdim=True))
    d = t + (0 if dres is None else dres.double())
    # A pairwise sum of P <= 2^15 squares (or products of two roundings) is
    # off by at most 17 roundings of its terms' magnitudes; inv by half of
    # the sum's 17 and 4 of its own operations (below 13); g by 1, h c by 2
    # inv, the mean and 4 products (below 50); 3 roundings for the rest.
    mags = inv * (g.abs() + xh.abs() * (g * xh).abs().mean(-1, keepdim=True))
    d_err = 64 * EPS32 * (mags + (0 if dres is None else dres.double().abs()))
    dw = (g64 * xh).reshape(-1, h.shape[-1]).sum(0)
    # every row's term: inv and two products (15 roundings); the sum: fewer
    # additions than rows in a CTA, its groups, parts of one warp and 5 more
    rows = h.numel() // h.shape[-1]
    adds = -(-rows // 152) + 32 + 20 + 5
    dw_err = (15 + min(rows + 5, adds)) * EPS32 * (g64 * xh).abs().reshape(-1, h.shape[-1]).sum(0)
    return d, d_err, dw, dw_err


def rotate64(x, angles, interleaved, scale, sign=1):
    """x: [b, s, heads, d] fp64; angles: [b, s, rot / 2] fp64."""
    c, s = (f(angles)[:, :, None] * scale for f in (torch.cos, lambda a: torch.sin(a) * sign))
    half = angles.shape[-1]
    rot = 2 * half
    y = x.clone()
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * c - b * s, a * s + b * c
    else:
        a, b = x[..., :half], x[..., half:rot]
        y[..., :half], y[..., half:rot] = a * c - b * s, a * s + b * c
    return y


def partner_sum(x, half, interleaved):
    """|a| + |b| of each column's pair; |x| past the turning columns."""
    rot = 2 * half
    m = x.abs().clone()
    if interleaved:
        t = m[..., 0:rot:2] + m[..., 1:rot:2]
        m[..., 0:rot:2], m[..., 1:rot:2] = t, t
    else:
        t = m[..., :half] + m[..., half:rot]
        m[..., :half], m[..., half:rot] = t, t
    return m


def rope_error(pair_sum, scale, turn_err=0.0):
    """How far a turned value may be from fp64: the angle (its top 32 bits
    rounded to fp32: pi 2^-25, plus 2 pi 2^-32, plus the caller's), cosine and
    sine within an ulp and their product with scale (3 roundings), 3 in the
    turn itself."""
    return abs(scale) * pair_sum * (np.pi * 2.0 ** -25 + 2 * np.pi * 2.0 ** -32 + turn_err + 7 * EPS32)


def assert_close(got, exact, err, what):
    """|got - exact| <= err + one rounding of a value within err of exact."""
    got, exact = got.detach().cpu(), exact.cpu()
    err = err.cpu() if torch.is_tensor(err) else torch.tensor(err, dtype=torch.float64)
    half = HALF_STEP[got.dtype]
    bound = err + half * (exact.abs() + err) + TINY[got.dtype]
    off = (got.double() - exact).abs()
    bad = ~(off <= bound)
    if bool(bad.any()):
        i = tuple(int(v) for v in bad.nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside the bound; first at {i}: got "
                             f"{float(got[i])}, exact {float(exact[i])}, bound {float(bound.expand_as(off)[i])}")


def assert_same_bits(got, expected, what):
    got, expected = got.detach().cpu().contiguous(), expected.contiguous()
    kind = torch.int32 if got.dtype == torch.float32 else torch.int16
    a, b = got.view(kind), expected.view(kind)
    nan = torch.isnan(got) & torch.isnan(expected)
    bad = (a != b) & ~nan
    if bool(bad.any()):
        i = tuple(int(v) for v in bad.nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} differ; first at {i}: got {float(got[i])}, "
                             f"expected {float(expected[i])}")
