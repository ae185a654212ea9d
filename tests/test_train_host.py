"""Dropout, RMSNorm gradient and rotary entry points on the host, without a
GPU: argument checks, which return before any CUDA call, the generator's
published test values, the frequencies, and the references themselves."""
import ctypes
import math

import numpy as np
import pytest
import torch

import deterministic_residual_add_gb300 as dr
import train_refs as tr
from deterministic_residual_add_gb300 import build as drbuild
from train_refs import CDropout as _Dropout, CHeads as _Heads, CRope as _Rope

MB = 1 << 20
BASE = 1 << 42
A, B, C, D, E, F, G, H, I = (BASE + i * 4096 * MB for i in range(9))
OK, NULL, SHAPE, HIDDEN, ALIGN, EPS, ALIAS, ARG, WORK = 0, 1, 2, 3, 4, 5, 6, 11, 12


def reaches_device(status):
    """The checks passed: what is left is the device, absent here."""
    return status not in (NULL, SHAPE, HIDDEN, ALIGN, EPS, ALIAS, ARG, WORK)


@pytest.fixture(scope="module")
def L():
    drbuild.build()
    L = dr.lib()
    for name in ("dropout_fwd", "dropout_add_fwd", "dropout_add_rmsnorm_fwd", "dropout_add_rmsnorm_bwd",
                 "add_rmsnorm_bwd", "rope_fwd", "rope_bwd", "qk_rmsnorm_rope_fwd", "qk_rmsnorm_rope_bwd"):
        tr.c_entry(L, name)
    return L


@pytest.mark.parametrize("rounds,counter,key,out", [
    (7, (0,) * 4, (0,) * 2, (0x5f6fb709, 0x0d893f64, 0x4f121f81, 0x4f730a48)),
    (10, (0,) * 4, (0,) * 2, (0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8)),
    (10, (0xffffffff,) * 4, (0xffffffff,) * 2, (0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd)),
    (10, (0x243f6a88, 0x85a308d3, 0x13198a2e, 0x03707344), (0xa4093822, 0x299f31d0),
     (0xd16cfe09, 0x94fdcceb, 0x5001e420, 0x24126ea1)),
])
def test_generator_known_answers(rounds, counter, key, out):
    assert tuple(int(v) for v in tr.philox4x32(counter, key, rounds)) == out


def test_mask_rates_and_independence():
    """Kept shares within 5 standard deviations of 1 - p, for every 16-bit
    lane, and masks of neighbouring seeds, offsets and rows uncorrelated."""
    rows, cols, p = 400, 1000, 0.1
    m = tr.keep_mask(rows, cols, p, 5, 3).double()
    q = 1 - tr.threshold(p) / 65536
    for lane in range(8):
        part = m[:, lane::8]
        assert abs(part.mean() - q) < 5 * math.sqrt(q * (1 - q) / part.numel())
    for other in (tr.keep_mask(rows, cols, p, 6, 3), tr.keep_mask(rows, cols, p, 5, 4),
                  tr.keep_mask(rows, cols, p, 5, 3 + (1 << 32)), tr.keep_mask(rows, cols, p, 5 + (1 << 32), 3),
                  m.roll(1, 0), m.roll(1, 1)):
        corr = ((m - q) * (other.double() - q)).mean() / (q * (1 - q))
        assert abs(corr) < 5 / math.sqrt(m.numel())


# ------------------------------------------------------------------ dropout
def drop(L, out=A, os=64, x=B, xs=64, n=4, h=64, p=0.1, step=None, dtype=0, none=False):
    d = _Dropout(p, 1, 2, step)
    return L.dropout_fwd(out, os, x, xs, n, h, None if none else ctypes.byref(d), dtype, None)


def drop_add(L, out=A, os=64, x=B, xs=64, r=C, rs=64, n=4, h=64, p=0.1, dtype=0):
    d = _Dropout(p, 1, 2, None)
    return L.dropout_add_fwd(out, os, x, xs, r, rs, n, h, ctypes.byref(d), dtype, None)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=3), ARG), (dict(dtype=-1), ARG), (dict(p=-0.1), ARG), (dict(p=1.5), ARG), (dict(p=math.nan), ARG),
    (dict(none=True), NULL), (dict(n=-1), SHAPE), (dict(n=1 << 31), SHAPE), (dict(h=0), SHAPE),
    (dict(h=1 << 31), SHAPE), (dict(xs=63), SHAPE), (dict(os=10), SHAPE), (dict(out=0), NULL), (dict(x=0), NULL),
    (dict(out=A + 1), ALIGN), (dict(x=B + 2, dtype=2), ALIGN), (dict(step=D + 4), ALIGN), (dict(n=0), OK),
    (dict(n=0, out=0, x=0), OK), (dict(out=B + 2), ALIAS), (dict(out=B + 128), ALIAS),
    (dict(out=B, os=128), ALIAS), (dict(step=A), ALIAS), (dict(xs=1 << 62, os=1 << 62), SHAPE),
])
def test_dropout_argument_errors(L, kw, code):
    assert drop(L, **kw) == code


def test_dropout_layouts_that_pass(L):
    assert reaches_device(drop(L, out=B))                                 # in place
    assert reaches_device(drop(L, n=1, xs=0, os=0))                       # one row: strides unused
    assert reaches_device(drop(L, out=A + 2, x=B + 6, h=61))              # odd width, element alignment
    assert reaches_device(drop(L, out=B + 128, os=128, xs=128))           # the other half of the same rows
    assert drop(L, out=B + 126, os=128, xs=128) == ALIAS                  # one element into it
    assert reaches_device(drop_add(L, out=C))
    assert drop_add(L, out=C + 2) == ALIAS
    assert drop_add(L, r=0) == NULL and drop_add(L, rs=3) == SHAPE and drop_add(L, r=C + 1) == ALIGN


# ------------------------------------- dropout + residual add + RMSNorm
def fwd(L, out=A, ro=B, x=C, r=D, w=E, eps=1e-6, n=4, h=1024, p=0.1, step=None, dtype=0):
    d = _Dropout(p, 1, 2, step)
    return L.dropout_add_rmsnorm_fwd(out, ro, x, r, w, eps, n, h, ctypes.byref(d), dtype, None)


def bwd(L, dx=A, dres=B, dw=C, dout=D, dro=E, h_=F, w=G, eps=1e-6, n=4, h=1024, p=0.1, dtype=0, ws=H, wsb=1 << 24):
    d = _Dropout(p, 1, 2, None)
    return L.dropout_add_rmsnorm_bwd(dx, dres, dw, dout, dro, h_, w, eps, n, h, ctypes.byref(d), dtype, ws, wsb, None)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=9), ARG), (dict(p=2.0), ARG), (dict(n=-1), SHAPE), (dict(n=1 << 31), SHAPE), (dict(h=0), SHAPE),
    (dict(h=1001), HIDDEN), (dict(h=32776), HIDDEN), (dict(eps=-1.0), EPS), (dict(eps=math.inf), EPS),
    (dict(n=0, out=0, x=0), OK), (dict(out=0), NULL), (dict(ro=0), NULL), (dict(x=0), NULL), (dict(r=0), NULL),
    (dict(w=0), NULL), (dict(out=A + 8), ALIGN), (dict(w=E + 2), ALIGN), (dict(out=B), ALIAS),
    (dict(out=C + 16), ALIAS), (dict(ro=E), ALIAS), (dict(out=E + 16), ALIAS), (dict(step=A), ALIAS),
])
def test_norm_forward_argument_errors(L, kw, code):
    assert fwd(L, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=9), ARG), (dict(p=-1.0), ARG), (dict(n=-1), SHAPE), (dict(h=12), HIDDEN), (dict(eps=math.nan), EPS),
    (dict(dres=0), NULL), (dict(dout=0), NULL), (dict(h_=0), NULL), (dict(w=0), NULL), (dict(dx=A + 4), ALIGN),
    (dict(dw=C + 2), ALIGN), (dict(dro=E + 4), ALIGN), (dict(ws=H + 8), ALIGN), (dict(ws=0), WORK),
    (dict(wsb=4 * 1024 - 1, n=1), WORK), (dict(dx=B), ALIAS), (dict(dx=D + 16), ALIAS), (dict(dres=G), ALIAS),
    (dict(dw=B), ALIAS), (dict(dw=F), ALIAS), (dict(ws=D), ALIAS), (dict(ws=C), ALIAS), (dict(n=0, dw=0), OK),
])
def test_norm_backward_argument_errors(L, kw, code):
    assert bwd(L, **kw) == code


def test_norm_backward_layouts_that_pass(L):
    assert reaches_device(bwd(L, dx=0, dro=0, dw=0, ws=0, wsb=0))
    assert reaches_device(bwd(L, dx=D, dres=E))
    assert reaches_device(bwd(L, dx=F, dres=D))
    assert reaches_device(fwd(L, out=C, ro=D)) and reaches_device(fwd(L, out=D, ro=C))


@pytest.mark.parametrize("dtype", [0, 1, 2])
def test_norm_workspace(L, dtype):
    """Whole partial sums of hidden floats, as many as rows at most, and
    enough for the call that asked."""
    for n in (1, 7, 152, 5000):
        for h in (8, 64, 1000, 1024, 1032, 2048, 5120, 8192, 16384, 32768):
            b = L.rmsnorm_bwd_workspace_bytes(n, h, dtype)
            assert b % (4 * h) == 0 and 4 * h <= b <= 4 * h * min(n, 608)
            assert bwd(L, n=n, h=h, dtype=dtype, wsb=b - 1) == WORK
            assert reaches_device(bwd(L, n=n, h=h, dtype=dtype, wsb=b))
    assert L.rmsnorm_bwd_workspace_bytes(0, 64, dtype) == 0
    assert L.rmsnorm_bwd_workspace_bytes(5, 63, dtype) == 0
    assert L.rmsnorm_bwd_workspace_bytes(5, 64, 7) == 0


# ------------------------------------------------------------------- rotary
def rope_of(**kw):
    f = dict(batch=2, seq=16, q_heads=4, k_heads=2, head_dim=128, rot_dim=128, interleaved=0, inv_freq=H,
             positions=None, position0=0, scale=1.0)
    f.update(kw)
    return _Rope(**f)


def bshd(data, heads, d=128, s=16):
    return _Heads(data, s * heads * d, heads * d, d)


def rope(L, qo=None, ko=None, q=None, k=None, dtype=0, **kw):
    r = rope_of(**kw)
    heads = (qo or bshd(A, 4), ko or bshd(B, 2), q or bshd(C, 4), k or bshd(D, 2))
    return L.rope_fwd(*map(ctypes.byref, heads), ctypes.byref(r), dtype, None)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=4), ARG), (dict(interleaved=2), ARG), (dict(scale=math.inf), ARG), (dict(batch=-1), SHAPE),
    (dict(seq=-2), SHAPE), (dict(q_heads=0), SHAPE), (dict(k_heads=-1), SHAPE), (dict(head_dim=0), SHAPE),
    (dict(rot_dim=0), SHAPE), (dict(rot_dim=63), SHAPE), (dict(rot_dim=130), SHAPE),
    (dict(head_dim=520, rot_dim=8), HIDDEN), (dict(head_dim=512, rot_dim=8), HIDDEN),
    (dict(q_heads=65537), SHAPE), (dict(batch=1 << 20, seq=1 << 20), SHAPE), (dict(batch=0), OK), (dict(seq=0), OK),
    (dict(inv_freq=None), NULL), (dict(inv_freq=H + 4), ALIGN), (dict(positions=I + 4), ALIGN),
    (dict(q=_Heads(0, 1, 1, 1)), NULL), (dict(qo=_Heads(A + 1, 8192, 512, 128)), ALIGN),
    (dict(qo=_Heads(A, -8192, 512, 128)), SHAPE), (dict(q=_Heads(C, 1 << 60, 512, 128)), SHAPE),
    (dict(qo=_Heads(A, 8192, 512, 0)), ALIAS), (dict(qo=_Heads(A, 0, 512, 128)), ALIAS),
    (dict(qo=_Heads(A, 8192, 511, 128)), ALIAS), (dict(ko=bshd(A, 2)), ALIAS), (dict(qo=bshd(D, 4)), ALIAS),
    (dict(qo=bshd(C + 2, 4)), ALIAS), (dict(ko=bshd(C, 2)), ALIAS), (dict(positions=A), ALIAS),
    (dict(inv_freq=B), ALIAS),
])
def test_rope_argument_errors(L, kw, code):
    assert rope(L, **kw) == code


def packed(data, first, total, d=128, s=16):
    """Heads first, ... of a packed [batch, seq, total, d] bf16 projection."""
    return _Heads(data + first * d * 2, s * total * d, total * d, d)


def test_rope_null_structures(L):
    r, q, none = rope_of(), bshd(A, 4), None
    assert L.rope_fwd(ctypes.byref(q), ctypes.byref(q), ctypes.byref(q), ctypes.byref(q), none, 0, None) == NULL
    for i in range(4):
        heads = [ctypes.byref(bshd(BASE + j * 4096 * MB, 4 if j % 2 == 0 else 2)) for j in range(4)]
        heads[i] = none
        assert L.rope_fwd(*heads, ctypes.byref(r), 0, None) == NULL
    alone = rope_of(k_heads=0)
    assert reaches_device(L.rope_fwd(ctypes.byref(bshd(A, 4)), none, ctypes.byref(bshd(B, 4)), none,
                                     ctypes.byref(alone), 0, None))


def test_rope_layouts_that_the_checks_pass(L):
    """Launches without a device fail with the CUDA status, after the checks."""
    q, k = packed(A, 0, 8), packed(A, 4, 8)
    for call in (rope(L), rope(L, qo=q, ko=k, q=q, k=k),            # in place in one packed tensor
                 rope(L, q=_Heads(C, 0, 0, 128)),                   # an expanded input
                 rope(L, qo=_Heads(A, 8192, 128, 2048)),            # heads before the sequence
                 rope(L, k_heads=0, ko=_Heads(0, 0, 0, 0), k=_Heads(0, 0, 0, 0)),
                 rope(L, batch=1, seq=1, qo=_Heads(A, 0, 0, 128)),  # strides of single elements are unused
                 rope(L, head_dim=512, rot_dim=512, qo=bshd(A, 4, 512), ko=bshd(B, 2, 512), q=bshd(C, 4, 512),
                      k=bshd(D, 2, 512))):
        assert reaches_device(call)
    # one head of q_out shared with k_out, one element of overlap between rows
    assert rope(L, qo=packed(A, 0, 8), ko=packed(A, 3, 8), q=bshd(C, 4), k=bshd(D, 2)) == ALIAS
    assert rope(L, qo=packed(A, 0, 8), ko=packed(A, 4, 8), q=packed(A, 4, 8)) == ALIAS
    assert rope(L, qo=packed(A, 0, 6), ko=packed(A, 5, 6)) == ALIAS


def norm_rope(L, qw=E, kw_=F, q_eps=1e-6, k_eps=1e-6, **kw):
    r = rope_of(**kw)
    heads = (bshd(A, 4), bshd(B, 2), bshd(C, 4), bshd(D, 2))
    return L.qk_rmsnorm_rope_fwd(*map(ctypes.byref, heads), qw, kw_, q_eps, k_eps, ctypes.byref(r), 0, None)


def norm_rope_bwd(L, dq=None, dk=None, dqw=None, dkw=None, gq=None, q=None, ws=None, wsb=0, batch=2, k_heads=2):
    r = rope_of(batch=batch, k_heads=k_heads)
    h = [ctypes.byref(t) for t in (dq or bshd(A, 4), dk or bshd(B, 2), gq or bshd(C, 4), bshd(D, 2), q or bshd(E, 4),
                                   bshd(F, 2))]
    return L.qk_rmsnorm_rope_bwd(*h[:2], dqw, dkw, *h[2:], G, G + 4096, 1e-6, 1e-6, ctypes.byref(r), 0, ws, wsb, None)


def test_norm_rope_argument_errors(L):
    assert norm_rope(L, qw=0) == NULL and norm_rope(L, kw_=0) == NULL and norm_rope(L, qw=E + 1) == ALIGN
    assert norm_rope(L, q_eps=-1.0) == EPS and norm_rope(L, k_eps=math.nan) == EPS
    assert norm_rope(L, qw=A) == ALIAS
    assert reaches_device(norm_rope(L))
    assert reaches_device(norm_rope_bwd(L))
    assert reaches_device(norm_rope_bwd(L, dq=bshd(C, 4), dk=bshd(F, 2)))
    need = L.qk_rmsnorm_rope_bwd_workspace_bytes(ctypes.byref(rope_of()), 0)
    assert need > 0 and need % (2 * 128 * 4) == 0
    assert norm_rope_bwd(L, dqw=I, ws=0) == WORK and norm_rope_bwd(L, dqw=I, ws=I + 4096, wsb=need - 1) == WORK
    assert norm_rope_bwd(L, dqw=I + 2) == ALIGN and norm_rope_bwd(L, dqw=I, ws=I + 8, wsb=need) == ALIGN
    assert norm_rope_bwd(L, dqw=I, dkw=I, ws=I + 4096, wsb=need) == ALIAS
    assert norm_rope_bwd(L, dqw=A, ws=I + 4096, wsb=need) == ALIAS
    assert norm_rope_bwd(L, dkw=I, ws=E, wsb=need) == ALIAS
    assert reaches_device(norm_rope_bwd(L, dkw=I, ws=I + 4096, wsb=need))
    assert norm_rope_bwd(L, dq=bshd(D, 4)) == ALIAS
    assert L.qk_rmsnorm_rope_bwd_workspace_bytes(ctypes.byref(rope_of(batch=0)), 0) == 0
    assert L.qk_rmsnorm_rope_bwd_workspace_bytes(ctypes.byref(rope_of(rot_dim=3)), 0) == 0


def test_norm_rope_gradient_without_k_heads(L):
    """dk_weight is an output there too (zeros), so its checks hold; it needs
    no workspace."""
    assert norm_rope_bwd(L, dkw=I + 2, k_heads=0) == ALIGN
    assert norm_rope_bwd(L, dkw=A, k_heads=0) == ALIAS and norm_rope_bwd(L, dkw=E, k_heads=0) == ALIAS
    assert reaches_device(norm_rope_bwd(L, dkw=I, k_heads=0))
    assert reaches_device(norm_rope_bwd(L, dkw=B, k_heads=0))  # k's tensors are not looked at
    assert norm_rope_bwd(L, dqw=I, dkw=I + 1024, k_heads=0) == WORK


def test_rope_frequencies(L):
    i = np.arange(32)
    f = 500.0 ** (-2.0 * i / 64)
    assert np.allclose(dr.rope_frequencies(64, 500.0).numpy(), f, rtol=1e-14)
    assert np.allclose(dr.rope_frequencies(64, 500.0, scaling="linear", factor=8).numpy(), f / 8, rtol=1e-14)
    wide = dr.rope_frequencies(64, 500.0, scaling="base", factor=8).numpy()
    assert np.allclose(wide, (500.0 * 8 ** (64 / 62)) ** (-2.0 * i / 64), rtol=1e-13)
    assert wide[0] == 1.0 and math.isclose(wide[-1], f[-1] / 8, rel_tol=1e-13)
    parts = dr.rope_frequencies(64, 500.0, scaling="by_parts", factor=8, original_length=512, low=1, high=32).numpy()
    turns = 512 * f / (2 * math.pi)
    assert np.allclose(parts[turns >= 32], f[turns >= 32], rtol=1e-15) and (turns >= 32).any()
    assert np.allclose(parts[turns <= 1], f[turns <= 1] / 8, rtol=1e-15) and (turns <= 1).any()
    mid = (turns > 1) & (turns < 32)
    r = (turns - 1) / 31
    assert mid.any() and np.allclose(parts[mid], (f * (r + (1 - r) / 8))[mid], rtol=1e-13)
    for kw in (dict(rot_dim=0), dict(rot_dim=7), dict(rot_dim=514), dict(rot_dim=64, base=0.0),
               dict(rot_dim=64, base=math.inf), dict(rot_dim=64, scaling="linear", factor=0.5),
               dict(rot_dim=64, scaling="linear", factor=math.nan), dict(rot_dim=2, scaling="base", factor=2.0),
               dict(rot_dim=64, scaling="by_parts", factor=2.0),
               dict(rot_dim=64, scaling="by_parts", factor=2.0, original_length=10, low=3, high=3)):
        with pytest.raises(dr.DraddError):
            dr.rope_frequencies(**kw)
    with pytest.raises(ValueError):
        dr.rope_frequencies(64, scaling="other")


def test_binding_refuses_host_tensors_and_types(L):
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    q = torch.zeros(1, 4, 2, 64, dtype=torch.bfloat16)
    w, f = torch.ones(64, dtype=torch.bfloat16), dr.rope_frequencies(64)
    for call in (lambda: dr.dropout_fwd(x, 0.1, seed=1), lambda: dr.dropout_add_fwd(x, x, 0.1, seed=1),
                 lambda: dr.dropout_add_rmsnorm_fwd(x, x, w, 0.1, seed=1),
                 lambda: dr.dropout_add_rmsnorm_bwd(x, x, x, w, 0.1, seed=1), lambda: dr.add_rmsnorm_bwd(x, x, x, w),
                 lambda: dr.rmsnorm_bwd(x, x, w), lambda: dr.rope_fwd(q, q, f), lambda: dr.rope_bwd(q, q, f),
                 lambda: dr.qk_rmsnorm_rope_fwd(q, q, w, w, f), lambda: dr.qk_rmsnorm_rope_bwd(q, q, q, q, w, w, f)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        dr.dropout_fwd(x.double(), 0.1, seed=1)


def test_binding_checks_types_before_anything_else(L):
    """Arguments that are not tensors or numbers, and a wrong number of them."""
    from deterministic_residual_add_gb300 import _binding, train
    x = torch.zeros(4, 64)
    for call in (lambda: dr.dropout_fwd(None, 0.1, seed=1), lambda: dr.dropout_fwd([1.0], 0.1, seed=1),
                 lambda: dr.dropout_add_fwd(x, None, 0.1, seed=1), lambda: dr.rope_fwd("q", None, None),
                 lambda: dr.dropout_add_rmsnorm_fwd(x, x, None, 0.1, seed=1),
                 lambda: _binding.dropout(x), lambda: _binding.rope()):
        with pytest.raises(TypeError):
            call()
    assert train._C is _binding


def test_references_agree_with_autograd():
    g = torch.Generator().manual_seed(3)
    h, dout, dres = (torch.randn(9, 40, generator=g, dtype=torch.float64, requires_grad=i == 0) for i in range(3))
    w = torch.randn(40, generator=g, dtype=torch.float64, requires_grad=True)
    y = h * (h.square().mean(-1, keepdim=True) + float(np.float32(1e-3))).rsqrt() * w
    dh, dw = torch.autograd.grad([y, h * 1.0], [h, w], [dout, dres])
    d, _, dw2, _ = tr.rmsnorm_bwd64(dout, dres, h.detach(), w.detach(), 1e-3)
    assert torch.allclose(d, dh, rtol=1e-12, atol=1e-12) and torch.allclose(dw, dw2, rtol=1e-12, atol=1e-12)
    x = torch.randn(2, 3, 4, 10, generator=g, dtype=torch.float64)
    ang = torch.randn(2, 3, 4, generator=g, dtype=torch.float64)
    for inter in (False, True):
        y = tr.rotate64(x, ang, inter, 1.0)
        assert torch.allclose(tr.rotate64(y, ang, inter, 1.0, sign=-1), x, atol=1e-12)
        z = torch.view_as_complex((x[..., :8].unflatten(-1, (4, 2)) if inter
                                   else x[..., :8].unflatten(-1, (2, 4)).transpose(-1, -2)).contiguous())
        z = z * torch.polar(torch.ones_like(ang), ang)[:, :, None]
        back = torch.view_as_real(z)
        back = back.flatten(-2) if inter else back.transpose(-1, -2).flatten(-2)
        assert torch.allclose(y[..., :8], back, atol=1e-12) and torch.equal(y[..., 8:], x[..., 8:])
