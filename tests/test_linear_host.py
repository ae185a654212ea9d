"""The entry points of include/dradd_linear.h on the host, without a GPU:
argument checks, which return before any CUDA call, workspace sizes, and the
references themselves."""
import ctypes
import math

import pytest
import torch

import deterministic_residual_add_gb300 as dr
import linear_refs as lr
from deterministic_residual_add_gb300 import build as drbuild
from linear_refs import CMatrix, CTeacher
from test_train_host import ALIAS, ALIGN, ARG, BASE, HIDDEN, MB, NULL, OK, SHAPE, WORK, reaches_device

A, B, C, D, E, F, G, H, I, J = (BASE + i * 65536 * MB for i in range(10))
NAMES = ("linear_act_add_fwd", "linear_act_add_bwd", "linear_cross_entropy_fwd", "linear_cross_entropy_bwd",
         "linear_distill_fwd", "linear_distill_bwd")


@pytest.fixture(scope="module")
def L():
    drbuild.build()
    L = dr.lib()
    for name in NAMES:
        lr.c_entry(L, name)
        lr.c_entry(L, name + "_workspace_bytes")
    return L


def m(data, stride):
    return ctypes.byref(CMatrix(data, stride))


def fwd(L, out=A, x=B, w=C, bias=D, res=E, act=0, rows=40, inner=64, cols=32, dtype=0, ws=H, wsb=1 << 40, os=32, xs=64,
        wst=64, rs=32):
    return L.linear_act_add_fwd(m(out, os), m(x, xs), m(w, wst), bias, m(res, rs), act, rows, inner, cols, dtype, ws, wsb,
                                None)


def bwd(L, dx=A, dw=B, db=C, dout=D, x=E, w=F, bias=G, act=4, rows=40, inner=64, cols=32, dtype=0, ws=H, wsb=1 << 40):
    return L.linear_act_add_bwd(dx, dw, db, m(dout, cols), m(x, inner), m(w, inner), bias, act, rows, inner, cols, dtype,
                                ws, wsb, None)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), ARG), (dict(dtype=-1), ARG), (dict(act=5), ARG), (dict(act=-1), ARG), (dict(rows=-1), SHAPE),
    (dict(rows=1 << 31), SHAPE), (dict(rows=(1 << 31) - 4095), SHAPE), (dict(inner=0), SHAPE),
    (dict(inner=60), HIDDEN), (dict(cols=0), SHAPE),
    (dict(cols=28), HIDDEN), (dict(inner=1 << 24), HIDDEN), (dict(cols=1 << 24), HIDDEN),
    (dict(rows=(1 << 31) - 4096, inner=(1 << 24) - 8), SHAPE), (dict(inner=(1 << 24) - 8, cols=(1 << 24) - 8), SHAPE),
    (dict(out=0), NULL), (dict(x=0), NULL), (dict(w=0), NULL), (dict(out=A + 8), ALIGN), (dict(x=B + 2), ALIGN),
    (dict(bias=D + 8), ALIGN), (dict(res=E + 4), ALIGN), (dict(xs=68), ALIGN), (dict(os=36), ALIGN),
    (dict(wst=60), ALIGN), (dict(xs=56), SHAPE), (dict(wst=0), SHAPE), (dict(rs=24), SHAPE), (dict(rows=0), OK),
    (dict(rows=0, out=0, x=0, w=0), OK), (dict(out=B), ALIAS), (dict(out=C), ALIAS), (dict(out=D), ALIAS),
    (dict(out=E + 64), ALIAS), (dict(res=A, rs=40), ALIAS), (dict(xs=1 << 62), SHAPE),
    (dict(inner=4096, wst=4096, xs=4096, ws=0), WORK), (dict(inner=4096, wst=4096, xs=4096, wsb=16), WORK),
    (dict(inner=4096, wst=4096, xs=4096, ws=H + 8), ALIGN), (dict(inner=4096, wst=4096, xs=4096, ws=A), ALIAS),
])
def test_linear_argument_errors(L, kw, code):
    assert fwd(L, **kw) == code


def test_linear_layouts_that_pass(L):
    assert reaches_device(fwd(L))
    assert reaches_device(fwd(L, bias=0, res=0))
    assert reaches_device(fwd(L, out=E))                           # in place of the residual
    assert reaches_device(fwd(L, rows=1, os=0, xs=0, rs=0, ws=0))  # one row: strides unused
    assert reaches_device(fwd(L, rows=16, ws=0, wsb=0))            # few rows need no workspace
    assert reaches_device(fwd(L, out=B + 128, os=128, xs=128))     # the other half of x's rows
    assert reaches_device(L.linear_act_add_fwd(m(A, 32), m(B, 64), m(C, 64), None, None, 0, 8, 64, 32, 0, None, 0, None))


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), ARG), (dict(act=9), ARG), (dict(rows=-1), SHAPE), (dict(inner=20), HIDDEN), (dict(cols=20), HIDDEN),
    (dict(dout=0), NULL), (dict(x=0), NULL), (dict(w=0), NULL), (dict(dx=A + 8), ALIGN), (dict(dw=B + 8), ALIGN),
    (dict(db=C + 8), ALIGN), (dict(bias=G + 2), ALIGN), (dict(dx=D), ALIAS), (dict(dx=E), ALIAS), (dict(dw=F), ALIAS),
    (dict(dw=A + 16), ALIAS), (dict(db=A), ALIAS), (dict(ws=0), WORK), (dict(wsb=8), WORK), (dict(ws=E), ALIAS),
    (dict(dx=0, dw=0, db=0), OK),
])
def test_linear_bwd_argument_errors(L, kw, code):
    assert bwd(L, **kw) == code


def test_linear_bwd_layouts_that_pass(L):
    assert reaches_device(bwd(L))
    assert reaches_device(bwd(L, dx=0)) and reaches_device(bwd(L, dw=0)) and reaches_device(bwd(L, db=0, bias=0))
    need = L.linear_act_add_bwd_workspace_bytes(40, 64, 32, 4, 1, 1, 1)
    assert need >= 40 * 32 * 2 and bwd(L, wsb=need - 1) == WORK and reaches_device(bwd(L, wsb=need))
    assert L.linear_act_add_bwd_workspace_bytes(1 << 13, 1 << 12, 1 << 12, 0, 1, 1, 0) == 0  # nothing between
    assert L.linear_act_add_bwd_workspace_bytes(40, 60, 32, 4, 1, 1, 1) == 0
    assert L.linear_act_add_fwd_workspace_bytes(0, 64, 64) == 0


def ce_fwd(L, loss=A, lse=B, x=C, w=D, target=E, rows=40, hidden=64, vocab=33, dtype=0, ws=H, wsb=1 << 40):
    return L.linear_cross_entropy_fwd(loss, lse, m(x, hidden), m(w, hidden), target, -100, rows, hidden, vocab, dtype, ws,
                                      wsb, None)


def ce_bwd(L, dx=A, dw=B, dloss=C, ls=1, dlse=D, es=1, x=E, w=F, target=G, lse=I, rows=40, hidden=64, vocab=33, dtype=0,
           ws=H, wsb=1 << 40):
    return L.linear_cross_entropy_bwd(dx, dw, dloss, ls, dlse, es, m(x, hidden), m(w, hidden), target, -100, lse, rows,
                                      hidden, vocab, dtype, ws, wsb, None)


def teach(index=E, logits=F, dtype=2, top=5, temperature=1.0):
    return ctypes.byref(CTeacher(index, logits, dtype, top, temperature))


def di_fwd(L, t, rows=40, hidden=64, vocab=33, ws=H, wsb=1 << 40):
    return L.linear_distill_fwd(A, B, m(C, hidden), m(D, hidden), t, rows, hidden, vocab, 0, ws, wsb, None)


def di_bwd(L, t, dx=A, ws=H, wsb=1 << 40):
    return L.linear_distill_bwd(dx, B, C, 1, None, 0, m(D, 64), m(G, 64), t, I, 40, 64, 33, 0, ws, wsb, None)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), ARG), (dict(rows=-1), SHAPE), (dict(rows=1 << 31), SHAPE), (dict(vocab=0), SHAPE),
    (dict(vocab=(1 << 30) + 1), SHAPE), (dict(hidden=0), SHAPE), (dict(hidden=12), HIDDEN), (dict(loss=0), NULL),
    (dict(rows=1 << 30, vocab=1 << 30), SHAPE),
    (dict(lse=0), NULL), (dict(x=0), NULL), (dict(w=0), NULL), (dict(target=0), NULL), (dict(loss=A + 2), ALIGN),
    (dict(x=C + 8), ALIGN), (dict(target=E + 4), ALIGN), (dict(loss=B), ALIAS), (dict(lse=C), ALIAS), (dict(ws=0), WORK),
    (dict(wsb=100), WORK), (dict(ws=D), ALIAS), (dict(rows=0), OK),
])
def test_cross_entropy_argument_errors(L, kw, code):
    assert ce_fwd(L, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), ARG), (dict(rows=-1), SHAPE), (dict(vocab=0), SHAPE), (dict(ls=2), SHAPE), (dict(es=-1), SHAPE),
    (dict(dloss=0), NULL), (dict(lse=0), NULL), (dict(target=0), NULL), (dict(dx=A + 8), ALIGN), (dict(dw=B + 2), ALIGN),
    (dict(dloss=C + 2), ALIGN), (dict(dx=B), ALIAS), (dict(dx=E), ALIAS), (dict(dw=F + 64), ALIAS), (dict(dx=G), ALIAS),
    (dict(ws=0), WORK), (dict(wsb=100), WORK), (dict(ws=I), ALIAS), (dict(dx=0, dw=0), OK),
])
def test_cross_entropy_bwd_argument_errors(L, kw, code):
    assert ce_bwd(L, **kw) == code


def test_losses_that_pass(L):
    assert reaches_device(ce_fwd(L)) and reaches_device(ce_bwd(L))
    assert reaches_device(ce_bwd(L, dlse=0)) and reaches_device(ce_bwd(L, ls=0, es=0)) and reaches_device(ce_bwd(L, dx=0))
    assert reaches_device(ce_fwd(L, wsb=L.linear_cross_entropy_fwd_workspace_bytes(40, 64, 33)))
    assert reaches_device(ce_bwd(L, wsb=L.linear_cross_entropy_bwd_workspace_bytes(40, 64, 33)))
    assert ce_bwd(L, wsb=L.linear_cross_entropy_bwd_workspace_bytes(40, 64, 33) - 1) == WORK
    assert reaches_device(di_fwd(L, teach())) and reaches_device(di_bwd(L, teach()))
    assert reaches_device(di_fwd(L, teach(), wsb=L.linear_distill_fwd_workspace_bytes(40, 64, 33, 5)))
    assert reaches_device(di_bwd(L, teach(), wsb=L.linear_distill_bwd_workspace_bytes(40, 64, 33, 5)))


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=3), ARG), (dict(temperature=0.0), ARG), (dict(temperature=-1.0), ARG), (dict(temperature=math.nan), ARG),
    (dict(temperature=math.inf), ARG), (dict(temperature=1e-45), ARG), (dict(top=0), SHAPE), (dict(top=1025), SHAPE),
    (dict(index=0), NULL), (dict(logits=0), NULL), (dict(index=E + 4), ALIGN), (dict(logits=F + 2), ALIGN),
])
def test_teacher_argument_errors(L, kw, code):
    assert di_fwd(L, teach(**kw)) == code and di_bwd(L, teach(**kw)) == code


def test_no_teacher(L):
    assert di_fwd(L, None) == NULL and di_bwd(L, None) == NULL
    assert di_bwd(L, teach(), dx=E) == ALIAS and di_bwd(L, teach(), ws=0) == WORK


def test_workspaces_stay_within_their_piece(L):
    """The largest listed sizes: dz of a piece is at most 256 MiB, and everything beside it is counted."""
    for rows, hidden, vocab in ((1, 64, 131072), (4096, 4096, 65536), (8192, 4096, 131072), (1 << 20, 1024, 50001)):
        n = L.linear_cross_entropy_bwd_workspace_bytes(rows, hidden, vocab)
        piece = max(256 << 20, rows * 512)
        # the rows of x, partial sums of dx (at most 32, where few rows make splits worth it), factors
        assert n <= piece + rows * hidden * (2 + 4 * 32) + rows * 16 + 4096
    assert L.linear_cross_entropy_fwd_workspace_bytes(4096, 4096, 128000) == 500 * 2 * 4096 * 8 + 4096 * 4
    for bad in ((0, 64, 10), (10, 60, 10), (10, 64, 0), (-1, 64, 10)):
        assert L.linear_cross_entropy_fwd_workspace_bytes(*bad) == 0
        assert L.linear_cross_entropy_bwd_workspace_bytes(*bad) == 0
        assert L.linear_distill_fwd_workspace_bytes(*bad, 4) == 0
    assert L.linear_distill_fwd_workspace_bytes(10, 64, 10, 0) == 0
    assert L.linear_distill_bwd_workspace_bytes(10, 64, 10, 2000) == 0


# --------------------------------------------------------------- references
def test_reference_gradients_against_differences():
    g = torch.Generator().manual_seed(1)
    x, w, b, dout = (torch.randn(*s, generator=g, dtype=torch.float64).half() for s in ((3, 8), (5, 8), (5,), (3, 5)))
    for act in ("gelu", "gelu_tanh", "silu"):
        for got, k in zip(lr.linear_grads(dout, x, w, b, act), range(3)):
            t = [x.double(), w.double(), b.double()]
            for at in ((0,) * t[k].dim(), (2, 3)[:t[k].dim()]):
                f = []
                for h in (-1e-6, 1e-6):
                    u = [v.clone() for v in t]
                    u[k][at] += h
                    f.append(float((lr.act64(u[0] @ u[1].t() + u[2], act) * dout.double()).sum()))
                assert abs(float(got[0][at]) - (f[1] - f[0]) / 2e-6) < 1e-6


def test_reference_loss_gradients_are_autograd_s():
    g = torch.Generator().manual_seed(2)
    x, w = (torch.randn(*s, generator=g).bfloat16() for s in ((6, 8), (11, 8)))
    index, logits = torch.stack([torch.randperm(11, generator=g)[:4] for _ in range(6)]), torch.randn(6, 4, generator=g)
    index[2] = -1
    index[3, 1] = -1
    share = lr.shares64(index, logits, 2.0)
    dloss, dlse = torch.rand(6, generator=g), torch.rand(6, generator=g)
    a, b = x.double().requires_grad_(), w.double().requires_grad_()
    z = a @ b.t() / 2.0
    lse = torch.logsumexp(z, 1)
    loss = (share * (torch.where(share > 0, share, 1.0).log() - z.gather(1, index.clamp(min=0)) + lse[:, None])).sum(1)
    want = torch.autograd.grad((loss * dloss.double()).sum() + (lse * dlse.double()).sum(), [a, b])
    got = lr.loss_grads(dloss, dlse, x, w, index, share, lse.detach(), 2.0)
    for (exact, _), t in zip(got, want):
        assert float((exact - t).abs().max()) < 1e-12
    assert float((lr.loss(x, w, index, share, 2.0)[0] - loss.detach()).abs().max()) < 1e-12


def test_python_refusals_without_a_gpu():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    w = torch.zeros(8, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        dr.linear_act_add_fwd(x, w)
    with pytest.raises(TypeError, match="bfloat16 or float16"):
        dr.linear_act_add_fwd(x.float(), w)
    with pytest.raises(ValueError, match="activation"):
        dr.linear_act_add_bwd(x, x, w, activation="swish")
    with pytest.raises(TypeError, match="teacher_logits"):
        dr.linear_distill_fwd(x, w, torch.zeros(4, 2, dtype=torch.int64), None)
    with pytest.raises(ValueError, match="CUDA"):
        dr.linear_cross_entropy_fwd(x, w, torch.zeros(4, dtype=torch.int64), stream=5)
