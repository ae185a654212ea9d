"""Dropout, dropout + residual add + RMSNorm and its gradients on the GPU:
the forwards bit for bit against fp32 operations rounded one by one, the
gradients against fp64 within derived bounds."""
import ctypes
import itertools

import numpy as np
import pytest
import torch

import deterministic_residual_add_gb300 as dr
import train_refs as tr

pytestmark = pytest.mark.gpu

DTYPES = [torch.bfloat16, torch.float16, torch.float32]
SEED, OFFSET = 0xDEADBEEF12345678, (7 << 32) + 5
EPS = 1e-6


def cuda():
    return torch.device("cuda", 0)


def normal(shape, dtype, seed, std=1.0, mean=0.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std + mean).to(dtype)


# ------------------------------------------------------------------ dropout
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 8), (3, 7), (5, 64), (33, 255), (2, 257), (17, 1001), (300, 512),
                                       (1, 100003), (70001, 9), (1000, 4096)])
def test_dropout_bits(rows, cols, dtype):
    x = normal((rows, cols), dtype, rows + cols)
    r = normal((rows, cols), dtype, rows + cols + 1, std=2.0)
    for p in (0.0, 0.1, 0.5, 1.0):
        got = dr.dropout_fwd(x.to(cuda()), p, seed=SEED, offset=OFFSET)
        d = tr.dropped32(x, p, SEED, OFFSET)
        tr.assert_same_bits(got, d.to(dtype), f"dropout p={p}")
        got = dr.dropout_add_fwd(x.to(cuda()), r.to(cuda()), p, seed=SEED, offset=OFFSET)
        tr.assert_same_bits(got, (r.float() + d).to(dtype), f"dropout add p={p}")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("cols", [8, 9, 15, 17, 63, 65, 71, 100, 127, 250, 254, 257, 511, 1023])
def test_dropout_of_widths_no_vector_divides(cols, dtype):
    """Contiguous rows back to back: vectors across one or more row ends, at
    every phase, in more than one round of the grid for the narrow ones."""
    for rows in (1, 2, 7, 1000):
        x = normal((rows, cols), dtype, rows + cols)
        got = dr.dropout_fwd(x.to(cuda()), 0.4, seed=SEED, offset=OFFSET)
        tr.assert_same_bits(got, tr.dropped32(x, 0.4, SEED, OFFSET).to(dtype), f"{rows} rows")
    x = normal((40009, 257), dtype, 3)  # 40 MB of fp32: several rounds of the largest grid
    xd = x.to(cuda())
    got = dr.dropout_add_fwd(xd, xd, 0.4, seed=SEED, offset=OFFSET, residual_out=xd)
    tr.assert_same_bits(got, (x.float() + tr.dropped32(x, 0.4, SEED, OFFSET)).to(dtype), "in place")


@pytest.mark.parametrize("dtype", DTYPES)
def test_dropout_strided_rows_and_neighbours(dtype):
    """Row-strided and unaligned views: the mask follows (row, column) of the
    view, and nothing outside it is written."""
    for cols, left, width in [(64, 0, 128), (64, 64, 128), (61, 3, 100), (1000, 1, 1003), (8, 8, 24)]:
        base = normal((37, width), dtype, cols)
        x = base[:, left:left + cols]
        xd = base.to(cuda())[:, left:left + cols]
        out = torch.full((37, width), 7.0, dtype=dtype, device=cuda())
        view = out[:, left:left + cols]
        assert dr.dropout_fwd(xd, 0.3, seed=SEED, out=view) is view
        want = torch.full((37, width), 7.0, dtype=dtype)
        want[:, left:left + cols] = tr.dropped32(x.contiguous(), 0.3, SEED).to(dtype)
        tr.assert_same_bits(out, want, f"strided {cols}")
        dr.dropout_fwd(xd, 0.3, seed=SEED, out=xd)  # in place
        tr.assert_same_bits(xd, want[:, left:left + cols].contiguous(), f"in place {cols}")


def test_dropped_places_hold_anything():
    x = torch.full((40, 96), float("nan"))
    x[:, ::2], x[::2] = float("inf"), float("-inf")
    keep = tr.keep_mask(40, 96, 0.5, 9)
    for h in (96, 95):
        for dtype in DTYPES:
            got = dr.dropout_fwd(x[:, :h].to(dtype).to(cuda()), 0.5, seed=9).cpu().float()
            k = keep[:, :h]
            assert bool((got[~k] == 0).all()) and not bool(torch.signbit(got[~k]).any())
            assert bool((got[k].nan_to_num(3.0, 4.0, 5.0) == x[:, :h][k].nan_to_num(3.0, 4.0, 5.0)).all())


def test_dropout_empty_and_refused():
    assert dr.dropout_fwd(torch.empty(0, 64, device=cuda()), 0.1, seed=1).shape == (0, 64)
    assert dr.dropout_fwd(torch.empty(5, 0, device=cuda()), 0.1, seed=1).shape == (5, 0)
    x = torch.zeros(8, 64, device=cuda())
    for bad in (-0.5, 1.01, float("nan")):
        with pytest.raises(dr.DraddError):
            dr.dropout_fwd(x, bad, seed=1)
    with pytest.raises(ValueError):
        dr.dropout_fwd(x.t(), 0.1, seed=1)
    with pytest.raises(TypeError):
        dr.dropout_add_fwd(x, x.half(), 0.1, seed=1)
    with pytest.raises(ValueError):
        dr.dropout_add_fwd(x, x[:4], 0.1, seed=1)
    with pytest.raises(TypeError):
        dr.dropout_fwd(x, 0.1, seed=1, step=torch.zeros(1, device=cuda()))


def test_step_in_a_captured_graph():
    """A replay reads the counter: every step has its own mask, forward and
    backward of a step the same one, without another capture."""
    x, r = normal((64, 256), torch.bfloat16, 1).to(cuda()), normal((64, 256), torch.bfloat16, 2).to(cuda())
    w, dout = normal(256, torch.bfloat16, 3, 0.1, 1.0).to(cuda()), normal((64, 256), torch.bfloat16, 4).to(cuda())
    step = torch.zeros(1, dtype=torch.int64, device=cuda())

    def run():
        out, ro = dr.dropout_add_rmsnorm_fwd(x, r, w, 0.2, EPS, seed=5, offset=40, step=step)
        return (out, ro, *dr.dropout_add_rmsnorm_bwd(dout, None, ro, w, 0.2, EPS, seed=5, offset=40, step=step),
                dr.dropout_fwd(x, 0.2, seed=5, offset=40, step=step))

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        captured = run()
        step += 1
    for k in range(3):
        step.fill_(k)
        g.replay()
        torch.cuda.synchronize()
        out, ro = dr.dropout_add_rmsnorm_fwd(x, r, w, 0.2, EPS, seed=5, offset=40 + k)
        dx, dres, dw = dr.dropout_add_rmsnorm_bwd(dout, None, ro, w, 0.2, EPS, seed=5, offset=40 + k)
        want = (out, ro, dx, dres, dw, dr.dropout_fwd(x, 0.2, seed=5, offset=40 + k))
        for a, b in zip(captured, want):
            assert torch.equal(a, b)
        assert int(step) == k + 1


def test_step_and_the_offsets_of_layers():
    """The step is added to the offset: layers at neighbouring offsets have
    masks of their own in every replay when it advances by their number, and
    share them when it advances by one."""
    layers, p = 3, 0.5
    x = torch.ones(8, 256, dtype=torch.bfloat16, device=cuda())
    step = torch.zeros(1, dtype=torch.int64, device=cuda())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        held = [dr.dropout_fwd(x, p, seed=SEED, offset=i, step=step) for i in range(layers)]

    def masks(advance):
        got = []
        for replay in range(4):
            step.fill_(replay * advance)
            g.replay()
            got += [(h != 0).cpu() for h in held]
        return got

    for advance in (layers, 1):
        for i, m in enumerate(masks(advance)):
            offset = i // layers * advance + i % layers
            assert torch.equal(m, tr.keep_mask(8, 256, p, SEED, offset))
    assert len({m.numpy().tobytes() for m in masks(layers)}) == 4 * layers
    assert len({m.numpy().tobytes() for m in masks(1)}) == layers + 3


# ------------------------------------- dropout + residual add + RMSNorm
HIDDENS = [8, 64, 72, 128, 200, 256, 504, 512, 1000, 1024, 1032, 2048, 4096, 5000, 8192, 8200, 16384, 32768]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("hidden", HIDDENS)
def test_norm_forward_bits(hidden, dtype):
    rows = 21 if hidden > 2048 else 133
    x, r = normal((rows, hidden), dtype, hidden), normal((rows, hidden), dtype, hidden + 1, std=2.0)
    w = normal(hidden, dtype, hidden + 2, 0.1, 1.0)
    for p in (0.0, 0.1):
        out, ro = dr.dropout_add_rmsnorm_fwd(x.to(cuda()), r.to(cuda()), w.to(cuda()), p, EPS, seed=SEED,
                                             offset=OFFSET)
        want, want_ro = tr.dropout_add_rmsnorm32(x, r, w, p, EPS, SEED, OFFSET)
        tr.assert_same_bits(ro, want_ro, f"residual_out p={p}")
        tr.assert_same_bits(out, want, f"out p={p}")
        if p == 0.0 and dtype == torch.bfloat16:
            a, b = dr.add_rmsnorm_fwd(x.to(cuda()), r.to(cuda()), w.to(cuda()), EPS)
            assert torch.equal(a, out) and torch.equal(b, ro)


@pytest.mark.parametrize("rows", [1, 2, 7, 151, 153, 607, 1000, 5001])
@pytest.mark.parametrize("hidden", [64, 1024, 4096])
def test_norm_forward_row_counts(rows, hidden):
    """More rows than a CTA, a wave and the ring take."""
    x, r = normal((rows, hidden), torch.bfloat16, rows), normal((rows, hidden), torch.bfloat16, rows + 1)
    w = normal(hidden, torch.bfloat16, 5, 0.1, 1.0)
    out, ro = dr.dropout_add_rmsnorm_fwd(x.to(cuda()), r.to(cuda()), w.to(cuda()), 0.1, EPS, seed=SEED)
    want, want_ro = tr.dropout_add_rmsnorm32(x, r, w, 0.1, EPS, SEED)
    tr.assert_same_bits(ro, want_ro, "residual_out")
    tr.assert_same_bits(out, want, "out")


def check_backward(rows, hidden, dtype, p, dres=True, eps=EPS, h=None):
    h = normal((rows, hidden), dtype, rows + hidden, std=2.0) if h is None else h
    dout = normal((rows, hidden), dtype, rows + hidden + 1)
    dro = normal((rows, hidden), dtype, rows + hidden + 2) if dres else None
    w = normal(hidden, dtype, hidden + 3, 0.1, 1.0)
    on = [None if t is None else t.to(cuda()) for t in (dout, dro, h, w)]
    dx, d, dw = dr.dropout_add_rmsnorm_bwd(*on, p, eps, seed=SEED, offset=OFFSET)
    e, e_err, ew, ew_err = tr.rmsnorm_bwd64(dout, dro, h, w, eps)
    tr.assert_close(d, e, e_err, "dresidual")
    tr.assert_close(dw, ew, ew_err, "dweight")
    keep = tr.keep_mask(rows, hidden, p, SEED, OFFSET).double()
    t = tr.threshold(p)
    s = 65536 / (65536 - t) if t < 65536 else 0.0
    tr.assert_close(dx, e * keep * s, keep * s * (e_err + 2 * tr.EPS32 * e.abs()), "dx")
    assert bool((dx.cpu()[keep == 0] == 0).all())
    return on, (dx, d, dw)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("hidden", HIDDENS)
def test_norm_backward(hidden, dtype):
    rows = 21 if hidden > 2048 else 133
    check_backward(rows, hidden, dtype, 0.1)


@pytest.mark.parametrize("rows", [1, 2, 7, 151, 153, 607, 1000, 5001])
@pytest.mark.parametrize("hidden", [64, 1024, 4096])
def test_norm_backward_row_counts(rows, hidden):
    check_backward(rows, hidden, torch.bfloat16, 0.1, dres=rows % 2 == 1)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("hidden", [1000, 4096])
def test_norm_backward_forms(hidden, dtype):
    """p = 0 and 1, no later gradient, no weight gradient, no dropout form,
    in place, a caller's workspace, and the same bits every time."""
    for p, dres in itertools.product((0.0, 1.0), (True, False)):
        on, (dx, d, dw) = check_backward(50, hidden, dtype, p, dres)
        dout, dro, h, w = on
        if p == 0.0:
            assert torch.equal(dx, d)
            dh, dw2 = dr.add_rmsnorm_bwd(dout, dro, h, w, EPS)
            assert torch.equal(dh, d) and torch.equal(dw2, dw)
            if not dres:
                dh, dw2 = dr.rmsnorm_bwd(dout, h, w, EPS)
                assert torch.equal(dh, d) and torch.equal(dw2, dw)
    on, (dx, d, dw) = check_backward(333, hidden, dtype, 0.25)
    dout, dro, h, w = on
    again = dr.dropout_add_rmsnorm_bwd(dout, dro, h, w, 0.25, EPS, seed=SEED, offset=OFFSET, weight_grad=False)
    assert again[2] is None and torch.equal(again[0], dx) and torch.equal(again[1], d)
    ws = torch.full((608 * hidden * 4,), 255, dtype=torch.uint8, device=cuda())
    again = dr.dropout_add_rmsnorm_bwd(dout, dro, h, w, 0.25, EPS, seed=SEED, offset=OFFSET, workspace=ws)
    assert all(torch.equal(a, b) for a, b in zip(again, (dx, d, dw)))
    with pytest.raises(dr.DraddError):
        dr.dropout_add_rmsnorm_bwd(dout, dro, h, w, 0.25, EPS, seed=SEED, workspace=ws[:64])
    for a, b in itertools.permutations(("dout", "dro", "h"), 2):
        t = {"dout": dout.clone(), "dro": dro.clone(), "h": h.clone()}
        got = dr.dropout_add_rmsnorm_bwd(t["dout"], t["dro"], t["h"], w, 0.25, EPS, seed=SEED, offset=OFFSET, dx=t[a],
                                         dresidual=t[b])
        assert got[0] is t[a] and torch.equal(t[a], dx) and torch.equal(t[b], d) and torch.equal(got[2], dw)
    x, r = dout.clone(), dro.clone()
    want = dr.dropout_add_rmsnorm_fwd(x, r, w, 0.25, EPS, seed=SEED)
    got = dr.dropout_add_rmsnorm_fwd(x, r, w, 0.25, EPS, seed=SEED, out=r, residual_out=x)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_norm_zero_rows_and_zero_inputs():
    w = torch.ones(4096, device=cuda())
    none = torch.empty(0, 4096, device=cuda())
    out, ro = dr.dropout_add_rmsnorm_fwd(none, none, w, 0.1, EPS, seed=1)
    assert out.shape == ro.shape == (0, 4096)
    dx, d, dw = dr.dropout_add_rmsnorm_bwd(none, None, none, w, 0.1, EPS, seed=1)
    assert dx.shape == (0, 4096) and bool((dw == 0).all())
    check_backward(9, 4096, torch.float32, 0.1, h=torch.zeros(9, 4096), eps=1e-2)
    check_backward(9, 64, torch.float32, 0.1, h=torch.zeros(9, 64), eps=1e-2)
    out, ro = dr.dropout_add_rmsnorm_fwd(torch.ones(3, 4096, device=cuda()), torch.zeros(3, 4096, device=cuda()), w,
                                         1.0, EPS, seed=1)
    assert bool((out == 0).all()) and bool((ro == 0).all())


def test_norm_gradients_against_differences():
    """Central differences of the fp32 forward along random directions.  The
    loss is a sum of n terms of size about 1 computed in fp64 from fp32
    outputs (each off by 2^-20 at most): the quotient with step 2^-7 is off
    by the third-order term, below step^2 of its size, and by the outputs'
    rounding over the step, below sqrt(n) 2^-20 2^7."""
    rows, hidden, p = 40, 512, 0.3
    x, r = normal((rows, hidden), torch.float32, 1), normal((rows, hidden), torch.float32, 2)
    w, c1, c2 = normal(hidden, torch.float32, 3, 0.1, 1.0), normal((rows, hidden), torch.float32, 4), normal(
        (rows, hidden), torch.float32, 5)
    x, r, w, c1, c2 = (t.to(cuda()) for t in (x, r, w, c1, c2))

    def loss(x, r, w):
        out, ro = dr.dropout_add_rmsnorm_fwd(x, r, w, p, EPS, seed=SEED)
        return float((out.double() * c1.double()).sum() + (ro.double() * c2.double()).sum())

    _, h = dr.dropout_add_rmsnorm_fwd(x, r, w, p, EPS, seed=SEED)
    grads = dr.dropout_add_rmsnorm_bwd(c1, c2, h, w, p, EPS, seed=SEED)
    step = 2.0 ** -7
    for i, g in enumerate(grads):
        v = normal(g.shape, torch.float32, 6 + i).to(cuda())
        v /= v.norm()
        args = [x, r, w]
        up, down = list(args), list(args)
        up[i], down[i] = args[i] + step * v, args[i] - step * v
        diff = (loss(*up) - loss(*down)) / (2 * step)
        want = float((g.double() * v.double()).sum())
        bound = step ** 2 * float(g.norm()) + (rows * hidden) ** 0.5 * 2.0 ** -13
        assert abs(diff - want) <= bound, (i, diff, want, bound)


def test_large_rows_and_offsets():
    """Elements past 2^31: the last rows of a tensor of 2^31 + 2^21 elements,
    in rows of 2048 and of 64 (more rows than 2^24)."""
    for cols in (2048, 64):
        rows = (2 ** 31 + 2 ** 21) // cols
        x = torch.ones(rows, cols, dtype=torch.bfloat16, device=cuda())
        got = dr.dropout_fwd(x, 0.5, seed=3, out=x)[-4:].cpu().float()
        b = np.broadcast_to(np.arange(cols // 8, dtype=np.uint64), (4, cols // 8))
        r = np.broadcast_to(np.arange(rows - 4, rows, dtype=np.uint64)[:, None], b.shape)
        words = tr.philox4x32((b, r, 0, 0), (3, 0))
        halves = np.stack([(w >> np.uint64(s)) & np.uint64(0xFFFF) for w in words for s in (0, 16)], axis=-1)
        assert torch.equal(got, torch.from_numpy(halves.reshape(4, cols) >= 32768).float() * 2)
        w = torch.ones(cols, dtype=torch.bfloat16, device=cuda())
        tail = torch.full((4, cols), 3.0, dtype=torch.bfloat16, device=cuda())
        x[-4:] = tail
        dh, _ = dr.add_rmsnorm_bwd(x, None, x, w, EPS, dh=x, weight_grad=False)
        want, _ = dr.add_rmsnorm_bwd(tail, None, tail, w, EPS, weight_grad=False)
        assert torch.equal(dh[-4:], want)
        del x, dh


def test_streams_and_pinned_memory():
    x, r = normal((64, 4096), torch.bfloat16, 1), normal((64, 4096), torch.bfloat16, 2)
    w, dout = normal(4096, torch.bfloat16, 3, 0.1, 1.0), normal((64, 4096), torch.bfloat16, 4)
    xd, rd, wd, dd = (t.to(cuda()) for t in (x, r, w, dout))
    want = dr.dropout_add_rmsnorm_fwd(xd, rd, wd, 0.1, EPS, seed=SEED)
    want_bwd = dr.dropout_add_rmsnorm_bwd(dd, None, want[1], wd, 0.1, EPS, seed=SEED)
    torch.cuda.synchronize()
    for stream in (torch.cuda.Stream(), torch.cuda.Stream().cuda_stream):
        got = dr.dropout_add_rmsnorm_fwd(xd, rd, wd, 0.1, EPS, seed=SEED, stream=stream)
        bwd = dr.dropout_add_rmsnorm_bwd(dd, None, got[1], wd, 0.1, EPS, seed=SEED, stream=stream)
        drop = dr.dropout_fwd(xd, 0.1, seed=SEED, stream=stream)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((*got, *bwd), (*want, *want_bwd)))
        tr.assert_same_bits(drop, tr.dropped32(x, 0.1, SEED).to(x.dtype), "dropout on another stream")
    # two backward passes at once on two streams, each with its own workspace
    streams = [torch.cuda.Stream() for _ in range(4)]
    many = [dr.dropout_add_rmsnorm_bwd(dd, None, want[1], wd, 0.1, EPS, seed=SEED, stream=s)
            for _ in range(8) for s in streams]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for got in many for a, b in zip(got, want_bwd))
    # buffers the device reaches over the host link take the direct kernels
    L = dr.lib()
    for name in ("dropout_fwd", "dropout_add_rmsnorm_fwd", "dropout_add_rmsnorm_bwd"):
        tr.c_entry(L, name)
    hx, hr, hw, hd = (t.pin_memory() for t in (x, r, w, dout))
    out, ro, dx, dres = (torch.empty_like(x).pin_memory() for _ in range(4))
    dw = torch.empty(4096, device=cuda())
    ws = torch.empty(L.rmsnorm_bwd_workspace_bytes(64, 4096, 0), dtype=torch.uint8, device=cuda())
    d = tr.CDropout(0.1, SEED, 0, None)
    s = torch.cuda.current_stream().cuda_stream
    assert L.dropout_add_rmsnorm_fwd(out.data_ptr(), ro.data_ptr(), hx.data_ptr(), hr.data_ptr(), hw.data_ptr(), EPS,
                                     64, 4096, ctypes.byref(d), 0, s) == 0
    assert L.dropout_add_rmsnorm_bwd(dx.data_ptr(), dres.data_ptr(), dw.data_ptr(), hd.data_ptr(), None,
                                     ro.data_ptr(), hw.data_ptr(), EPS, 64, 4096, ctypes.byref(d), 0, ws.data_ptr(),
                                     ws.numel(), s) == 0
    torch.cuda.synchronize()
    for a, b in zip((out, ro, dx, dres, dw), (*want, *want_bwd)):
        assert torch.equal(a.cpu(), b.cpu())
    # narrow rows, and dropout alone
    for n, h in ((50, 200), (50, 1000)):
        hx, hr, hw = (normal(sh, torch.bfloat16, 5 + i).pin_memory() for i, sh in enumerate(((n, h), (n, h), (h,))))
        out, ro, dx, dres = (torch.empty_like(hx).pin_memory() for _ in range(4))
        dw = torch.empty(h, device=cuda())
        want = dr.dropout_add_rmsnorm_fwd(hx.to(cuda()), hr.to(cuda()), hw.to(cuda()), 0.1, EPS, seed=SEED)
        want_bwd = dr.dropout_add_rmsnorm_bwd(hx.to(cuda()), None, want[1], hw.to(cuda()), 0.1, EPS, seed=SEED)
        assert L.dropout_add_rmsnorm_fwd(out.data_ptr(), ro.data_ptr(), hx.data_ptr(), hr.data_ptr(), hw.data_ptr(),
                                         EPS, n, h, ctypes.byref(d), 0, s) == 0
        assert L.dropout_add_rmsnorm_bwd(dx.data_ptr(), dres.data_ptr(), dw.data_ptr(), hx.data_ptr(), None,
                                         ro.data_ptr(), hw.data_ptr(), EPS, n, h, ctypes.byref(d), 0, ws.data_ptr(),
                                         ws.numel(), s) == 0
        torch.cuda.synchronize()
        for a, b in zip((out, ro, dx, dres, dw), (*want, *want_bwd)):
            assert torch.equal(a.cpu(), b.cpu())
        for cols in (h, h - 1):
            x = hx[:, :cols].contiguous().pin_memory()
            got = torch.empty_like(x).pin_memory()
            assert L.dropout_fwd(got.data_ptr(), cols, x.data_ptr(), cols, n, cols, ctypes.byref(d), 0, s) == 0
            torch.cuda.synchronize()
            tr.assert_same_bits(got, tr.dropped32(x, 0.1, SEED).to(x.dtype), "pinned dropout")
    assert dr.device_status() == 0
