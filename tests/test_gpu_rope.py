"""Rotary positions of q and k, plain and behind their RMSNorm, and the
gradients, on the GPU against fp64 within derived bounds."""
import ctypes
import itertools
from fractions import Fraction

import numpy as np
import pytest
import torch

import deterministic_residual_add_gb300 as dr
import train_refs as tr

pytestmark = pytest.mark.gpu

DTYPES = [torch.bfloat16, torch.float16, torch.float32]
EPS = 1e-6
# 1 / (2 pi) to 60 digits
INV_TAU = Fraction(159154943091895335768883763372514362034459645740456448747667, 10 ** 60)


def cuda():
    return torch.device("cuda", 0)


def normal(shape, dtype, seed, std=1.0, mean=0.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std + mean).to(dtype)


def case(b, s, hq, hk, d, dtype, seed=0):
    """q and k as slices of a packed projection beside v, on the host."""
    packed = normal((b, s, hq + 2 * hk, d), dtype, seed + b * s + d)
    return packed, packed[:, :, :hq], packed[:, :, hq:hq + hk]


def angles_of(positions, freq):
    return positions.double()[..., None] * freq


def turn_bound(positions):
    """fp64 rounding of the angle, in the kernel's fraction and in the
    reference: three half steps of fp64 of the turns each, at frequencies
    of at most one radian."""
    return float(positions.abs().max()) * 2.0 ** -50


def check_rope(b, s, hq, hk, d, rot, inter, dtype, positions=None, position0=0, scale=1.0, grad=False):
    packed, q, k = case(b, s, hq, hk, d, dtype)
    dev = packed.to(cuda())
    qd, kd = dev[:, :, :hq], dev[:, :, hq:hq + hk]
    freq = dr.rope_frequencies(rot)
    pos = positions if positions is not None else (position0 + torch.arange(s)).expand(b, s)
    fn = dr.rope_bwd if grad else dr.rope_fwd
    got = fn(qd, kd, freq.to(cuda()), None if positions is None else positions.to(cuda()),
             position0=position0, interleaved=inter, scale=scale)
    for x, y, name in ((q, got[0], "q"), (k, got[1], "k")):
        want = tr.rotate64(x.double(), angles_of(pos, freq), inter, scale, -1 if grad else 1)
        err = tr.rope_error(tr.partner_sum(x.double(), rot // 2, inter), scale, turn_bound(pos))
        err[..., rot:] = 0.0
        tr.assert_close(y, want, err, name)
        tr.assert_same_bits(y[..., rot:], x[..., rot:].contiguous(), f"{name}: columns that pass")


SHAPES = [  # batch, seq, q heads, k heads, head dim, rotary dim
    (1, 1, 1, 1, 2, 2), (1, 1, 32, 8, 128, 128), (8, 1, 32, 8, 128, 64), (2, 17, 4, 2, 64, 64), (1, 33, 3, 1, 96, 96),
    (3, 5, 7, 7, 80, 20), (1, 9, 2, 1, 48, 12), (2, 3, 5, 1, 256, 256), (1, 4, 2, 2, 512, 512), (1, 4, 2, 2, 496, 8),
    (1, 7, 1, 1, 33, 6), (1, 700, 6, 2, 32, 32), (2, 450, 8, 8, 192, 64), (1, 3, 200, 100, 16, 16), (5, 3, 2, 2, 8, 4),
]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("shape", SHAPES)
def test_rope(shape, inter, dtype):
    b, s = shape[:2]
    check_rope(*shape, inter, dtype)
    check_rope(*shape, inter, dtype, position0=100000, scale=1.25)
    pos = torch.randint(-5000, 5000, (b, s), generator=torch.Generator().manual_seed(4))
    check_rope(*shape, inter, dtype, positions=pos, grad=True, scale=0.75)


# many tokens of few heads: (batch, seq, q heads, k heads, head dim, rotary dim)
MANY = [(1, 9731, 2, 2, 128, 32), (3, 3301, 4, 1, 128, 128), (1, 19467, 7, 1, 32, 32), (2, 4999, 1, 3, 80, 80),
        (1, 5003, 3, 1, 256, 128), (7, 2800, 1, 1, 64, 64), (1, 20001, 1, 1, 24, 6)]


# tokens shared between warps unevenly, and several tokens a warp
SHARED = [(3, 499, 32, 8, 128, 128), (1, 1499, 32, 8, 64, 32), (2, 2903, 9, 5, 96, 96), (1, 20011, 30, 30, 8, 8),
          (1, 5003, 17, 4, 40, 10)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("shape", MANY + SHARED)
def test_rope_many_tokens(shape, inter, dtype):
    check_rope(*shape, inter, dtype, position0=3)
    b, s = shape[:2]
    pos = torch.randint(0, 5000, (b, s), generator=torch.Generator().manual_seed(4))
    check_rope(*shape, inter, dtype, positions=pos, grad=True, scale=0.75)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("shape", MANY + SHARED)
def test_norm_rope_many_tokens(shape, inter, dtype):
    check_norm_rope(shape, inter, dtype)


def test_far_positions():
    """Positions up to 2^40 and of either sign: the angle modulo one turn in
    exact rational arithmetic."""
    freq = dr.rope_frequencies(64, 10000.0)
    pos = torch.tensor([[0, 1, -1, 2 ** 20 + 1, 2 ** 31 - 1, -(2 ** 33) + 5, 2 ** 40 + 12345]])
    q = torch.zeros(1, pos.shape[1], 1, 64)
    q[..., :32] = 1.0  # (1, 0) turns to (cos, sin)
    got, none = dr.rope_fwd(q.to(cuda()), None, freq.to(cuda()), pos.to(cuda()))
    assert none is None
    for i, p in enumerate(pos[0].tolist()):
        turns = [float((Fraction(f) * p * INV_TAU) % 1) for f in freq.tolist()]
        ang = torch.tensor(turns, dtype=torch.float64) * (2 * np.pi)
        want = torch.cat([torch.cos(ang), torch.sin(ang)])
        # the kernel's fraction of a turn: two roundings of fp64 and one of 2^-64, times the position
        err = tr.rope_error(torch.ones(64, dtype=torch.float64), 1.0, 2 * np.pi * abs(p) * 0.16 * 2.0 ** -52)
        tr.assert_close(got[0, i, 0], want, err, f"position {p}")


@pytest.mark.parametrize("base", [100.0, 1e4, 1e9])
def test_angles_within_their_stated_bound(base):
    """|position| 2^-53 and 2^-32 turns, then fp32's rounding: near zero, for
    pairs that turn by less than fp32 holds of a turn, and far out.  The
    cosine and sine add an ulp and two roundings (4 half steps) of their own
    size."""
    freq = dr.rope_frequencies(128, base)
    pos = torch.tensor([[0, 1, -1, 2, 5, 37, -1000, 4095, 100003, 2 ** 24 + 1, -(2 ** 31) + 7]])
    q = torch.zeros(1, pos.shape[1], 1, 128)
    q[..., :64] = 1.0
    got = dr.rope_fwd(q.to(cuda()), None, freq.to(cuda()), pos.to(cuda()))[0][0, :, 0].double().cpu()
    for i, p in enumerate(pos[0].tolist()):
        turns = [(Fraction(f) * p * INV_TAU) % 1 for f in freq.tolist()]
        turns = torch.tensor([float(t - 1 if 2 * t >= 1 else t) for t in turns], dtype=torch.float64)
        ang = turns * (2 * np.pi)
        off = 2 * np.pi * (abs(p) * 2.0 ** -53 + 2.0 ** -32) + ang.abs() * 2.0 ** -24
        for name, value, j in (("cos", torch.cos(ang), 0), ("sin", torch.sin(ang), 64)):
            d = (got[i, j:j + 64] - value).abs()
            assert bool((d <= off + 4 * tr.EPS32 * value.abs()).all()), (name, p, float(d.max()))


def test_layouts_in_place_and_neighbours():
    """Packed, expanded, transposed and element-aligned tensors; what is not
    part of q and k stays as it was."""
    freq = dr.rope_frequencies(64).to(cuda())
    for dtype, inter, d in itertools.product(DTYPES, (False, True), (64, 100)):
        packed, q, k = case(2, 9, 4, 2, d, dtype)
        dev = packed.to(cuda())
        want = dr.rope_fwd(q.to(cuda()), k.to(cuda()), freq, position0=3, interleaved=inter)
        got = dr.rope_fwd(dev[:, :, :4], dev[:, :, 4:6], freq, position0=3, interleaved=inter, q_out=dev[:, :, :4],
                          k_out=dev[:, :, 4:6])
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        tr.assert_same_bits(dev[:, :, 6:], packed[:, :, 6:], "v")
        # [batch, heads, seq, dim] memory, one element past alignment
        room = torch.zeros(2 * 4 * 9 * d + 1, dtype=dtype, device=cuda())
        qt = room[1:].view(2, 4, 9, d).transpose(1, 2)
        qt.copy_(q)
        back = dr.rope_fwd(qt, None, freq, position0=3, interleaved=inter, q_out=qt)[0]
        assert torch.equal(back, want[0])
        # an expanded input
        one = q[:1, :, :1].to(cuda()).expand(2, 9, 4, d)
        assert torch.equal(dr.rope_fwd(one, None, freq, interleaved=inter)[0],
                           dr.rope_fwd(one.contiguous(), None, freq, interleaved=inter)[0])
        with pytest.raises(dr.DraddError):
            dr.rope_fwd(q.to(cuda()), None, freq, q_out=one)
        with pytest.raises(dr.DraddError):
            dr.rope_fwd(dev[:, :, :4], dev[:, :, 4:6], freq, q_out=dev[:, :, 1:5])


def test_overlapping_inputs_and_pinned_memory():
    """Inputs whose rows overlap by all but one element, whatever that does to
    their alignment, and buffers the device reaches over the host link."""
    freq = dr.rope_frequencies(64).to(cuda())
    w = normal(64, torch.bfloat16, 2, 0.1, 1.0).to(cuda())
    for dtype, strides in itertools.product(DTYPES, ((0, 1, 64, 1), (64, 64, 1, 1), (1, 8, 64, 1), (3, 0, 2, 1))):
        room = normal((4096,), dtype, 5).to(cuda())
        q = room.as_strided((2, 9, 4, 64), strides)
        assert torch.equal(dr.rope_fwd(q, None, freq)[0], dr.rope_fwd(q.contiguous(), None, freq)[0])
        a = dr.qk_rmsnorm_rope_fwd(q, None, w.to(dtype), None, freq)[0]
        assert torch.equal(a, dr.qk_rmsnorm_rope_fwd(q.contiguous(), None, w.to(dtype), None, freq)[0])
    L = dr.lib()
    q = normal((2, 9, 4, 64), torch.bfloat16, 6)
    want = dr.rope_fwd(q.to(cuda()), None, freq, position0=7)[0]
    host, out = q.pin_memory(), torch.empty_like(q).pin_memory()
    heads = [tr.CHeads(t.data_ptr(), 9 * 256, 256, 64) for t in (out, host)]
    r = tr.CRope(2, 9, 4, 0, 64, 64, 0, freq.data_ptr(), None, 7, 1.0)
    assert tr.c_entry(L, "rope_fwd")(ctypes.byref(heads[0]), None, ctypes.byref(heads[1]), None, ctypes.byref(r), 0,
                      torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()
    assert torch.equal(out, want.cpu())


def test_columns_that_pass_hold_anything():
    q = torch.full((1, 5, 2, 64), float("nan"))
    q[..., :24] = 1.0
    q[..., 30:] = float("inf")
    for dtype, inter in itertools.product(DTYPES, (False, True)):
        freq = dr.rope_frequencies(24).to(cuda())
        got = dr.rope_fwd(q.to(dtype).to(cuda()), None, freq, position0=2, interleaved=inter)[0].cpu().float()
        assert bool(torch.isfinite(got[..., :24]).all())
        assert bool(torch.isnan(got[..., 24:30]).all()) and bool((got[..., 30:] == float("inf")).all())


@pytest.mark.parametrize("dim,rot", [(64, 24), (64, 32), (64, 4), (100, 36), (33, 6), (128, 64)])
def test_columns_not_written_in_place(dim, rot):
    """In place, bits that a copy through fp32 would not keep (a signalling
    NaN) stay: in the halves layout past rot, interleaved past the next
    multiple of 16; between, a NaN stays a NaN."""
    for inter in (False, True):
        x = normal((2, 37, 3, dim), torch.bfloat16, 1)
        x.view(torch.int16)[..., rot:] = 0x7F81
        on = x.to(cuda())
        freq = dr.rope_frequencies(rot).to(cuda())
        want = dr.rope_fwd(on, None, freq, position0=4, interleaved=inter)[0]
        got = dr.rope_fwd(on, None, freq, position0=4, interleaved=inter, q_out=on)[0]
        assert torch.equal(got[..., :rot], want[..., :rot]) and bool(torch.isnan(got[..., rot:]).all())
        kept = -(-rot // 16) * 16 if inter else rot
        assert bool((got.view(torch.int16)[..., kept:] == 0x7F81).all())


def test_refusals_and_empty():
    q = torch.zeros(2, 3, 4, 64, device=cuda(), dtype=torch.bfloat16)
    f = dr.rope_frequencies(64).to(cuda())
    w = torch.ones(64, device=cuda(), dtype=torch.bfloat16)
    for bad in (lambda: dr.rope_fwd(q, q[:1], f), lambda: dr.rope_fwd(q[0], None, f),
                lambda: dr.rope_fwd(q, q[..., :32], f), lambda: dr.rope_fwd(q.transpose(2, 3), None, f),
                lambda: dr.rope_fwd(q, None, f, torch.zeros(5, dtype=torch.int64, device=cuda())),
                lambda: dr.rope_fwd(q, None, f, torch.zeros(2, 3, dtype=torch.int64, device=cuda()), position0=1),
                lambda: dr.rope_fwd(q, None, dr.rope_frequencies(64)),
                lambda: dr.rope_fwd(q, None, f, q_out=q[:, :2])):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: dr.rope_fwd(q, None, f.float()), lambda: dr.rope_fwd(q, q.float(), f),
                lambda: dr.rope_fwd(q, None, f, torch.zeros(2, 3, dtype=torch.int32, device=cuda())),
                lambda: dr.qk_rmsnorm_rope_fwd(q, None, w.float(), None, f)):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: dr.rope_fwd(q, None, dr.rope_frequencies(66).to(cuda())),
                lambda: dr.rope_fwd(q, None, f, scale=float("nan")),
                lambda: dr.qk_rmsnorm_rope_fwd(q, None, w, None, f, -1.0)):
        with pytest.raises(dr.DraddError):
            bad()
    e = q[:0]
    assert dr.rope_fwd(e, e, f)[1].shape == (0, 3, 4, 64)
    got = dr.qk_rmsnorm_rope_bwd(e, e, e, e, w, w, f)
    assert got[0].shape == (0, 3, 4, 64) and bool((got[2] == 0).all()) and bool((got[3] == 0).all())


# --------------------------------------------------------- behind the norm
def norm_bounds(x, w, eps):
    """z = x inv w in fp64 and how far the kernel's may be: the sum of at
    most 512 squares (10 roundings, half of them in inv), inv's own 4, two
    products."""
    inv = 1 / torch.sqrt(x.square().mean(-1, keepdim=True) + float(np.float32(eps)))
    z = x * inv * w
    return z, 12 * tr.EPS32


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("shape", SHAPES)
def test_norm_rope(shape, inter, dtype):
    check_norm_rope(shape, inter, dtype)


def check_norm_rope(shape, inter, dtype):
    b, s, hq, hk, d, rot = shape
    packed, q, k = case(b, s, hq, hk, d, dtype)
    dev = packed.to(cuda())
    qw, kw = normal(d, dtype, 1, 0.1, 1.0), normal(d, dtype, 2, 0.1, 1.0)
    freq = dr.rope_frequencies(rot)
    pos = torch.randint(0, 9000, (b, s), generator=torch.Generator().manual_seed(4))
    on = dict(positions=pos.to(cuda()), interleaved=inter, scale=1.125)
    args = (qw.to(cuda()), kw.to(cuda()), freq.to(cuda()), 1e-6, 1e-3)
    got = dr.qk_rmsnorm_rope_fwd(dev[:, :, :hq], dev[:, :, hq:hq + hk], *args, **on)
    dy = [normal(x.shape, dtype, 9 + i) for i, x in enumerate((q, k))]
    grads = dr.qk_rmsnorm_rope_bwd(dy[0].to(cuda()), dy[1].to(cuda()), dev[:, :, :hq], dev[:, :, hq:hq + hk], *args,
                                   **on)
    ang = angles_of(pos, freq)
    for i, (x, w, eps) in enumerate(((q, qw, 1e-6), (k, kw, 1e-3))):
        x, w, g = x.double(), w.double(), dy[i].double()
        z, rel = norm_bounds(x, w, eps)
        want = tr.rotate64(z, ang, inter, 1.125)
        pair = tr.partner_sum(z, rot // 2, inter)
        err = tr.rope_error(pair, 1.125, turn_bound(pos)) + 1.125 * rel * pair
        err[..., rot:] = rel * z.abs()[..., rot:]
        tr.assert_close(got[i], want, err, f"out {i}")
        # gradients: g turned back, then the norm's
        t = tr.rotate64(g, ang, inter, 1.125, -1)
        t_err = tr.rope_error(tr.partner_sum(g, rot // 2, inter), 1.125, turn_bound(pos))
        t_err[..., rot:] = 0.0
        e, e_err, ew, ew_err = tr.rmsnorm_bwd64(t, None, x, w, eps)
        inv = 1 / torch.sqrt(x.square().mean(-1, keepdim=True) + float(np.float32(eps)))
        xh = (x * inv).abs()
        wt = t_err * w.abs()
        e_err = e_err + 1.01 * inv * (wt + xh * (wt * xh).mean(-1, keepdim=True))
        tr.assert_close(grads[i], e, e_err, f"grad {i}")
        n = b * s * x.shape[2]
        ew_err = ew_err + 1.01 * (t_err * xh).reshape(-1, d).sum(0) + min(n, 400) * tr.EPS32 * (
            t.abs() * xh).reshape(-1, d).sum(0)
        tr.assert_close(grads[2 + i], ew, ew_err, f"weight grad {i}")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("inter", [False, True])
def test_norm_rope_forms(inter, dtype):
    """In place, q alone, without weight gradients, a caller's workspace, one
    weight's gradient, other streams and a captured graph: the same bits."""
    packed, q, k = case(2, 300, 8, 2, 128, dtype)
    dev = packed.to(cuda())
    q, k = q.to(cuda()), k.to(cuda())
    w = [normal(128, dtype, i, 0.1, 1.0).to(cuda()) for i in (1, 2)]
    f = dr.rope_frequencies(96).to(cuda())
    on = dict(position0=50, interleaved=inter)
    want = dr.qk_rmsnorm_rope_fwd(q, k, *w, f, **on)
    got = dr.qk_rmsnorm_rope_fwd(dev[:, :, :8], dev[:, :, 8:10], *w, f, q_out=dev[:, :, :8], k_out=dev[:, :, 8:10],
                                 **on)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    alone = dr.qk_rmsnorm_rope_fwd(q, None, w[0], None, f, **on)
    assert torch.equal(alone[0], want[0]) and alone[1] is None
    # the norm alone is the framework's own, and the turn alone is rope_fwd's: both compose to within the rounding
    # between them, which test_norm_rope bounds
    dy = [normal(t.shape, dtype, 5).to(cuda()) for t in (q, k)]
    want = dr.qk_rmsnorm_rope_bwd(*dy, q, k, *w, f, **on)
    got = dr.qk_rmsnorm_rope_bwd(*dy, q, k, *w, f, weight_grad=False, **on)
    assert got[2] is None and got[3] is None and all(torch.equal(a, b) for a, b in zip(got[:2], want))
    for target in ("x", "dy"):
        x2, y2 = [q.clone(), k.clone()], [t.clone() for t in dy]
        dst = x2 if target == "x" else y2
        got = dr.qk_rmsnorm_rope_bwd(*y2, *x2, *w, f, dq=dst[0], dk=dst[1], **on)
        assert got[0] is dst[0] and all(torch.equal(a, b) for a, b in zip(got, want))
    ws = torch.full((1 << 20,), 255, dtype=torch.uint8, device=cuda())
    got = dr.qk_rmsnorm_rope_bwd(*dy, q, k, *w, f, workspace=ws, **on)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    with pytest.raises(dr.DraddError):
        dr.qk_rmsnorm_rope_bwd(*dy, q, k, *w, f, workspace=ws[:512], **on)
    only = dr.qk_rmsnorm_rope_bwd(dy[0], None, q, None, w[0], None, f, **on)
    assert torch.equal(only[0], want[0]) and only[1] is None and only[3] is None
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = dr.qk_rmsnorm_rope_bwd(*dy, q, k, *w, f, stream=s, **on)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    pos = torch.zeros(2, 300, dtype=torch.int64, device=cuda())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        held = dr.qk_rmsnorm_rope_bwd(*dy, q, k, *w, f, positions=pos, interleaved=inter)
        turned = dr.rope_fwd(q, k, f, pos, interleaved=inter)
    pos.copy_(50 + torch.arange(300, device=cuda()))
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(held, want))
    assert all(torch.equal(a, b) for a, b in zip(turned, dr.rope_fwd(q, k, f, position0=50, interleaved=inter)))


def test_offsets_past_32_bits():
    """A cache of which the addressed rows lie past 2^31 elements."""
    d, s = 64, 3
    room = torch.zeros(2 ** 31 + 2 * s * d, dtype=torch.bfloat16, device=cuda())
    cache = room.as_strided((2, s, 1, d), (2 ** 31 + s * d, d, d, 1))
    x = normal((2, s, 1, d), torch.bfloat16, 3).to(cuda())
    cache.copy_(x)
    f = dr.rope_frequencies(d).to(cuda())
    w = torch.ones(d, dtype=torch.bfloat16, device=cuda())
    want = dr.rope_fwd(x, None, f, position0=9)[0]
    assert torch.equal(dr.rope_fwd(cache, None, f, position0=9)[0], want)
    assert torch.equal(dr.rope_fwd(cache, None, f, position0=9, q_out=cache)[0], want)
    assert int(torch.count_nonzero(room)) <= 2 * s * d
    z = dr.qk_rmsnorm_rope_fwd(want, None, w, None, f)[0]
    assert torch.equal(dr.qk_rmsnorm_rope_fwd(cache, None, w, None, f, q_out=cache)[0], z)


def test_a_block_of_them_together():
    """The operators as a pre-norm block's training step uses them: dropout +
    residual add + norm, a projection, q/k norm and rotation, and back, fp32,
    against autograd in fp64 through the same masks."""
    b, s, hq, hk, d, p = 2, 40, 4, 2, 64, 0.2
    hidden = 256
    x, r = normal((b, s, hidden), torch.float32, 1), normal((b, s, hidden), torch.float32, 2)
    w = normal(hidden, torch.float32, 3, 0.1, 1.0)
    proj = normal((hidden, (hq + hk) * d), torch.float32, 4, hidden ** -0.5)
    qw, kw = normal(d, torch.float32, 5, 0.1, 1.0), normal(d, torch.float32, 6, 0.1, 1.0)
    cq, ck, cr = (normal(sh, torch.float32, 7 + i) for i, sh in enumerate(
        ((b, s, hq, d), (b, s, hk, d), (b, s, hidden))))
    freq = dr.rope_frequencies(d)

    X, R, W, P, QW, KW, CQ, CK, CR, FR = (t.to(cuda()) for t in (x, r, w, proj, qw, kw, cq, ck, cr, freq))
    out, h = dr.dropout_add_rmsnorm_fwd(X, R, W, p, EPS, seed=11, offset=2)
    packed = (out.double() @ P.double()).float().view(b, s, hq + hk, d)
    q, k = packed[:, :, :hq], packed[:, :, hq:]
    qo, ko = dr.qk_rmsnorm_rope_fwd(q, k, QW, KW, FR)
    dpacked = torch.empty_like(packed)
    _, _, dqw, dkw = dr.qk_rmsnorm_rope_bwd(CQ, CK, q, k, QW, KW, FR, dq=dpacked[:, :, :hq], dk=dpacked[:, :, hq:])
    dout = (dpacked.view(b, s, -1).double() @ P.double().t()).float()
    dx, dres, dw = dr.dropout_add_rmsnorm_bwd(dout, CR, h, W, p, EPS, seed=11, offset=2)
    got = [qo, ko, h, dx, dres, dw, dqw, dkw]

    leaves = [t.double().requires_grad_() for t in (x, r, w, qw, kw)]
    x6, r6, w6, qw6, kw6 = leaves
    keep = tr.keep_mask(b * s, hidden, p, 11, 2).view(b, s, hidden).double()
    h6 = r6 + x6 * keep * (65536 / (65536 - tr.threshold(p)))

    def norm(t, g):
        return t * (t.square().mean(-1, keepdim=True) + EPS).rsqrt() * g

    y6 = (norm(h6, w6) @ proj.double()).view(b, s, hq + hk, d)
    ang = torch.arange(s).double()[:, None] * freq
    ang = ang.expand(b, s, -1)
    q6 = tr.rotate64(norm(y6[:, :, :hq], qw6), ang, False, 1.0)
    k6 = tr.rotate64(norm(y6[:, :, hq:], kw6), ang, False, 1.0)
    grads = torch.autograd.grad([q6, k6, h6 * 1.0], leaves, [cq.double(), ck.double(), cr.double()])
    want = [q6, k6, h6, *grads]
    # Each stage keeps a relative error of some tens of roundings in the
    # 2-norm (the bounds of the single operators above); six stages and the
    # two fp32 roundings of the projections stay below 2^-16.
    for i, (a, e) in enumerate(zip(got, want)):
        e = e.detach()
        assert float((a.double().cpu() - e).norm() / e.norm()) < 2.0 ** -16, i
