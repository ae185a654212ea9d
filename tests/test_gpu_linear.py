"""Matrix products with bias, activation and residual, cross entropy and
distillation without kept logits, and their gradients, against fp64.

Every element is held to the bound of linear_refs; where sums are long, the
result as a whole also to half a step of its type: one rounding has a root
mean square below 0.4 of that, and the gradients have two."""
import math
import threading

import pytest
import torch

import deterministic_residual_add_gb300 as dr
import linear_refs as lr
from linear_refs import HALF_STEP, assert_close, norm_off

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16


@pytest.fixture(autouse=True)
def status_clear():
    yield
    assert dr.device_status(clear=True) == 0


class Make:
    def __init__(self, seed, dtype):
        self.g = torch.Generator(device="cuda").manual_seed(seed)
        self.dtype = dtype

    def __call__(self, *shape, std=1.0, dtype=None):
        return (torch.randn(shape, generator=self.g, device="cuda") * std).to(dtype or self.dtype)

    def words(self, high, *shape):
        return torch.randint(0, high, shape, generator=self.g, device="cuda")

    def top(self, rows, vocab, top):
        """Different words in no order."""
        return torch.rand(rows, vocab, generator=self.g, device="cuda").topk(top, dim=1).indices


def linear_case(rows, inner, cols, dtype, bias=True, residual=True, seed=0):
    n = Make(seed + rows + inner, dtype)
    return (n(rows, inner), n(cols, inner, std=inner ** -0.5), n(cols, std=0.5) if bias else None,
            n(rows, cols, std=2.0) if residual else None, n(rows, cols))


def check_linear(x, w, b, r, dout, act):
    got = dr.linear_act_add_fwd(x, w, b, r, activation=act)
    want, err = lr.linear(x, w, b, r, act)
    assert_close(got, want, err, "out")
    grads = dr.linear_act_add_bwd(dout, x, w, b, activation=act)
    for name, g, (want, err) in zip(("dx", "dweight", "dbias"), grads, lr.linear_grads(dout, x, w, b, act)):
        if g is None:
            assert name == "dbias" and b is None
            continue
        assert_close(g, want, err, name)
        if act != "relu" and want.numel() > 1000 and min(x.shape[0], w.shape[0]) > 16:
            assert norm_off(g, want) < HALF_STEP[x.dtype], name


# one token to several tiles; odd numbers of rows, inner dimensions and
# columns around tiles of 64, 128 and 256; one CTA a tile and two; split sums
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("rows,inner,cols,act", [
    (1, 8, 8, "none"), (1, 4096, 1024, "silu"), (2, 72, 24, "gelu"), (8, 264, 1000, "gelu_tanh"),
    (9, 1000, 264, "relu"), (16, 520, 136, "none"), (17, 64, 256, "silu"), (64, 4096, 264, "gelu"),
    (127, 72, 520, "relu"), (128, 128, 128, "none"), (129, 136, 248, "gelu_tanh"), (255, 64, 8, "silu"),
    (5, 8192, 4104, "none"), (12, 4096, 4104, "silu"), (40, 2048, 20008, "silu"), (257, 2048, 264, "none"),
    (300, 520, 1032, "gelu"), (1000, 256, 512, "silu"), (1536, 1024, 776, "gelu_tanh")])
def test_linear(rows, inner, cols, act, dtype):
    check_linear(*linear_case(rows, inner, cols, dtype), act)


@pytest.mark.parametrize("bias,residual", [(False, False), (True, False), (False, True)])
@pytest.mark.parametrize("rows", [3, 40, 200])
def test_linear_without_bias_or_residual(rows, bias, residual):
    check_linear(*linear_case(rows, 136, 264, BF16, bias, residual), "silu")


@pytest.mark.parametrize("act", lr.ACTS)
@pytest.mark.parametrize("rows", [4, 40, 300])
def test_activations(rows, act):
    """Values far to both sides, zeros, and the largest ones: bias carries them past the product."""
    n = Make(3, F16)
    cols = 520
    b = torch.linspace(-30, 30, cols, device="cuda").to(F16)
    b[:6] = torch.tensor([0.0, -0.0, 60000.0, -60000.0, 1e-7, -1e-7], device="cuda")
    x, w = n(rows, 64, std=0.01), n(cols, 64, std=0.1)
    x[0] = 0  # z is the bias
    check_linear(x, w, b, None, n(rows, cols), act)


def test_activation_gradient_against_differences():
    n = Make(5, F16)
    x, w, b, dout = n(3, 16), n(24, 16, std=0.25), n(24), n(3, 24)
    for act in ("gelu", "gelu_tanh", "silu"):
        f = lambda x_, w_, b_: (lr.act64(x_.double() @ w_.double().t() + b_.double(), act) * dout.double()).sum()
        dx, dw, db = dr.linear_act_add_bwd(dout, x, w, b, activation=act)
        for got, t, args in ((dx, x, 0), (dw, w, 1), (db, b, 2)):
            for at in ((0,) * t.dim(), tuple(s - 1 for s in t.shape)):
                lo, hi, h = [x.double(), w.double(), b.double()], [x.double(), w.double(), b.double()], 1e-5
                lo[args], hi[args] = lo[args].clone(), hi[args].clone()
                lo[args][at] -= h
                hi[args][at] += h
                want = float(f(*hi) - f(*lo)) / (2 * h)
                # two roundings of terms whose magnitudes add up to at most 24 * 2
                assert abs(float(got[at]) - want) < 2 * 2.0 ** -11 * 24


@pytest.mark.parametrize("rows", [5, 48, 140])
def test_linear_strides_and_neighbours(rows):
    """Slices of packed rows in and out, shapes of more dimensions; what lies beside the output stays."""
    n = Make(rows, BF16)
    inner, cols = 136, 264
    packed = n(rows, 3 * inner)
    x, w = packed[:, inner:2 * inner], n(cols, 2 * inner, std=0.1)[:, 8:8 + inner]
    r = n(rows, cols + 24)[:, 8:8 + cols]
    room = torch.full((rows + 2, cols + 48), float("nan"), dtype=BF16, device="cuda")
    out = room[1:-1, 8:8 + cols]
    got = dr.linear_act_add_fwd(x, w, None, r, activation="silu", out=out)
    assert got.data_ptr() == out.data_ptr()
    want, err = lr.linear(x, w, None, r, "silu")
    assert_close(out, want, err, "out")
    assert room[0].isnan().all() and room[-1].isnan().all()
    assert room[:, :8].isnan().all() and room[:, 8 + cols:].isnan().all()
    again = dr.linear_act_add_fwd(x.contiguous(), w.contiguous(), None, r.contiguous(), activation="silu")
    assert torch.equal(again, out)
    # in place of the residual, and with leading dimensions
    deep = dr.linear_act_add_fwd(x.contiguous().view(rows, 1, inner), w, None, activation="silu")
    assert deep.shape == (rows, 1, cols)
    assert torch.equal(deep.view(rows, cols), dr.linear_act_add_fwd(x, w, activation="silu"))
    inplace = r.clone()
    dr.linear_act_add_fwd(x, w, None, inplace, activation="silu", out=inplace)
    assert torch.equal(inplace, again)
    dout = n(rows, 2 * cols)[:, cols:]
    for act in ("none", "gelu"):
        for a, b in zip(dr.linear_act_add_bwd(dout, x, w, activation=act)[:2],
                        dr.linear_act_add_bwd(dout.contiguous(), x.contiguous(), w.contiguous(), activation=act)):
            assert torch.equal(a, b)


def test_linear_some_gradients():
    x, w, b, _, dout = linear_case(150, 136, 264, BF16)
    for act in ("none", "silu"):
        full = dr.linear_act_add_bwd(dout, x, w, b, activation=act)
        only_x = dr.linear_act_add_bwd(dout, x, w, b, activation=act, weight_grad=False)
        only_w = dr.linear_act_add_bwd(dout, x, w, b, activation=act, input_grad=False)
        assert only_x[1] is None and only_x[2] is None and only_w[0] is None
        # how the sums are split may differ where one product runs alone
        want = lr.linear_grads(dout, x, w, b, act)
        assert_close(only_x[0], *want[0], "dx")
        assert_close(only_w[1], *want[1], "dweight")
        assert torch.equal(only_w[2], full[2])
    room = [torch.full((s.numel() + 16,), float("nan"), dtype=BF16, device="cuda") for s in (x, w, b)]
    views = [m[8:-8].view(s.shape) for m, s in zip(room, (x, w, b))]
    dr.linear_act_add_bwd(dout, x, w, b, activation="silu", dx=views[0], dweight=views[1], dbias=views[2])
    for m, v, f in zip(room, views, full):
        assert torch.equal(v, f) and m[:8].isnan().all() and m[-8:].isnan().all()


def test_linear_no_rows():
    n = Make(1, BF16)
    x, w, b = n(0, 64), n(32, 64), n(32)
    assert dr.linear_act_add_fwd(x, w, b).shape == (0, 32)
    dw = torch.full((32, 64), float("nan"), dtype=BF16, device="cuda")
    dx, dw, db = dr.linear_act_add_bwd(n(0, 32), x, w, b, activation="silu", dweight=dw)
    assert dx.shape == (0, 64) and not dw.any() and not db.any()


def test_row_of_nan_stays_a_row():
    for rows in (6, 60, 400):
        x, w, b, r, _ = linear_case(rows, 136, 264, BF16)
        want = dr.linear_act_add_fwd(x, w, b, r, activation="gelu")
        x[1], x[3] = float("nan"), float("inf")
        got = dr.linear_act_add_fwd(x, w, b, r, activation="gelu")
        assert got[1].isnan().all() and not got[3].isfinite().any()
        keep = [i for i in range(rows) if i not in (1, 3)]
        assert torch.equal(got[keep], want[keep])


# ------------------------------------------------------------------- losses
def loss_case(rows, hidden, vocab, dtype, top=0, seed=0):
    n = Make(seed + rows + vocab, dtype)
    w = n(vocab, hidden, std=1.5 * hidden ** -0.5)
    words = n.words(vocab, rows)
    x = (n(rows, hidden, dtype=torch.float32) +
         w[words].float() * 4 * torch.rand(rows, 1, generator=n.g, device="cuda")).to(dtype)
    if not top:
        target = words.clone()
        target[::5] = -100
        return x, w, target
    return x, w, n.top(rows, vocab, top), n(rows, top, std=2.0, dtype=torch.float32)


def weights_for(rows, dtype, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    size = 8.0 if dtype == F16 else 1.0 / rows
    return (size * (0.5 + torch.rand(rows, generator=g, device="cuda")),
            0.01 * size * torch.randn(rows, generator=g, device="cuda"))


def check_grads(got, want, dtype, rows):
    for name, g, (exact, err) in zip(("dx", "dweight"), got, want):
        assert_close(g, exact, err, name)
        if rows > 16 and exact.numel() > 1000:
            assert norm_off(g, exact) < HALF_STEP[dtype], name


def check_ce(x, w, target, ignore_index=-100):
    loss, lse = dr.linear_cross_entropy_fwd(x, w, target, ignore_index=ignore_index)
    index, share = lr.ce_shares(target, ignore_index)
    want, err, want_lse, lse_err = lr.loss(x, w, index, share)
    assert_close(loss, want, err, "loss")
    assert_close(lse, want_lse, lse_err, "lse")
    assert not loss[target == ignore_index].any()
    dloss, dlse = weights_for(x.shape[0], x.dtype)
    got = dr.linear_cross_entropy_bwd(dloss, dlse, x, w, target, lse, ignore_index=ignore_index)
    check_grads(got, lr.loss_grads(dloss, dlse, x, w, index, share, lse), x.dtype, x.shape[0])
    return got


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("rows,hidden,vocab", [
    (1, 8, 1), (1, 64, 1001), (2, 136, 2), (33, 264, 127), (64, 4096, 255), (100, 512, 3001), (128, 64, 256),
    (20, 2056, 20001), (129, 72, 257), (257, 1024, 1000), (511, 256, 5001), (1024, 128, 8000),
    (1500, 64, 300)])
def test_cross_entropy(rows, hidden, vocab, dtype):
    check_ce(*loss_case(rows, hidden, vocab, dtype))


def test_cross_entropy_in_pieces():
    """Three pieces of the vocabulary, the last one smaller and odd."""
    rows, vocab = 4096, 70001
    x, w, target = loss_case(rows, 64, vocab, BF16)
    target[1], target[2], target[3], target[4] = 0, vocab - 1, 32768, 65535
    check_ce(x, w, target)


def test_long_sums_of_the_vocabulary():
    """Few rows over many words: dx is the sum of splits."""
    check_ce(*loss_case(40, 264, 60001, F16))


def test_ignored_and_masked_rows_count_for_nothing():
    """Whatever they hold: NaN and infinities in x, lse and dloss."""
    for rows, hidden, vocab in ((24, 72, 300), (300, 136, 1000)):
        x, w, target = loss_case(rows, hidden, vocab, BF16)
        target[:] = target.clamp(min=0)
        dloss, _ = weights_for(rows, BF16)
        bad = torch.arange(rows, device="cuda") % 3 == 1
        zero = torch.arange(rows, device="cuda") % 3 == 2
        target[bad] = -100
        dloss[zero] = 0
        lse = dr.linear_cross_entropy_fwd(x, w, target)[1]
        want = dr.linear_cross_entropy_bwd(dloss, None, x, w, target, lse)
        x2, lse2, dloss2 = x.clone(), lse.clone(), dloss.clone()
        x2[bad], x2[zero] = float("nan"), float("inf")
        lse2[bad], lse2[zero], dloss2[bad] = float("nan"), float("-inf"), float("nan")
        got = dr.linear_cross_entropy_bwd(dloss2, None, x2, w, target, lse2)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        assert not got[0][bad].any() and not got[0][zero].any()
        loss = dr.linear_cross_entropy_fwd(x2, w, target)[0]
        assert not loss[bad].any()


def test_every_row_ignored():
    x, w, target = loss_case(50, 64, 300, BF16)
    target[:] = -100
    loss, lse = dr.linear_cross_entropy_fwd(x, w, target)
    assert not loss.any() and lse.isfinite().all()
    dx, dw = dr.linear_cross_entropy_bwd(torch.ones(50, device="cuda"), None, x, w, target, lse)
    assert not dx.any() and not dw.any()
    # lse's own gradient goes on
    index, share = lr.ce_shares(target, -100)
    dlse = torch.rand(50, device="cuda")
    check_grads(dr.linear_cross_entropy_bwd(torch.ones(50, device="cuda"), dlse, x, w, target, lse),
                lr.loss_grads(torch.ones(50, device="cuda"), dlse, x, w, index, share, lse), BF16, 50)


def test_targets_that_are_no_words():
    x, w, target = loss_case(40, 64, 300, BF16)
    target[1], target[2], target[3], target[4] = 300, -1, 1 << 40, -(1 << 40)
    loss, lse = dr.linear_cross_entropy_fwd(x, w, target)
    assert loss[1:5].isnan().all() and loss[6:].isfinite().all() and lse.isfinite().all()
    dx, _ = dr.linear_cross_entropy_bwd(torch.ones(40, device="cuda"), None, x, w, target, lse)
    assert dx[1:5].isnan().all() and dx[6:].isfinite().all()
    # a word may be the one to ignore
    target[1:5] = 7
    check_ce(x, w, target.clamp(min=0), ignore_index=7)


def test_row_of_nan_logits_stays_a_row():
    for rows in (30, 200):
        x, w, target = loss_case(rows, 64, 700, BF16)
        want = dr.linear_cross_entropy_fwd(x, w, target)
        x[1], x[3] = float("nan"), float("inf")
        got = dr.linear_cross_entropy_fwd(x, w, target)
        keep = [i for i in range(rows) if i not in (1, 3)]
        for a, b in zip(got, want):
            assert a[1].isnan() and not a[3].isfinite()
            assert torch.equal(a[keep], b[keep])


def test_far_apart_logits():
    """Logits of +-3000: no exponential overflows, and the softmax is one word."""
    n = Make(2, BF16)
    x, w = n(20, 64, std=20.0), n(400, 64, std=20.0)
    target = n.words(400, 20)
    loss, lse = dr.linear_cross_entropy_fwd(x, w, target)
    index, share = lr.ce_shares(target, -100)
    want, err, want_lse, lse_err = lr.loss(x, w, index, share)
    assert_close(loss, want, err, "loss")
    assert_close(lse, want_lse, lse_err, "lse")


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_one_value_for_all_rows(dtype):
    """The gradient of a mean: an expanded number, or one without dimensions."""
    x, w, target = loss_case(60, 136, 900, dtype)
    lse = dr.linear_cross_entropy_fwd(x, w, target)[1]
    v = 0.25
    full = torch.full((60,), v, device="cuda")
    want = dr.linear_cross_entropy_bwd(full, full, x, w, target, lse)
    one = torch.tensor(v, device="cuda")
    for d in (one, one.expand(60)):
        got = dr.linear_cross_entropy_bwd(d, d, x, w, target, lse)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    deep = dr.linear_cross_entropy_bwd(one.expand(5, 12), None, x.view(5, 12, 136), w, target.view(5, 12),
                                       lse.view(5, 12))
    flat = dr.linear_cross_entropy_bwd(full, None, x, w, target, lse)
    assert torch.equal(deep[0].view(60, 136), flat[0]) and torch.equal(deep[1], flat[1])
    none = dr.linear_cross_entropy_bwd(full, torch.zeros(60, device="cuda"), x, w, target, lse)
    assert torch.equal(none[0], flat[0]) and torch.equal(none[1], flat[1])


def test_small_losses_of_many_tokens_in_fp16():
    """Factors of 1e-7: dz would vanish among fp16's smallest numbers."""
    rows, hidden, vocab = 200, 64, 500
    x, w, target = loss_case(rows, hidden, vocab, F16)
    x, w = (x.float() * 60).to(F16), (w.float() / 60).to(F16)
    lse = dr.linear_cross_entropy_fwd(x, w, target)[1]
    dloss = torch.full((rows,), 1e-5, device="cuda")
    index, share = lr.ce_shares(target, -100)
    want = lr.loss_grads(dloss, None, x, w, index, share, lse)
    got = dr.linear_cross_entropy_bwd(dloss, None, x, w, target, lse)
    check_grads(got[1:], want[1:], F16, rows)
    assert_close(got[0], *want[0], "dx")


def test_loss_some_gradients_and_given_outputs():
    for rows, vocab in ((40, 1000), (300, 700)):
        x, w, target = loss_case(rows, 136, vocab, BF16)
        loss = torch.full((rows + 8,), float("nan"), device="cuda")
        lse = loss.clone()
        dr.linear_cross_entropy_fwd(x, w, target, loss=loss[4:-4], lse=lse[4:-4])
        for t in (loss, lse):
            assert t[:4].isnan().all() and t[-4:].isnan().all() and t[4:-4].isfinite().all()
        lse = lse[4:-4].clone()
        dloss, dlse = weights_for(rows, BF16)
        full = dr.linear_cross_entropy_bwd(dloss, dlse, x, w, target, lse)
        dx, none = dr.linear_cross_entropy_bwd(dloss, dlse, x, w, target, lse, weight_grad=False)
        assert none is None and torch.equal(dx, full[0])
        none, dw = dr.linear_cross_entropy_bwd(dloss, dlse, x, w, target, lse, input_grad=False)
        assert none is None and torch.equal(dw, full[1])
        room = [torch.full((t.numel() + 16,), float("nan"), dtype=BF16, device="cuda") for t in (x, w)]
        views = [m[8:-8].view(t.shape) for m, t in zip(room, (x, w))]
        dr.linear_cross_entropy_bwd(dloss, dlse, x, w, target, lse, dx=views[0], dweight=views[1])
        for m, v, f in zip(room, views, full):
            assert torch.equal(v, f) and m[:8].isnan().all() and m[-8:].isnan().all()


def test_loss_strides():
    n = Make(9, BF16)
    rows, hidden, vocab = 150, 136, 900
    x = n(rows, 2 * hidden)[:, hidden:]
    w = n(vocab, hidden + 24, std=0.1)[:, 16:16 + hidden]
    target = n.words(vocab, rows)
    a = dr.linear_cross_entropy_fwd(x, w, target)
    b = dr.linear_cross_entropy_fwd(x.contiguous(), w.contiguous(), target)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    dloss = torch.rand(rows, device="cuda")
    a, b = (dr.linear_cross_entropy_bwd(dloss, None, x_, w_, target, a[1])
            for x_, w_ in ((x, w), (x.contiguous(), w.contiguous())))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_loss_no_rows():
    w = torch.ones(30, 64, dtype=BF16, device="cuda")
    x, t = w[:0], torch.zeros(0, dtype=torch.int64, device="cuda")
    loss, lse = dr.linear_cross_entropy_fwd(x, w, t)
    assert loss.shape == lse.shape == (0,)
    dw = torch.full_like(w, float("nan"))
    dx, dw = dr.linear_cross_entropy_bwd(loss, None, x, w, t, lse, dweight=dw)
    assert dx.shape == (0, 64) and not dw.any()
    i, l = torch.zeros(0, 3, dtype=torch.int64, device="cuda"), torch.zeros(0, 3, device="cuda")
    assert dr.linear_distill_fwd(x, w, i, l)[0].shape == (0,)
    assert not dr.linear_distill_bwd(loss, None, x, w, i, l, lse)[1].any()


def test_words_behind_32_bits():
    """A weight of more than 2^31 elements: the last rows are reached."""
    hidden, vocab, rows = 4096, 600000, 5
    g = torch.Generator(device="cuda").manual_seed(4)
    w = torch.zeros(vocab, hidden, dtype=BF16, device="cuda")
    last = vocab - 1000
    w[last:] = (torch.randn(1000, hidden, generator=g, device="cuda") / 32).to(BF16)
    x = torch.randn(rows, hidden, generator=g, device="cuda").to(BF16)
    target = torch.tensor([0, last, vocab - 1, vocab - 500, -100], device="cuda")
    loss, lse = dr.linear_cross_entropy_fwd(x, w, target)
    z = x.double() @ w[last:].double().t()
    want = torch.logsumexp(torch.cat([z, torch.full((rows, 1), math.log(last), device="cuda").double()], 1), 1)
    bound = lr.sum_err(hidden) * float((x.double().abs() @ w[last:].double().abs().t()).max()) + 6000 * 2.0 ** -24
    assert_close(lse, want, bound, "lse")
    at = torch.tensor([0.0, float(z[1, 0]), float(z[2, 999]), float(z[3, 500])], device="cuda").double()
    assert_close(loss[:4], (want[:4] - at), 2 * bound, "loss")
    dloss = torch.ones(rows, device="cuda")
    dx, dw = dr.linear_cross_entropy_bwd(dloss, None, x, w, target, lse)
    p = torch.exp(z - lse.double()[:, None])
    p[1, 0] -= 1
    p[2, 999] -= 1
    p[3, 500] -= 1
    p[4] = 0
    assert norm_off(dw[last:], p.t() @ x.double()) < 2 * HALF_STEP[BF16]
    assert norm_off(dx, p @ w[last:].double()) < 2 * HALF_STEP[BF16]


# ------------------------------------------------------------- distillation
def check_distill(x, w, index, logits, temperature):
    loss, lse = dr.linear_distill_fwd(x, w, index, logits, temperature=temperature)
    share = lr.shares64(index, logits, temperature)
    want, err, want_lse, lse_err = lr.loss(x, w, index, share, temperature)
    assert_close(loss, want, err, "loss")
    assert_close(lse, want_lse, lse_err, "lse")
    dloss, dlse = weights_for(x.shape[0], x.dtype)
    got = dr.linear_distill_bwd(dloss, dlse, x, w, index, logits, lse, temperature=temperature)
    check_grads(got, lr.loss_grads(dloss, dlse, x, w, index, share, lse, temperature), x.dtype, x.shape[0])
    return loss, lse, got


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("rows,hidden,vocab,top,temperature", [
    (1, 8, 1, 1, 1.0), (3, 64, 100, 7, 2.0), (33, 264, 1001, 20, 0.5), (130, 136, 700, 64, 1.0),
    (257, 72, 2000, 129, 1.5), (40, 64, 1100, 1024, 3.0), (300, 128, 300, 300, 1.0)])
def test_distillation(rows, hidden, vocab, top, temperature, dtype):
    check_distill(*loss_case(rows, hidden, vocab, dtype, top), temperature)


def test_distillation_in_pieces():
    x, w, index, logits = loss_case(4096, 64, 70001, BF16, 9)
    index[0, :4] = torch.tensor([0, 70000, 32768, 65536], device="cuda")
    index[0, 4:] = torch.tensor([1, 2, 3, 4, 5], device="cuda")
    check_distill(x, w, index, logits, 1.0)


def test_empty_entries_and_rows():
    x, w, index, logits = loss_case(90, 136, 500, BF16, 12)
    index[::3, ::2] = -1
    logits[::3, ::2] = float("nan")      # what an empty entry holds does not matter
    index[4], logits[7] = -5, float("-inf")
    logits[10, :3] = float("-inf")
    clean = logits.masked_fill(index < 0, 0.0)
    loss, lse = dr.linear_distill_fwd(x, w, index, logits, temperature=1.5)
    share = lr.shares64(index, clean, 1.5)
    want, err, want_lse, lse_err = lr.loss(x, w, index, share, 1.5)
    assert_close(loss, want, err, "loss")
    assert float(loss[4]) == 0 and float(loss[7]) == 0
    dloss, _ = weights_for(90, BF16)
    got = dr.linear_distill_bwd(dloss, None, x, w, index, logits, lse, temperature=1.5)
    check_grads(got, lr.loss_grads(dloss, None, x, w, index, share, lse, 1.5), BF16, 90)
    assert not got[0][4].any() and not got[0][7].any()
    x2 = x.clone()
    x2[4], x2[7] = float("nan"), float("inf")
    again = dr.linear_distill_bwd(dloss, None, x2, w, index, logits, lse, temperature=1.5)
    assert torch.equal(again[0], got[0]) and torch.equal(again[1], got[1])


def test_words_listed_twice_and_in_any_order():
    x, w, index, logits = loss_case(70, 64, 400, BF16, 10)
    index[:, 5] = index[:, 2]
    index[3, :] = 17
    loss, lse, got = check_distill(x, w, index, logits, 1.0)
    order = torch.tensor([9, 3, 0, 7, 5, 1, 8, 2, 4, 6], device="cuda")
    other = dr.linear_distill_fwd(x, w, index[:, order].contiguous(), logits[:, order].contiguous())
    share = lr.shares64(index, logits, 1.0)
    want, err, _, _ = lr.loss(x, w, index, share)
    assert_close(other[0], want, err, "loss in another order")


def test_entries_that_are_no_words():
    x, w, index, logits = loss_case(40, 64, 300, BF16, 6)
    index[1, 2], index[2, 0] = 300, 1 << 40
    loss, lse = dr.linear_distill_fwd(x, w, index, logits)
    assert loss[1:3].isnan().all() and loss[3:].isfinite().all() and lse.isfinite().all()
    dx, _ = dr.linear_distill_bwd(torch.ones(40, device="cuda"), None, x, w, index, logits, lse)
    assert dx[1:3].isnan().all() and dx[3:].isfinite().all()


@pytest.mark.parametrize("logits_dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_teacher_types(logits_dtype):
    x, w, index, logits = loss_case(50, 64, 300, F16, 8)
    check_distill(x, w, index, logits.to(logits_dtype), 1.0)


def test_one_entry_is_cross_entropy():
    x, w, target = loss_case(130, 136, 700, BF16)
    counted = torch.where(target < 0, torch.full_like(target, -1), target)
    ce = dr.linear_cross_entropy_fwd(x, w, target)
    di = dr.linear_distill_fwd(x, w, counted[:, None], torch.zeros(130, 1, device="cuda"))
    assert torch.equal(ce[1], di[1]) and torch.equal(ce[0], di[0])
    dloss, dlse = weights_for(130, BF16)
    a = dr.linear_cross_entropy_bwd(dloss, dlse, x, w, target, ce[1])
    b = dr.linear_distill_bwd(dloss, dlse, x, w, counted[:, None], torch.zeros(130, 1, device="cuda"), ce[1])
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


# ------------------------------------------------------------------ together
def program(seed, rows=333):
    """The end of a model: the last product into the residual stream, the norm, and both losses, forwards
    and backwards."""
    n = Make(seed, BF16)
    hidden, inner, vocab = 512, 1024, 3001
    a, w1, res = n(rows, inner), n(hidden, inner, std=inner ** -0.5), n(rows, hidden)
    b1, norm, head = n(hidden, std=0.5), n(hidden, std=0.1) + 1, n(vocab, hidden, std=hidden ** -0.5)
    target = n.words(vocab, rows)
    target[::4] = -100
    index, logits = n.top(rows, vocab, 16), n(rows, 16, dtype=torch.float32)
    dloss = torch.full((rows,), 1.0 / rows, device="cuda")

    def run():
        h = dr.linear_act_add_fwd(a, w1, b1, res, activation="gelu_tanh")
        y = dr.rmsnorm_fwd(h, norm, 1e-6)
        loss, lse = dr.linear_cross_entropy_fwd(y, head, target)
        kl, kl_lse = dr.linear_distill_fwd(y, head, index, logits, temperature=2.0)
        dy, dhead = dr.linear_cross_entropy_bwd(dloss, None, y, head, target, lse)
        dy2, dhead2 = dr.linear_distill_bwd(dloss, None, y, head, index, logits, kl_lse, temperature=2.0)
        dh, dnorm = dr.rmsnorm_bwd(dr.residual_add_fwd(dy, dy2), h, norm, 1e-6)
        da, dw1, db1 = dr.linear_act_add_bwd(dh, a, w1, b1, activation="gelu_tanh")
        return [h, y, loss, lse, kl, kl_lse, dy, dhead, dy2, dhead2, dh, dnorm, da, dw1, db1]

    def exact():
        t = [v.double().requires_grad_() for v in (a, w1, b1, norm, head)]
        h = res.double() + lr.act64(t[0] @ t[1].t() + t[2], "gelu_tanh")
        y = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + 1e-6) * t[3]
        z = y @ t[4].t()
        ce = torch.nn.functional.cross_entropy(z, target, reduction="none", ignore_index=-100)
        q = lr.shares64(index, logits, 2.0)
        kl = (q * (q.log() - torch.log_softmax(z / 2, 1).gather(1, index))).sum(1)
        grads = torch.autograd.grad(((ce + kl) * dloss.double()).sum(), t)
        return ce.detach(), kl.detach(), grads

    return run, exact


def same(got, want):
    return len(got) == len(want) and all(torch.equal(a.view(torch.uint8), b.view(torch.uint8))
                                         for a, b in zip(got, want))


@pytest.mark.parametrize("rows", [20, 333])
def test_together(rows):
    """Every tensor between is rounded to bf16, by at most 2^-8: a few of those reach each result."""
    run, exact = program(1, rows)
    got = run()
    ce, kl, grads = exact()
    assert float((got[2].double() - ce).abs().max()) < 0.1 and float((got[4].double() - kl).abs().max()) < 0.1
    assert norm_off(got[12], grads[0]) < 4 * 2.0 ** -8
    assert norm_off(got[13], grads[1]) < 4 * 2.0 ** -8
    assert norm_off(got[14], grads[2]) < 4 * 2.0 ** -8
    assert norm_off(got[11], grads[3]) < 4 * 2.0 ** -8
    assert norm_off(got[7].double() + got[9].double(), grads[4]) < 4 * 2.0 ** -8
    assert same(run(), got)


def test_gradient_of_a_program_s_function():
    """The calls under autograd, as a program uses them."""
    class Loss(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, w, target):
            loss, lse = dr.linear_cross_entropy_fwd(x, w, target)
            ctx.save_for_backward(x, w, target, lse)
            return loss, lse

        @staticmethod
        def backward(ctx, dloss, dlse):
            x, w, target, lse = ctx.saved_tensors
            return (*dr.linear_cross_entropy_bwd(dloss, dlse, x, w, target, lse), None)

    x, w, target = loss_case(60, 136, 900, BF16)
    x.requires_grad_()
    w.requires_grad_()
    loss, lse = Loss.apply(x, w, target)
    (loss.mean() + 0.01 * lse.square().mean()).backward()  # dloss arrives expanded
    with torch.no_grad():
        one = torch.full((60,), 1 / 60, device="cuda")
        want = dr.linear_cross_entropy_bwd(one, 0.02 / 60 * lse, x, w, target, lse)
    assert norm_off(x.grad, want[0].double()) < 2.0 ** -8 and norm_off(w.grad, want[1].double()) < 2.0 ** -8


def test_streams_and_threads():
    programs = [program(i)[0] for i in range(3)]
    want = [p() for p in programs]
    torch.cuda.synchronize()
    failed = []

    def work(i):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                results = [programs[i]() for _ in range(6)]
            stream.synchronize()
            if not all(same(r, want[i]) for r in results):
                failed.append(f"thread {i}: other bits")
        except Exception as e:  # reported by the main thread
            failed.append(f"thread {i}: {e!r}")

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(programs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join(120)
    assert not failed and not any(t.is_alive() for t in threads), failed


def test_stream_argument():
    x, w, b, r, _ = linear_case(200, 136, 264, BF16)
    want = dr.linear_act_add_fwd(x, w, b, r)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = dr.linear_act_add_fwd(x, w, b, r, stream=s)
    raw = dr.linear_act_add_fwd(x, w, b, r, stream=s.cuda_stream)
    s.synchronize()
    assert torch.equal(got, want) and torch.equal(raw, want)


def test_captured_graphs_side_by_side():
    programs = [program(10 + i)[0] for i in range(2)]
    want = [p() for p in programs]
    torch.cuda.synchronize()
    graphs, outs, streams = [], [], []
    for p in programs:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(p())
        graphs.append(graph)
        streams.append(torch.cuda.Stream())
    for _ in range(4):
        for o in outs:
            for t in o:
                t.zero_()
        torch.cuda.synchronize()
        for graph, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                graph.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert same(o, w)


# ------------------------------------------------------------------ refusals
def test_refusals():
    n = Make(1, BF16)
    x, w, b, t = n(20, 64), n(32, 64), n(32), torch.zeros(20, dtype=torch.int64, device="cuda")
    with pytest.raises(TypeError, match="bfloat16 or float16"):
        dr.linear_act_add_fwd(x.float(), w.float())
    with pytest.raises(TypeError, match="weight must hold"):
        dr.linear_act_add_fwd(x, w.half())
    with pytest.raises(ValueError, match="weight has shape"):
        dr.linear_act_add_fwd(x, n(32, 72))
    with pytest.raises(ValueError, match="activation must be one of"):
        dr.linear_act_add_fwd(x, w, activation="tanh")
    with pytest.raises(ValueError, match="residual has shape"):
        dr.linear_act_add_fwd(x, w, b, n(20, 40))
    with pytest.raises(ValueError, match="contiguous"):
        dr.linear_act_add_fwd(n(64, 20).t(), w)
    for bad in (lambda: dr.linear_act_add_fwd(n(20, 60), n(32, 60)),           # not a multiple of 8
                lambda: dr.linear_act_add_fwd(x, n(30, 64)),
                lambda: dr.linear_act_add_fwd(n(20, 68)[:, 4:], w),             # misaligned
                lambda: dr.linear_act_add_fwd(n(20, 68)[:, :64], w),            # a row stride of 68
                lambda: dr.linear_act_add_fwd(x, n(64, 64), out=x),                     # the output over x
                lambda: dr.linear_act_add_fwd(n(40, 4096), n(64, 4096), workspace=n(8)),
                lambda: dr.linear_cross_entropy_fwd(x, w, t, workspace=n(8)),
                lambda: dr.linear_cross_entropy_bwd(torch.ones(20, device="cuda"), None, x, w, t,
                                                    torch.ones(20, device="cuda"), dx=x),
                lambda: dr.linear_distill_fwd(x, w, t[:, None], torch.zeros(20, 1, device="cuda"), temperature=0.0),
                lambda: dr.linear_distill_fwd(x, w, torch.zeros(20, 1025, dtype=torch.int64, device="cuda"),
                                              torch.zeros(20, 1025, device="cuda"))):
        with pytest.raises(dr.DraddError):
            bad()
    with pytest.raises(TypeError, match="target must hold"):
        dr.linear_cross_entropy_fwd(x, w, t.int())
    with pytest.raises(ValueError, match="target has shape"):
        dr.linear_cross_entropy_fwd(x, w, t[:-1])
    with pytest.raises(TypeError, match="teacher_logits"):
        dr.linear_distill_fwd(x, w, t[:, None], None)
    with pytest.raises(ValueError, match="teacher_logits has shape"):
        dr.linear_distill_fwd(x, w, t[:, None], torch.zeros(20, 2, device="cuda"))
    with pytest.raises(ValueError, match="one value for all rows"):
        dr.linear_cross_entropy_bwd(torch.ones(40, device="cuda")[::2], None, x, w, t, torch.ones(20, device="cuda"))
    with pytest.raises(ValueError, match="not asked for"):
        dr.linear_act_add_bwd(n(20, 32), x, w, dx=n(20, 64), input_grad=False)
    with pytest.raises(ValueError, match="is on cpu"):
        dr.linear_act_add_fwd(x, w.cpu())
