"""Matrix products and losses where they could go wrong beside the sizes of
test_gpu_linear.py: workspaces at their least alignment, workers that take
several tiles, few rows, long sums, rows that the call in front writes."""
import pytest
import torch

import deterministic_residual_add_gb300 as dr
import linear_refs as lr
from linear_refs import HALF_STEP, norm_off
from test_gpu_linear import (BF16, F16, Make, check_ce, check_linear, linear_case, loss_case, same,  # noqa: F401
                             status_clear, weights_for)

pytestmark = pytest.mark.gpu


def workspace_for(name, *sizes):
    """A workspace of the stated size that lies on 16 bytes and not on 32, between bytes that have to stay."""
    need = lr.c_entry(dr.lib(), name + "_workspace_bytes")(*sizes)
    assert need > 0
    room = torch.full((need + 64,), 0xA5, dtype=torch.uint8, device="cuda")
    start = 16 if room.data_ptr() % 32 == 0 else 32
    part = room[start:start + need]
    assert part.data_ptr() % 32 == 16
    return part, lambda: bool((room[:start] == 0xA5).all() and (room[start + need:] == 0xA5).all())


@pytest.mark.parametrize("rows,inner,cols", [(40, 4096, 264), (200, 2048, 136)])
def test_split_products_in_a_workspace_on_16_bytes(rows, inner, cols):
    """Split sums: the product and its activation's derivative, dx and dweight."""
    x, w, b, r, dout = linear_case(rows, inner, cols, BF16)
    ws, kept = workspace_for("linear_act_add_fwd", rows, inner, cols)
    want = dr.linear_act_add_fwd(x, w, b, r, activation="silu")
    assert torch.equal(dr.linear_act_add_fwd(x, w, b, r, activation="silu", workspace=ws), want) and kept()
    ws, kept = workspace_for("linear_act_add_bwd", rows, inner, cols, dr.ACTIVATIONS["silu"], 1, 1, 1)
    want = dr.linear_act_add_bwd(dout, x, w, b, activation="silu")
    assert same(dr.linear_act_add_bwd(dout, x, w, b, activation="silu", workspace=ws), want) and kept()


def test_long_weight_gradient_in_a_workspace_on_16_bytes():
    """4000 rows of 64 by 72: dweight is one tile, its sum of 63 steps is split."""
    x, w, b, _, dout = linear_case(4000, 64, 72, F16)
    ws, kept = workspace_for("linear_act_add_bwd", 4000, 64, 72, 0, 1, 1, 1)
    want = dr.linear_act_add_bwd(dout, x, w, b)
    assert same(dr.linear_act_add_bwd(dout, x, w, b, workspace=ws), want) and kept()


# logits of few words summed up in the workspace; dx from splits; pieces of the vocabulary
@pytest.mark.parametrize("rows,hidden,vocab", [(40, 2048, 1001), (300, 1024, 500), (40, 264, 60001), (4096, 64, 70001)])
def test_losses_in_a_workspace_on_16_bytes(rows, hidden, vocab):
    x, w, target = loss_case(rows, hidden, vocab, BF16)
    ws, kept = workspace_for("linear_cross_entropy_fwd", rows, hidden, vocab)
    want = dr.linear_cross_entropy_fwd(x, w, target)
    assert same(dr.linear_cross_entropy_fwd(x, w, target, workspace=ws), want) and kept()
    dloss, dlse = weights_for(rows, BF16)
    ws, kept = workspace_for("linear_cross_entropy_bwd", rows, hidden, vocab)
    grads = dr.linear_cross_entropy_bwd(dloss, dlse, x, w, target, want[1])
    assert same(dr.linear_cross_entropy_bwd(dloss, dlse, x, w, target, want[1], workspace=ws), grads) and kept()
    index, logits = target[:, None].expand(rows, 3).contiguous(), torch.zeros(rows, 3, device="cuda")
    ws, kept = workspace_for("linear_distill_fwd", rows, hidden, vocab, 3)
    want = dr.linear_distill_fwd(x, w, index, logits)
    assert same(dr.linear_distill_fwd(x, w, index, logits, workspace=ws), want) and kept()
    ws, kept = workspace_for("linear_distill_bwd", rows, hidden, vocab, 3)
    grads = dr.linear_distill_bwd(dloss, dlse, x, w, index, logits, want[1])
    assert same(dr.linear_distill_bwd(dloss, dlse, x, w, index, logits, want[1], workspace=ws), grads) and kept()


# Tiles of 256 rows by pairs of CTAs: 170 for 76 pairs in two bands, the last row and the last 8 columns tiles of their
# own; sums of 33 steps (the deep form of the epilogues) and of 5.  Tiles of 128 rows by single CTAs: 157 for 152.
@pytest.mark.parametrize("act,bias,residual", [("none", False, False), ("silu", True, True), ("gelu", True, False),
                                               ("relu", False, True)])
@pytest.mark.parametrize("rows,inner,cols", [(2305, 2056, 4104), (2305, 264, 4104), (100, 2056, 40008),
                                             (100, 264, 40008)])
def test_several_tiles_a_worker(rows, inner, cols, act, bias, residual):
    """The next tile's residual or dout comes into the box that the last tile's results leave from."""
    x, w, b, r, dout = linear_case(rows, inner, cols, BF16 if bias else F16, bias, residual)
    check_linear(x, w, b, r, dout, act)
    want = dr.linear_act_add_fwd(x, w, b, r, activation=act)
    grads = dr.linear_act_add_bwd(dout, x, w, b, activation=act)
    for _ in range(3):
        assert torch.equal(dr.linear_act_add_fwd(x, w, b, r, activation=act), want)
        again = dr.linear_act_add_bwd(dout, x, w, b, activation=act)
        assert all(p is q or torch.equal(p, q) for p, q in zip(again, grads))
    if residual:
        inplace = r.clone()
        dr.linear_act_add_fwd(x, w, b, inplace, activation=act, out=inplace)
        assert torch.equal(inplace, want)


def test_losses_of_long_sums_in_two_bands():
    """10 tile rows, of which L2 keeps 5 with sums this long: bands of 8 and 2."""
    check_ce(*loss_case(2305, 16392, 700, BF16))


# logits summed in one go and from splits, by single CTAs and by pairs
LONG_SUMS = [(40, 8192, 1001), (300, 8192, 500), (64, 8192, 20001), (300, 16384, 20001)]


def check_logits(x, w, target, off):
    """lse and loss against fp64, where every logit may be off by `off` of its size and no more."""
    z = x.double() @ w.double().t()
    want = torch.logsumexp(z, 1)
    at = z.gather(1, target[:, None])[:, 0]
    loss, lse = dr.linear_cross_entropy_fwd(x, w, target)
    high = z.abs().amax(1)
    # beside the logits: exponentials and their sums 2^-22, a rounding for a part joined, the exponents' own
    bound = off * high + (-(-w.shape[0] // 128) + 96) * 2.0 ** -24 + 8 * 2.0 ** -24 * (want.abs() + high)
    assert float(((lse - want).abs() / bound).max()) <= 1
    bound = bound + off * high + 65 * 2.0 ** -24 * (at.abs() + want.abs() + 1)
    assert float(((loss - (want - at)).abs() / bound).max()) <= 1


@pytest.mark.parametrize("rows,hidden,vocab", LONG_SUMS)
def test_logits_of_one_term_are_exact(rows, hidden, vocab):
    """One nonzero number a row of x: its products are whole in fp32 and nothing is cut off, however long the rows.
    Logits of some hundreds: what lies between one of them and the result are a few roundings."""
    g = torch.Generator(device="cuda").manual_seed(hidden + vocab)
    x = torch.zeros(rows, hidden, dtype=BF16, device="cuda")
    x[torch.arange(rows), torch.randint(0, hidden, (rows,), generator=g, device="cuda")] = 150.0
    w = torch.randn(vocab, hidden, generator=g, device="cuda").to(BF16)
    check_logits(x, w, torch.randint(0, vocab, (rows,), generator=g, device="cuda"), 0.0)


@pytest.mark.parametrize("rows,hidden,vocab", LONG_SUMS)
def test_long_sums_of_one_sign(rows, hidden, vocab):
    """A sum is taken out after 512 terms, 32 steps of 16.  A step cuts off at most 2^-23 of the sum so far, which with
    terms of one sign is i / 32 of the run's: 16.5 * 2^-23 in all, of the run's sum and so of all of them.  Beside it
    each joined run is rounded, 2^-24 of the sum so far.  Without the breaks 8192 terms lose 8.7e-6."""
    g = torch.Generator(device="cuda").manual_seed(hidden + vocab)
    x = torch.randn(rows, hidden, generator=g, device="cuda").abs().to(BF16)
    w = (torch.randn(vocab, hidden, generator=g, device="cuda").abs() * (80 / hidden)).to(BF16)
    runs = hidden // 512
    check_logits(x, w, torch.randint(0, vocab, (rows,), generator=g, device="cuda"),
                 16.5 * 2.0 ** -23 + (runs + 1) / 2 * 2.0 ** -24)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("rows,hidden,vocab", LONG_SUMS)
def test_gradients_of_long_sums_of_one_sign(rows, hidden, vocab, dtype):
    """Logits of about 50: what each lacks is the same for all of a row, and 8.7e-6 of them would be 4.4e-4 of every
    p, which the differences that dx is made of show many times over."""
    g = torch.Generator(device="cuda").manual_seed(hidden + vocab)
    x = torch.randn(rows, hidden, generator=g, device="cuda").abs().to(dtype)
    w = (torch.randn(vocab, hidden, generator=g, device="cuda").abs() * (80 / hidden)).to(dtype)
    target = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
    dloss = torch.full((rows,), 8.0, device="cuda")
    lse = dr.linear_cross_entropy_fwd(x, w, target)[1]
    got = dr.linear_cross_entropy_bwd(dloss, None, x, w, target, lse)
    z = x.double() @ w.double().t()
    dz = torch.softmax(z, 1).scatter_add_(1, target[:, None], torch.full((rows, 1), -1.0, device="cuda").double()) * 8
    assert norm_off(got[0], dz @ w.double()) < HALF_STEP[dtype]
    assert norm_off(got[1], dz.t() @ x.double()) < HALF_STEP[dtype]


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("rows,inner,cols", [
    (1, 8192, 6144), (8, 1024, 24576), (3, 8, 3648), (9, 5120, 4096), (16, 1024, 14592),  # their own kernel
    (8, 10240, 520), (1, 64, 3656), (2, 512, 8200), (2, 1024, 24584), (16, 5128, 264), (9, 2048, 14600),  # tiles
    (12, 512, 14600)])
def test_few_rows_on_both_sides_of_the_choice(rows, inner, cols, dtype):
    check_linear(*linear_case(rows, inner, cols, dtype), "silu")


@pytest.mark.parametrize("rows", [1, 8, 16, 64, 200])
def test_rows_from_the_grid_in_front(rows):
    """x, bias and residual are written by the call in front, which a product may start beside: buffers that are used
    again and again never give an older content."""
    n = Make(rows, BF16)
    inner, cols, turns = 512, 264, 24
    w, norm = n(cols, inner, std=inner ** -0.5), n(inner)
    inputs, biases, rest = n(turns, rows, inner), n(turns, 1, cols), n(turns, rows, cols)
    x, b, r = torch.empty_like(inputs[0]), torch.empty_like(biases[0]), torch.empty_like(rest[0])
    zero, zeros = torch.zeros_like(b), torch.zeros_like(r)
    want = []
    for i in range(turns):
        y = dr.rmsnorm_fwd(inputs[i], norm, 1e-6)
        torch.cuda.synchronize()
        want.append(dr.linear_act_add_fwd(y, w, biases[i, 0], rest[i], activation="silu"))
        torch.cuda.synchronize()
    got = []
    for i in range(turns):
        dr.residual_add_fwd(biases[i], zero, residual_out=b)
        dr.residual_add_fwd(rest[i], zeros, residual_out=r)
        dr.rmsnorm_fwd(inputs[i], norm, 1e-6, out=x)
        got.append(dr.linear_act_add_fwd(x, w, b[0], r, activation="silu"))
    assert same(got, want)
