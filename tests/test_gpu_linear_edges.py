"""Matrix products and losses where they could go wrong beside the sizes of
test_gpu_linear.py: workspaces at their least alignment, workers that take
several tiles."""
import pytest
import torch

import deterministic_residual_add_gb300 as dr
import linear_refs as lr
from test_gpu_linear import (BF16, F16, check_ce, check_linear, linear_case, loss_case, same,  # noqa: F401
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
