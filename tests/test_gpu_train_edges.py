"""The training and rotary calls where something outside the call could show
in its results."""
import pytest
import torch

import deterministic_residual_add_gb300 as dr

pytestmark = pytest.mark.gpu


def cuda():
    return torch.device("cuda", 0)


def normal(shape, dtype, seed, std=1.0, mean=0.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std + mean).to(dtype).to(cuda())


def same(got, want):
    return len(got) == len(want) and all(torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))
                                         for a, b in zip(got, want))


# ---------------------------------------------------------- shared memory
def leave_in_shared_memory(pattern):
    """Fills most of every SM's shared memory with a 16-bit pattern: the norm's
    gradient stages rows of 8192 through it, four 48 KB slots and one CTA an SM."""
    rows = torch.full((152 * 8, 8192), pattern, dtype=torch.int16, device=cuda()).view(torch.bfloat16)
    dr.add_rmsnorm_bwd(rows, rows, rows, torch.ones(8192, dtype=torch.bfloat16, device=cuda()), weight_grad=False)
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dim,rot", [(80, 40), (96, 24), (33, 6), (32, 8), (40, 10), (24, 6), (128, 128), (496, 8)])
@pytest.mark.parametrize("tokens,hq,hk", [(300, 4, 2), (9001, 2, 1)])
def test_rotary_calls_whatever_shared_memory_holds(tokens, hq, hk, dim, rot, inter, dtype):
    """Rotary widths that do not fill the tables of cosines and sines: the
    rest of a table is whatever an earlier kernel left there, NaN included."""
    q, k, gq, gk = (normal((1, tokens, h, dim), dtype, i) for i, h in enumerate((hq, hk, hq, hk)))
    qw, kw = normal(dim, dtype, 5, 0.1, 1.0), normal(dim, dtype, 6, 0.1, 1.0)
    freq = dr.rope_frequencies(rot, device=cuda())
    on = dict(position0=5, interleaved=inter)
    calls = (lambda: dr.rope_fwd(q, k, freq, **on), lambda: dr.qk_rmsnorm_rope_fwd(q, k, qw, kw, freq, **on),
             lambda: dr.qk_rmsnorm_rope_bwd(gq, gk, q, k, qw, kw, freq, **on))
    for i, call in enumerate(calls):
        leave_in_shared_memory(0)
        want = call()
        torch.cuda.synchronize()
        leave_in_shared_memory(-1)
        got = call()
        torch.cuda.synchronize()
        assert all(bool(torch.isfinite(t).all()) for t in got), f"call {i}: not finite"
        assert same(got, want), f"call {i}: other bits"
