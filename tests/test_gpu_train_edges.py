"""The training and rotary calls where something outside the call could show
in its results: what earlier kernels left in shared memory, and calls of
other sizes made by other threads at the same time.  And k without heads,
inputs that require gradients, and the forward that goes with rmsnorm_bwd."""
import threading

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


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("tokens,hq,hk,dim,rot", [(9001, 2, 1, 64, 64), (300, 7, 3, 96, 96), (300, 7, 3, 40, 10),
                                                  (40, 32, 8, 128, 64)])
def test_a_head_of_nan_reaches_no_other(tokens, hq, hk, dim, rot, dtype):
    """Steps with fewer heads than lane groups, several tokens a step: what
    one head or token holds stays its own (but for the weights' gradients)."""
    q, k, gq, gk = (normal((1, tokens, h, dim), dtype, i) for i, h in enumerate((hq, hk, hq, hk)))
    qw, kw = normal(dim, dtype, 5, 0.1, 1.0), normal(dim, dtype, 6, 0.1, 1.0)
    freq = dr.rope_frequencies(rot, device=cuda())
    bad = torch.zeros(1, tokens, hq, 1, dtype=torch.bool, device=cuda())
    bad[:, ::5, hq - 1] = True
    bad[:, 3::7, 0] = True

    def calls(q, gq):
        return (dr.rope_fwd(q, k, freq), dr.qk_rmsnorm_rope_fwd(q, k, qw, kw, freq),
                dr.qk_rmsnorm_rope_bwd(gq, gk, q, k, qw, kw, freq))

    want = calls(q, gq)
    for nq, ng in ((q.masked_fill(bad, float("nan")), gq), (q, gq.masked_fill(bad, float("inf")))):
        for i, (got, w) in enumerate(zip(calls(nq, ng), want)):
            assert same([got[0].masked_fill(bad, 0), got[1]], [w[0].masked_fill(bad, 0), w[1]]), i
    assert same(calls(nq, ng)[2][3:], want[2][3:])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("hidden", [8, 72, 200, 504, 1000, 2056, 5000, 9000])
def test_norm_calls_whatever_shared_memory_holds(hidden, dtype):
    """Lanes and slots without a row, columns past the row's last."""
    for rows in (1, 5, 307):
        x, r, g = (normal((rows, hidden), dtype, i) for i in range(3))
        w = normal(hidden, dtype, 4, 0.1, 1.0)
        for call in (lambda: list(dr.dropout_add_rmsnorm_fwd(x, r, w, 0.25, seed=1)),
                     lambda: list(dr.dropout_add_rmsnorm_bwd(g, r, x, w, 0.25, seed=1)),
                     lambda: list(dr.add_rmsnorm_bwd(g, None, x, w))):
            leave_in_shared_memory(0)
            want = call()
            torch.cuda.synchronize()
            leave_in_shared_memory(-1)
            got = call()
            torch.cuda.synchronize()
            assert all(bool(torch.isfinite(t).all()) for t in got) and same(got, want), rows


# ------------------------------------------------- other sizes at the same time
def norm_calls(rows, hidden, dtype):
    x, r, g = (normal((rows, hidden), dtype, i) for i in range(3))
    w = normal(hidden, dtype, 4, 0.1, 1.0)
    return (lambda: list(dr.dropout_add_rmsnorm_fwd(x, r, w, 0.25, seed=1)),
            lambda: list(dr.dropout_add_rmsnorm_bwd(g, r, x, w, 0.25, seed=1)))


def rope_calls(rot, dim, dtype):
    q, k, gq, gk = (normal((1, 64, h, dim), dtype, i) for i, h in enumerate((4, 2, 4, 2)))
    qw, kw = normal(dim, dtype, 5, 0.1, 1.0), normal(dim, dtype, 6, 0.1, 1.0)
    freq = dr.rope_frequencies(rot, device=cuda())
    return (lambda: list(dr.qk_rmsnorm_rope_fwd(q, k, qw, kw, freq)),
            lambda: list(dr.qk_rmsnorm_rope_bwd(gq, gk, q, k, qw, kw, freq)))


# (call 0 or 1, makers): sizes that one kernel serves with different amounts of shared memory
SIDE_BY_SIDE = {
    "norm, 100 and 304 rows of 8192 bf16": (0, lambda: norm_calls(100, 8192, torch.bfloat16),
                                            lambda: norm_calls(304, 8192, torch.bfloat16)),
    "norm, rows of 8192 and 4104 bf16": (0, lambda: norm_calls(100, 8192, torch.bfloat16),
                                         lambda: norm_calls(100, 4104, torch.bfloat16)),
    "norm gradient, rows of 8192 and 6000 fp32": (1, lambda: norm_calls(50, 8192, torch.float32),
                                                  lambda: norm_calls(50, 6000, torch.float32)),
    "norm gradient, rows of 4096 and 2056 fp16": (1, lambda: norm_calls(50, 4096, torch.float16),
                                                  lambda: norm_calls(50, 2056, torch.float16)),
    "rotary gradient, 128 and 32 of 128 bf16": (1, lambda: rope_calls(128, 128, torch.bfloat16),
                                                lambda: rope_calls(32, 128, torch.bfloat16)),
    "rotary, 128 and 32 of 128 fp32": (0, lambda: rope_calls(128, 128, torch.float32),
                                       lambda: rope_calls(32, 128, torch.float32)),
}


@pytest.mark.parametrize("name", SIDE_BY_SIDE)
def test_threads_with_other_sizes(name):
    which, *makers = SIDE_BY_SIDE[name]
    programs = [m()[which] for m in makers] * 2
    want = [p() for p in programs]
    torch.cuda.synchronize()
    failed = []
    start = threading.Barrier(len(programs))

    def work(i):
        try:
            stream = torch.cuda.Stream()
            start.wait(60)
            with torch.cuda.stream(stream):
                for _ in range(10):
                    results = [programs[i]() for _ in range(150)]
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


# --------------------------------------------------------------- no k heads
@pytest.mark.parametrize("batch", [2, 0])
def test_k_of_no_heads(batch):
    """A sum over no heads is zero: k's weight gradient, given or not."""
    q, gq = normal((batch, 7, 4, 64), torch.bfloat16, 1), normal((batch, 7, 4, 64), torch.bfloat16, 2)
    k = q[:, :, :0]
    w = normal(64, torch.bfloat16, 3, 0.1, 1.0)
    freq = dr.rope_frequencies(64, device=cuda())
    alone = dr.qk_rmsnorm_rope_bwd(gq, None, q, None, w, None, freq)
    for _ in range(3):
        torch.full((64,), float("nan"), device=cuda())  # what the next allocation of this size may find
        got = dr.qk_rmsnorm_rope_bwd(gq, k, q, k, w, w, freq)
        assert same([got[0], got[2]], [alone[0], alone[2]]) and got[1].shape == k.shape
        assert bool((got[3] == 0).all())
    mine = torch.full((64,), float("nan"), device=cuda())
    got = dr.qk_rmsnorm_rope_bwd(gq, k, q, k, w, w, freq, dk_weight=mine)
    assert got[3] is mine and bool((mine == 0).all()) and same([got[0], got[2]], [alone[0], alone[2]])
    assert dr.qk_rmsnorm_rope_bwd(gq, k, q, k, w, w, freq, weight_grad=False)[2:] == (None, None)


# ----------------------------------------------------------------- autograd
class DropNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, weight, p, seed):
        out, h = dr.dropout_add_rmsnorm_fwd(x, residual, weight, p, seed=seed)
        ctx.save_for_backward(h, weight)
        ctx.how = p, seed
        return out, h

    @staticmethod
    def backward(ctx, dout, dh):
        h, weight = ctx.saved_tensors
        p, seed = ctx.how
        dx, dres, dw = dr.dropout_add_rmsnorm_bwd(dout.contiguous(), dh.contiguous(), h, weight, p, seed=seed)
        return dx, dres, dw.to(weight.dtype), None, None


def test_inputs_that_require_gradients():
    """A call's results carry no graph; inside a program's own Function the
    gradients are those of the calls."""
    x, r, g, gh = (normal((40, 512), torch.float32, i) for i in range(4))
    w = normal(512, torch.float32, 5, 0.1, 1.0)
    leaves = [t.clone().requires_grad_() for t in (x, r, w)]
    out, h = dr.dropout_add_rmsnorm_fwd(*leaves, 0.2, seed=7)
    assert not out.requires_grad and not h.requires_grad
    freq = dr.rope_frequencies(64, device=cuda())
    q = normal((1, 40, 8, 64), torch.float32, 6).requires_grad_()
    assert not dr.rope_fwd(q, None, freq)[0].requires_grad
    out2, h2 = DropNorm.apply(*leaves, 0.2, 7)
    assert same([out2.detach(), h2.detach()], [out, h])
    got = torch.autograd.grad([out2, h2], leaves, [g, gh])
    assert same(got, dr.dropout_add_rmsnorm_bwd(g, gh, h, w, 0.2, seed=7))


@pytest.mark.parametrize("hidden", [200, 4096])
def test_norm_forward_without_a_residual(hidden):
    """With p = 0 and a residual of zeros the forward is the plain norm's, and
    rmsnorm_bwd its gradient: the same bits as from its residual_out."""
    w, zeros = normal(hidden, torch.bfloat16, 5, 0.1, 1.0), torch.zeros(30, hidden, dtype=torch.bfloat16, device=cuda())
    x, g = normal((30, hidden), torch.bfloat16, 1), normal((30, hidden), torch.bfloat16, 2)
    out, h = dr.dropout_add_rmsnorm_fwd(x, zeros, w, 0.0, seed=1)
    assert same([out, h], [dr.rmsnorm_fwd(x, w), x])
    for dtype in (torch.bfloat16, torch.float16, torch.float32):
        x, g, z, v = (t.to(dtype) for t in (x, g, zeros, w))
        h = dr.dropout_add_rmsnorm_fwd(x, z, v, 0.0, seed=1)[1]
        assert same(dr.rmsnorm_bwd(g, x, v), dr.add_rmsnorm_bwd(g, None, h, v))
