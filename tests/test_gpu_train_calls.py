"""The training and rotary calls in company: threads on streams of
their own, and captured graphs replayed side by side.  Every result has to
have the bits of the same call made alone."""
import threading

import pytest
import torch

import deterministic_residual_add_gb300 as dr

pytestmark = pytest.mark.gpu

SHAPE = (2, 333, 6, 2, 128)  # batch, seq, q heads, k heads, head dim


def calls(seed):
    """The calls of one program over inputs of its own, outputs as one list."""
    dev = torch.device("cuda", 0)
    g = torch.Generator().manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g).to(torch.bfloat16).to(dev)

    b, s, hq, hk, d = SHAPE
    x, residual, dout, dres = (normal(777, 2048) for _ in range(4))
    weight, qw, kw = normal(2048), normal(d), normal(d)
    q, k, gq, gk = (normal(b, s, h, d) for h in (hq, hk, hq, hk))
    freq = dr.rope_frequencies(64, device=dev)

    def program():
        y, h = dr.dropout_add_rmsnorm_fwd(x, residual, weight, 0.25, seed=seed, offset=3)
        dx, dh, dw = dr.dropout_add_rmsnorm_bwd(dout, dres, h, weight, 0.25, seed=seed, offset=3)
        qr, kr = dr.qk_rmsnorm_rope_fwd(q, k, qw, kw, freq)
        dq, dk, dqw, dkw = dr.qk_rmsnorm_rope_bwd(gq, gk, q, k, qw, kw, freq)
        r = dr.rope_fwd(q, k, freq, interleaved=True)
        return [y, h, dx, dh, dw, qr, kr, dq, dk, dqw, dkw, *r, dr.dropout_add_fwd(x, residual, 0.5, seed=seed),
                dr.dropout_fwd(x, 0.5, seed=seed)]

    return program


def same(got, want):
    return len(got) == len(want) and all(torch.equal(a.view(torch.uint8), b.view(torch.uint8))
                                         for a, b in zip(got, want))


def test_threads_on_streams_of_their_own():
    programs = [calls(i) for i in range(4)]
    want = [p() for p in programs]
    torch.cuda.synchronize()
    failed = []

    def work(i):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                results = [programs[i]() for _ in range(20)]
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


def test_captured_graphs_side_by_side():
    programs = [calls(10 + i) for i in range(2)]
    want = [p() for p in programs]
    torch.cuda.synchronize()
    graphs, outs, streams = [], [], []
    for p in programs:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(p())
        graphs.append(graph)
        streams.append(torch.cuda.Stream())
    for _ in range(10):
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


def test_fp32_tensors_on_16_byte_boundaries():
    """fp32 blocks at 32-byte boundaries move in one store, others in two:
    the same bits, and the neighbours stay."""
    dev = torch.device("cuda", 0)
    g = torch.Generator().manual_seed(3)

    def normal(*shape):
        return torch.randn(*shape, generator=g).to(dev)

    def moved(shape):
        """A contiguous fp32 tensor 16 bytes past a 32-byte boundary, inside a buffer of NaN."""
        n = torch.Size(shape).numel()
        buf = torch.full((n + 16,), float("nan"), device=dev)
        return buf, buf[4:4 + n].view(shape)

    def put(t):
        m = moved(t.shape)[1]
        assert m.data_ptr() % 32 == 16
        return m.copy_(t)

    for rows, hidden in ((37, 264), (300, 1024), (500, 4096)):
        x, r, d, w = normal(rows, hidden), normal(rows, hidden), normal(rows, hidden), normal(hidden)
        want = [dr.dropout_fwd(x, 0.3, seed=1), dr.dropout_add_fwd(x, r, 0.3, seed=1),
                *dr.dropout_add_rmsnorm_fwd(x, r, w, 0.3, seed=1)]
        want += dr.dropout_add_rmsnorm_bwd(d, r, want[3], w, 0.3, seed=1)[:2]
        bufs, o = zip(*(moved((rows, hidden)) for _ in want))
        dr.dropout_fwd(put(x), 0.3, seed=1, out=o[0])
        dr.dropout_add_fwd(put(x), put(r), 0.3, seed=1, residual_out=o[1])
        dr.dropout_add_rmsnorm_fwd(put(x), put(r), put(w), 0.3, seed=1, out=o[2], residual_out=o[3])
        dr.dropout_add_rmsnorm_bwd(put(d), put(r), o[3], put(w), 0.3, seed=1, dx=o[4], dresidual=o[5])
        for b, got, t in zip(bufs, o, want):
            assert same([got], [t]) and b[:4].isnan().all() and b[-12:].isnan().all()
    # heads 100 elements apart: every other one on a 32-byte boundary
    freq = dr.rope_frequencies(96, device=dev)
    q, dq, w = normal(2, 41, 6, 96), normal(2, 41, 6, 96), normal(96)
    want = [dr.rope_fwd(q, None, freq)[0], dr.qk_rmsnorm_rope_fwd(q, None, w, None, freq)[0],
            dr.qk_rmsnorm_rope_bwd(dq, None, q, None, w, None, freq)[0]]
    bufs = [torch.full((2, 41, 6, 100), float("nan"), device=dev) for _ in want]
    o = [b[..., :96] for b in bufs]
    dr.rope_fwd(q, None, freq, q_out=o[0])
    dr.qk_rmsnorm_rope_fwd(q, None, w, None, freq, q_out=o[1])
    dr.qk_rmsnorm_rope_bwd(dq, None, q, None, w, None, freq, dq=o[2])
    for b, got, t in zip(bufs, o, want):
        assert same([got.contiguous()], [t]) and b[..., 96:].isnan().all()
