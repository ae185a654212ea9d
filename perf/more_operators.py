"""Cases, plain forms and exact results of the matrix products with something fused behind them.

  linear       linear_act_add_fwd and _bwd: residual + activation(x W^T + bias), and its gradients
  ce           linear_cross_entropy_fwd and _bwd: softmax cross entropy of the logits x W^T, which are not
               kept, and its gradients
  distill      linear_distill_fwd and _bwd: the divergence of the softmax of x W^T from a teacher's top
               logits, and its gradients

With `own` false, run() is the plain form: elementary torch operations in fp32.  With `own` true it calls
the framework.  exact() gives the same results from the definitions in fp64.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
IGNORED = -100


def _linear(name, op, dtype, rows, inner, cols, act, bias, residual):
    return {"name": name, "op": op, "dtype": dtype, "rows": rows, "inner": inner, "cols": cols, "act": act,
            "bias": bias, "residual": residual}


def _loss(name, op, dtype, rows, inner, vocab, top, temperature):
    return {"name": name, "op": op, "dtype": dtype, "rows": rows, "inner": inner, "vocab": vocab, "top": top,
            "temperature": temperature}


def listed():
    return [
        # serving: the projection behind attention for one token, into the residual stream
        _linear("linear_1_4096x4096_bf16", "linear", "bf16", 1, 4096, 4096, "none", False, True),
        # serving: the first half of an MLP for 48 sequences' tokens
        _linear("linear_48_8192x5120_fp16", "linear", "fp16", 48, 5120, 8192, "gelu", True, False),
        # a prompt batch: the second half of an MLP, into the residual stream
        _linear("linear_8192_4096x16384_bf16", "linear", "bf16", 8192, 16384, 4096, "none", True, True),
        # training: gradients of a small layer for an odd number of tokens
        _linear("linear_bwd_1999_4096x1024_fp16", "linear_bwd", "fp16", 1999, 1024, 4096, "gelu_tanh", True, False),
        # training: gradients of the first half of an MLP for 8192 tokens
        _linear("linear_bwd_8192_16384x4096_bf16", "linear_bwd", "bf16", 8192, 4096, 16384, "silu", True, False),
        # scoring a few given tokens
        _loss("ce_64_4096x32768_bf16", "ce", "bf16", 64, 4096, 32768, 0, 1.0),
        # evaluation: 4096 tokens over a large vocabulary
        _loss("ce_4096_4096x128000_bf16", "ce", "bf16", 4096, 4096, 128000, 0, 1.0),
        # training a small model: odd numbers of tokens and words
        _loss("ce_bwd_511_1024x50001_fp16", "ce_bwd", "fp16", 511, 1024, 50001, 0, 1.0),
        # training: gradients of hidden states and weights for 4096 tokens
        _loss("ce_bwd_4096_4096x65536_bf16", "ce_bwd", "bf16", 4096, 4096, 65536, 0, 1.0),
        # a short answer against a teacher's 20 likeliest words
        _loss("distill_33_2048x32001_fp16", "distill", "fp16", 33, 2048, 32001, 20, 2.0),
        # a batch against a teacher's 64 likeliest words
        _loss("distill_2048_4096x65536_bf16", "distill", "bf16", 2048, 4096, 65536, 64, 1.0),
        # its gradients, 128 words a token
        _loss("distill_bwd_2048_4096x65536_bf16", "distill_bwd", "bf16", 2048, 4096, 65536, 128, 1.5),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "linear", "linear_bwd", "linear_bwd", "ce", "ce", "ce_bwd", "ce_bwd", "distill",
                     "distill_bwd"])
    case = {"op": op, "dtype": rng.choice(["bf16", "bf16", "fp16"])}
    if op.startswith("linear"):
        inner, cols = 8 * _log(rng, 32, 2048), 8 * _log(rng, 32, 2048)
        # the largest listed ones: 8192 x 4096 x 16384 numbers to multiply, 16384 x 8192 in a tensor
        most = min(8192, 8192 * 4096 * 16384 // (inner * cols), 8192 * 16384 // max(inner, cols))
        rows = _log(rng, 1, 64) if rng.random() < 0.35 else _log(rng, 1, most)
        return case | {"rows": min(rows, most), "inner": inner, "cols": cols,
                       "act": rng.choice(["none", "none", "relu", "gelu", "gelu_tanh", "silu"]),
                       "bias": rng.random() < 0.6, "residual": op == "linear" and rng.random() < 0.5}
    inner = 8 * _log(rng, 32, 1024)
    vocab = _log(rng, 1000, min(131072, 65536 * 4096 // inner))
    rows = _log(rng, 1, min(8192, 4096 * 4096 * 65536 // (inner * vocab), 4096 * 65536 // vocab))
    top = _log(rng, 1, 256) if op.startswith("distill") else 0
    return case | {"rows": rows, "inner": inner, "vocab": vocab, "top": min(top, vocab),
                   "temperature": rng.choice([1.0, 1.0, 2.0, 0.7]) if top else 1.0}


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, std=1.0):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.float32).mul_(std)

    s = {"case": case}
    n, k = case["rows"], case["inner"]
    if case["op"].startswith("linear"):
        m = case["cols"]
        s["x"], s["weight"] = normal(n, k).to(dt), normal(m, k, std=k ** -0.5).to(dt)
        s["bias"] = normal(m, std=0.5).to(dt) if case["bias"] else None
        s["residual"] = normal(n, m, std=2.0).to(dt) if case["residual"] else None
        if case["op"] == "linear_bwd":
            s["dout"] = normal(n, m).to(dt)
        return s
    v = case["vocab"]
    # logits with a deviation of 1.5, and the words that follow likelier than the others, some by much
    weight = normal(v, k, std=1.5 * k ** -0.5)
    words = torch.randint(0, v, (n,), generator=g, device=dev)
    x = normal(n, k) + weight[words] * (4.0 * torch.rand(n, 1, generator=g, device=dev))
    s["x"], s["weight"] = x.to(dt), weight.to(dt)
    skipped = torch.rand(n, generator=g, device=dev) < 0.1  # padding, or a prompt's own words
    if case["op"].startswith("ce"):
        s["target"] = words.masked_fill(skipped, IGNORED)
    else:
        # a teacher near the student: its likeliest words, in its order
        logits = s["x"].float() @ s["weight"].float().t()
        top = (logits + normal(n, v, std=0.3)).topk(case["top"], dim=1)
        s["teacher_index"] = top.indices.masked_fill(skipped[:, None], -1)
        s["teacher_logits"] = top.values
    if case["op"].endswith("bwd"):
        scaled = s["x"].float() @ s["weight"].float().t() / case["temperature"]
        s["lse"] = scaled.logsumexp(1)
        # the mean over the tokens, weighted; with 16-bit floats of few exponents the loss is scaled up
        size = 8.0 if case["dtype"] == "fp16" else 1.0 / n
        s["dloss"] = size * (0.5 + torch.rand(n, generator=g, device=dev))
        s["dlse"] = 2e-4 * s["lse"] * size  # of a small penalty on the squared lse
    return s


# ------------------------------------------------------------------ plain forms
def _act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, 0.0)
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    return z


def _slope(z, act):
    if act == "relu":
        return (z > 0).float()
    if act == "gelu":
        return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * c * (1.0 + 3 * 0.044715 * z * z)
    if act == "silu":
        f = 1.0 / (1.0 + torch.exp(-z))
        return f * (1.0 + z * (1.0 - f))
    return torch.ones_like(z)


def _shares(s):
    """The words of every token and their share of the teacher's distribution."""
    if s["case"]["op"].startswith("ce"):
        index = s["target"][:, None]
        return index.clamp(min=0), (index != IGNORED).float()
    index, logits = s["teacher_index"], s["teacher_logits"] / s["case"]["temperature"]
    e = torch.exp(logits - logits.amax(1, keepdim=True)) * (index >= 0)
    return index.clamp(min=0), e / e.sum(1, keepdim=True).clamp(min=1e-30)


def _plain(s):
    case = s["case"]
    dt = DTYPES[case["dtype"]]
    x, w = s["x"].float(), s["weight"].float()
    if case["op"].startswith("linear"):
        if case["op"] == "linear" or case["act"] != "none":
            z = x @ w.t()
            if s["bias"] is not None:
                z = z + s["bias"].float()
        if case["op"] == "linear":
            y = _act(z, case["act"])
            return (y if s["residual"] is None else y + s["residual"].float()).to(dt)
        dz = s["dout"].float()
        if case["act"] != "none":
            dz = dz * _slope(z, case["act"])
        return (dz @ w).to(dt), (dz.t() @ x).to(dt), dz.sum(0).to(dt) if s["bias"] is not None else None
    z = (x @ w.t()) / case["temperature"]
    index, share = _shares(s)
    if not case["op"].endswith("bwd"):
        high = z.amax(1, keepdim=True)
        lse = torch.log(torch.exp(z - high).sum(1)) + high[:, 0]
        entropy = torch.where(share > 0, share * torch.log(share.clamp(min=1e-30)), 0.0).sum(1)
        return entropy + (share * (lse[:, None] - z.gather(1, index))).sum(1), lse
    g = s["dloss"] * (share.sum(1) > 0)
    dz = torch.exp(z - s["lse"][:, None]) * (g + s["dlse"])[:, None]
    dz.scatter_add_(1, index, -share * g[:, None])
    dz = dz / case["temperature"]
    return (dz @ w).to(dt), (dz.t() @ x).to(dt)


def run(s):
    if not own:
        return _plain(s)
    import deterministic_residual_add_gb300 as dr

    case, op = s["case"], s["case"]["op"]
    if op == "linear":
        return dr.linear_act_add_fwd(s["x"], s["weight"], s["bias"], s["residual"], activation=case["act"])
    if op == "linear_bwd":
        return dr.linear_act_add_bwd(s["dout"], s["x"], s["weight"], s["bias"], activation=case["act"])
    if op == "ce":
        return dr.linear_cross_entropy_fwd(s["x"], s["weight"], s["target"], ignore_index=IGNORED)
    if op == "ce_bwd":
        return dr.linear_cross_entropy_bwd(s["dloss"], s["dlse"], s["x"], s["weight"], s["target"], s["lse"],
                                           ignore_index=IGNORED)
    if op == "distill":
        return dr.linear_distill_fwd(s["x"], s["weight"], s["teacher_index"], s["teacher_logits"],
                                     temperature=case["temperature"])
    return dr.linear_distill_bwd(s["dloss"], s["dlse"], s["x"], s["weight"], s["teacher_index"],
                                 s["teacher_logits"], s["lse"], temperature=case["temperature"])


def work(case):
    """Inputs read once, outputs written once; of the arithmetic, the matrix products."""
    n, k, op = case["rows"], case["inner"], case["op"]
    if op.startswith("linear"):
        m = case["cols"]
        few = m if case["bias"] else 0
        if op == "linear":
            return {"bytes": 2 * (n * k + m * k + few + n * m * (2 if case["residual"] else 1)), "flops": 2 * n * m * k}
        products = 2 if case["act"] == "none" else 3
        return {"bytes": 2 * (n * m + 2 * n * k + 2 * m * k + 2 * few), "flops": 2 * products * n * m * k}
    v = case["vocab"]
    few = n * (8 if op.startswith("ce") else 12 * case["top"])
    if not op.endswith("bwd"):
        return {"bytes": 2 * (n * k + v * k) + few + 8 * n, "flops": 2 * n * v * k}
    return {"bytes": 4 * (n * k + v * k) + few + 12 * n, "flops": 6 * n * v * k}


# ------------------------------------------------------------------ exact results
def exact(case, seed):
    """The forwards in fp64, and the backwards by differentiating them there."""
    s = prepare(case, seed)
    backward = case["op"].endswith("bwd")
    with torch.set_grad_enabled(backward):
        x, w = s["x"].double().requires_grad_(backward), s["weight"].double().requires_grad_(backward)
        z = torch.einsum("nk,mk->nm", x, w)
        if case["op"].startswith("linear"):
            b = s["bias"].double().requires_grad_(backward) if case["bias"] else None
            z = z if b is None else b + z
            act = case["act"]
            if act == "relu":
                y = z.clamp(min=0)
            elif act == "gelu":  # z times the normal distribution's function
                y = z * torch.erfc(z / -math.sqrt(2.0)) / 2
            elif act == "gelu_tanh":  # (1 + tanh u) / 2 is the logistic function of 2 u
                y = z * torch.sigmoid(math.sqrt(8 / math.pi) * (z + 0.044715 * z.pow(3)))
            else:
                y = z * torch.sigmoid(z) if act == "silu" else z
            if not backward:
                return y if s["residual"] is None else s["residual"].double() + y
            grads = torch.autograd.grad(y, [x, w] + ([b] if b is not None else []), s["dout"].double())
            return grads[0], grads[1], grads[2] if b is not None else None
        logp = torch.log_softmax(z / case["temperature"], dim=1)
        lse = (z / case["temperature"])[:, 0] - logp[:, 0]
        if case["op"].startswith("ce"):
            counted = s["target"] != IGNORED
            rows = torch.arange(case["rows"], device=z.device)
            loss = -logp[rows, torch.where(counted, s["target"], 0)]
        else:
            counted = (s["teacher_index"] >= 0).any(1)
            teacher = torch.log_softmax(s["teacher_logits"].double() / case["temperature"], dim=1)
            student = logp.gather(1, s["teacher_index"].clamp(min=0))
            loss = (teacher.exp() * (teacher - student)).sum(1)
        loss = torch.where(counted, loss, torch.zeros_like(loss))
        if not backward:
            return loss, lse
        total = (loss * s["dloss"].double()).sum() + (lse * s["dlse"].double()).sum()
        return torch.autograd.grad(total, [x, w])
