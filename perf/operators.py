"""Cases, plain forms and exact results of the training and rotary operators.

  dropout         dropout_fwd, dropout_add_fwd: dropout whose mask is a function of (seed, offset, row,
                  column) and is never stored, with the residual add
  dropout_norm    dropout_add_rmsnorm_fwd and _bwd: dropout + residual add + RMSNorm, and its gradients
  rope            rope_fwd and _bwd: rotary positions of q and k
  norm_rope       qk_rmsnorm_rope_fwd and _bwd: per-head RMSNorm and rotary positions of q and k

With `own` false, run() is the plain form: elementary torch operations in fp32 (angles in fp64).  With
`own` true it calls the framework.  exact() gives the same results from the definitions in fp64.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
EPS = 1e-6
OFFSET = 11


def _rows(name, op, dtype, rows, hidden, p):
    return {"name": name, "op": op, "dtype": dtype, "rows": rows, "hidden": hidden, "p": p}


def _heads(name, op, dtype, batch, seq, q_heads, k_heads, dim, rot, interleaved, start, factor):
    return {"name": name, "op": op, "dtype": dtype, "batch": batch, "seq": seq, "q_heads": q_heads,
            "k_heads": k_heads, "dim": dim, "rot": rot, "interleaved": interleaved, "start": start,
            "factor": factor}


def listed():
    return [
        # dropout of a training step's embeddings: 8192 tokens
        _rows("dropout_8192x4096_bf16", "dropout", "bf16", 8192, 4096, 0.1),
        # the same with the residual add, on rows that no vector width divides
        _rows("dropout_add_777x1001_fp16", "dropout_add", "fp16", 777, 1001, 0.25),
        # the framework's smallest workload: a few tokens, where the call's latency counts
        _rows("dropout_norm_64x1024_bf16", "dropout_norm", "bf16", 64, 1024, 0.1),
        # a training step's branch output, residual and norm at the framework's largest single-tile row
        _rows("dropout_norm_4096x8192_bf16", "dropout_norm", "bf16", 4096, 8192, 0.1),
        # its gradients in fp32, as a user checking a run trains; a width between powers of two
        _rows("dropout_norm_bwd_1999x5120_fp32", "dropout_norm_bwd", "fp32", 1999, 5120, 0.2),
        # its gradients for 8192 tokens
        _rows("dropout_norm_bwd_8192x8192_bf16", "dropout_norm_bwd", "bf16", 8192, 8192, 0.1),
        # serving: one token of each of 64 sequences, far positions, part of the head, neighbouring pairs
        _heads("rope_decode64_fp16", "rope", "fp16", 64, 1, 32, 8, 128, 64, True, 131000, 1.0),
        # a prompt batch: 4096 tokens, halves layout, whole heads, stretched context
        _heads("rope_prefill4096_bf16", "rope", "bf16", 2, 2048, 32, 8, 128, 128, False, 0, 4.0),
        # its gradient with fp32 tensors and an odd number of tokens, heads of 96
        _heads("rope_bwd_1533_fp32", "rope_bwd", "fp32", 3, 511, 16, 16, 96, 96, False, 0, 1.0),
        # serving: one token of each of 8 sequences, norm and rotation of 32 + 8 heads
        _heads("norm_rope_decode8_bf16", "norm_rope", "bf16", 8, 1, 32, 8, 128, 128, False, 30000, 1.0),
        # a prompt of 8192 tokens
        _heads("norm_rope_prefill8192_bf16", "norm_rope", "bf16", 1, 8192, 32, 8, 128, 128, False, 0, 1.0),
        # training: gradients of q, k and both weights for 4096 tokens
        _heads("norm_rope_bwd_4096_bf16", "norm_rope_bwd", "bf16", 2, 2048, 32, 8, 128, 128, False, 0, 1.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["dropout", "dropout_add", "dropout_norm", "dropout_norm", "dropout_norm_bwd",
                     "dropout_norm_bwd", "rope", "rope_bwd", "norm_rope", "norm_rope", "norm_rope_bwd",
                     "norm_rope_bwd"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    case = {"op": op, "dtype": dtype}
    if op.startswith("dropout"):
        hidden = _log(rng, 64, 16384)
        if op in ("dropout_norm", "dropout_norm_bwd"):
            hidden = max(64, hidden // 8 * 8)  # rows of whole 8-element blocks
        most = 8192 * 8192 // (2 if dtype == "fp32" else 1)
        rows = _log(rng, 1, min(16384, most // hidden))
        return case | {"rows": rows, "hidden": hidden, "p": rng.choice([0.0, 0.05, 0.1, 0.2, 0.5])}
    dim = rng.choice([32, 64, 80, 96, 128, 128, 192, 256])
    rot = rng.choice([dim, dim, dim // 2, dim // 4])
    rot -= rot % 2
    k_heads = rng.choice([1, 2, 4, 8, 8])
    q_heads = k_heads * rng.choice([1, 2, 4, 7])
    most = 8192 * 40 * 128 // ((q_heads + k_heads) * dim * (2 if dtype == "fp32" else 1))
    if rng.random() < 0.4:  # serving: one token a sequence
        batch, seq, start = _log(rng, 1, min(512, most)), 1, _log(rng, 1, 1 << 20)
    else:
        batch = rng.choice([1, 1, 2, 3])
        seq, start = _log(rng, 2, max(2, min(16384, most // batch))), rng.choice([0, 0, 100000])
    return case | {"batch": batch, "seq": seq, "q_heads": q_heads, "k_heads": k_heads, "dim": dim, "rot": rot,
                   "interleaved": rng.random() < 0.4, "start": start, "factor": rng.choice([1.0, 1.0, 4.0, 16.0])}


def _inv_freq(rot, factor):
    """Radians per position; a factor > 1 stretches the context by enlarging the base."""
    base = 10000.0 * (factor ** (rot / (rot - 2)) if factor != 1.0 and rot > 2 else 1.0)
    return base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, std=1.0, mean=0.0):
        t = torch.randn(shape, generator=g, device=dev, dtype=torch.float32)
        return t.mul_(std).add_(mean).to(dt)

    s = {"case": case, "seed": 0x9E3779B97F4A7C15 * (seed + 1) % (1 << 63), "p": case.get("p", 0.0)}
    if case["op"].startswith("dropout"):
        n, h = case["rows"], case["hidden"]
        s["x"] = normal(n, h)
        if case["op"] in ("dropout_add", "dropout_norm"):
            s["residual"] = normal(n, h, std=2.0)
        if case["op"].startswith("dropout_norm"):
            s["weight"] = normal(h, std=0.1, mean=1.0)
        if case["op"] == "dropout_norm_bwd":
            s["h"] = s.pop("x").mul_(2.0)  # the forward's residual_out
            s["dout"] = normal(n, h)
            s["dres"] = normal(n, h)
        return s
    b, n, hq, hk, d = (case[k] for k in ("batch", "seq", "q_heads", "k_heads", "dim"))
    # q and k lie in one projection's output, beside v, as a fused projection leaves them
    packed = normal(b, n, hq + 2 * hk, d)
    s["q"], s["k"] = packed[:, :, :hq], packed[:, :, hq:hq + hk]
    start = torch.full((b, 1), case["start"], device=dev, dtype=torch.int64)
    if n == 1:  # every sequence at a position of its own
        start += torch.randint(0, 4096, (b, 1), generator=g, device=dev)
    s["positions"] = start + torch.arange(n, device=dev)
    s["inv_freq"] = _inv_freq(case["rot"], case["factor"]).to(dev)
    s["scale"] = 0.1 * math.log(case["factor"]) + 1.0
    if case["op"].startswith("norm"):
        s["q_weight"], s["k_weight"] = normal(d, std=0.1, mean=1.0), normal(d, std=0.1, mean=1.0)
    if case["op"] == "norm_rope_bwd":
        s["dq"], s["dk"] = normal(b, n, hq, d), normal(b, n, hk, d)
    return s


# ------------------------------------------------------------------ plain forms
def _drop_numbers(p):
    """The 16-bit threshold below which an element is dropped, and the factor of the others."""
    t = round(float(np.float32(p)) * 65536)
    return t, float(np.float32(65536.0 / (65536 - t))) if t < 65536 else 0.0


def _keep(seed, rows, hidden, p, device):
    """The mask: 16 bits an element from Philox4x32 with 7 rounds (Salmon, Moraes, Dror and Shaw, 2011),
    one counter for 8 neighbouring columns of a row."""
    m32 = 0xFFFFFFFF
    blocks = (hidden + 7) // 8
    c0 = torch.arange(blocks, device=device, dtype=torch.int64).expand(rows, blocks)
    c1 = torch.arange(rows, device=device, dtype=torch.int64)[:, None].expand(rows, blocks)
    c2 = torch.full_like(c0, OFFSET & m32)
    c3 = torch.full_like(c0, OFFSET >> 32)
    k0, k1 = seed & m32, seed >> 32
    for _ in range(7):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57  # modulo 2^64; the high words are masked below
        c0, c1, c2, c3 = ((b >> 32) & m32) ^ c1 ^ k0, b & m32, ((a >> 32) & m32) ^ c3 ^ k1, a & m32
        k0, k1 = (k0 + 0x9E3779B9) & m32, (k1 + 0xBB67AE85) & m32
    half = torch.stack([c0 & 0xFFFF, c0 >> 16, c1 & 0xFFFF, c1 >> 16, c2 & 0xFFFF, c2 >> 16, c3 & 0xFFFF, c3 >> 16],
                       dim=-1).reshape(rows, blocks * 8)[:, :hidden]
    return half >= _drop_numbers(p)[0]


def _dropped(v, s, rows, hidden):
    keep = _keep(s["seed"], rows, hidden, s["p"], v.device)
    return torch.where(keep, v * _drop_numbers(s["p"])[1], 0.0)


def _rotate(x, s, case, sign):
    """x: fp32 [b, s, heads, dim]."""
    ang = s["positions"].double()[:, :, None, None] * s["inv_freq"]
    c, sn = ang.cos().float() * s["scale"], ang.sin().float() * (sign * s["scale"])
    rot = case["rot"]
    if case["interleaved"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([a * c - b * sn, a * sn + b * c], dim=-1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat([a * c - b * sn, a * sn + b * c], dim=-1)
    return torch.cat([y, x[..., rot:]], dim=-1)


def _plain(s):
    case = s["case"]
    op, dt = case["op"], DTYPES[case["dtype"]]
    if op in ("dropout", "dropout_add", "dropout_norm"):
        acc = _dropped(s["x"].float(), s, *s["x"].shape)
        if op == "dropout":
            return acc.to(dt)
        acc = acc + s["residual"].float()
        if op == "dropout_add":
            return acc.to(dt)
        inv = 1.0 / torch.sqrt(acc.square().mean(-1, keepdim=True) + EPS)
        return (acc * inv * s["weight"].float()).to(dt), acc.to(dt)
    if op == "dropout_norm_bwd":
        h, dout = s["h"].float(), s["dout"].float()
        inv = 1.0 / torch.sqrt(h.square().mean(-1, keepdim=True) + EPS)
        xh, g = h * inv, dout * s["weight"].float()
        d = s["dres"].float() + inv * (g - xh * (g * xh).mean(-1, keepdim=True))
        return _dropped(d, s, *d.shape).to(dt), d.to(dt), (dout * xh).sum(0)
    if op == "rope":
        return [_rotate(s[n].float(), s, case, 1.0).to(dt) for n in ("q", "k")]
    if op == "rope_bwd":
        return [_rotate(s[n].float(), s, case, -1.0).to(dt) for n in ("q", "k")]
    grads, sums = [], []
    for n in ("q", "k"):
        x, w = s[n].float(), s[n + "_weight"].float()
        inv = 1.0 / torch.sqrt(x.square().mean(-1, keepdim=True) + EPS)
        if op == "norm_rope":
            grads.append(_rotate(x * inv * w, s, case, 1.0).to(dt))
            continue
        g = _rotate(s["d" + n].float(), s, case, -1.0)
        xh, gw = x * inv, g * w
        grads.append((inv * (gw - xh * (gw * xh).mean(-1, keepdim=True))).to(dt))
        sums.append((g * xh).sum((0, 1, 2)))
    return grads + sums


def run(s):
    if not own:
        return _plain(s)
    import deterministic_residual_add_gb300 as dr

    case, op = s["case"], s["case"]["op"]
    if op.startswith("dropout"):
        rng = {"seed": s["seed"], "offset": OFFSET}
        if op == "dropout":
            return dr.dropout_fwd(s["x"], s["p"], **rng)
        if op == "dropout_add":
            return dr.dropout_add_fwd(s["x"], s["residual"], s["p"], **rng)
        if op == "dropout_norm":
            return dr.dropout_add_rmsnorm_fwd(s["x"], s["residual"], s["weight"], s["p"], EPS, **rng)
        return dr.dropout_add_rmsnorm_bwd(s["dout"], s["dres"], s["h"], s["weight"], s["p"], EPS, **rng)
    how = {"positions": s["positions"], "interleaved": case["interleaved"], "scale": s["scale"]}
    if op == "rope":
        return dr.rope_fwd(s["q"], s["k"], s["inv_freq"], **how)
    if op == "rope_bwd":
        return dr.rope_bwd(s["q"], s["k"], s["inv_freq"], **how)
    if op == "norm_rope":
        return dr.qk_rmsnorm_rope_fwd(s["q"], s["k"], s["q_weight"], s["k_weight"], s["inv_freq"], EPS, EPS, **how)
    return dr.qk_rmsnorm_rope_bwd(s["dq"], s["dk"], s["q"], s["k"], s["q_weight"], s["k_weight"], s["inv_freq"],
                                  EPS, EPS, **how)


def work(case):
    """Inputs read once and outputs written once; the generator's integer steps are not counted as flops."""
    size, op = BYTES[case["dtype"]], case["op"]
    if op.startswith("dropout"):
        h = case["hidden"]
        n = case["rows"] * h
        if op == "dropout":
            return {"bytes": 2 * n * size, "flops": n}
        if op == "dropout_add":
            return {"bytes": 3 * n * size, "flops": 2 * n}
        if op == "dropout_norm":
            return {"bytes": (4 * n + h) * size, "flops": 6 * n}
        return {"bytes": (5 * n + h) * size + 4 * h, "flops": 15 * n}
    tokens = case["batch"] * case["seq"]
    n = tokens * (case["q_heads"] + case["k_heads"]) * case["dim"]
    turned = 3 * (n // case["dim"]) * case["rot"]
    extra = 8 * tokens + 4 * case["rot"]
    if op in ("rope", "rope_bwd"):
        return {"bytes": 2 * n * size + extra, "flops": turned}
    extra += 2 * case["dim"] * size
    if op == "norm_rope":
        return {"bytes": 2 * n * size + extra, "flops": turned + 4 * n}
    return {"bytes": 3 * n * size + extra + 8 * case["dim"], "flops": turned + 12 * n}


# ------------------------------------------------------------------ exact results
def _kept64(s, rows, hidden):
    """The factor of every element, in fp64, from the generator in numpy's unsigned integers."""
    p = float(np.float32(s["p"]))
    limit = int(np.rint(p * 65536))
    col, row = np.meshgrid(np.arange(-(-hidden // 8), dtype=np.uint64), np.arange(rows, dtype=np.uint64))
    low, shift = np.uint64(0xFFFFFFFF), np.uint64(32)
    x = [col, row, np.uint64(OFFSET % (1 << 32)), np.uint64(OFFSET >> 32)]
    key = [s["seed"] % (1 << 32), s["seed"] >> 32]
    for i in range(7):
        left, right = x[0] * np.uint64(0xD2511F53), x[2] * np.uint64(0xCD9E8D57)
        ka = np.uint64((key[0] + i * 0x9E3779B9) % (1 << 32))
        kb = np.uint64((key[1] + i * 0xBB67AE85) % (1 << 32))
        x = [(right >> shift) ^ x[1] ^ ka, right & low, (left >> shift) ^ x[3] ^ kb, left & low]
    words = np.stack([np.broadcast_to(w, col.shape).astype("<u4") for w in x], axis=-1)
    bits = np.ascontiguousarray(words).view("<u2").reshape(rows, -1)[:, :hidden]
    keep = torch.from_numpy(bits >= limit).to("cuda")
    return keep.double() * (65536 / (65536 - limit) if limit < 65536 else 0.0)


def _turned64(x, s, case):
    """The rotation as a product of complex numbers."""
    rot = case["rot"]
    turn = torch.polar(torch.tensor(s["scale"], dtype=torch.float64, device=x.device).expand(1),
                       torch.zeros(1, dtype=torch.float64, device=x.device))
    ang = s["positions"].double().unsqueeze(-1) * s["inv_freq"]
    turn = turn * torch.polar(torch.ones_like(ang), ang).unsqueeze(2)
    head = x[..., :rot]
    if case["interleaved"]:
        z = torch.view_as_complex(head.unflatten(-1, (rot // 2, 2)).contiguous()) * turn
        head = torch.view_as_real(z).flatten(-2)
    else:
        z = torch.complex(*head.unflatten(-1, (2, rot // 2)).unbind(-2)) * turn
        head = torch.cat([z.real, z.imag], dim=-1)
    return torch.cat([head, x[..., rot:]], dim=-1)


def _normed64(x, w):
    return x * (x.pow(2).mean(-1, keepdim=True) + EPS).rsqrt() * w


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]

    def leaf(name):
        return s[name].double().requires_grad_(op.endswith("_bwd"))

    if op in ("dropout", "dropout_add", "dropout_norm"):
        acc = s["x"].double() * _kept64(s, *s["x"].shape)
        if op == "dropout":
            return acc
        acc = acc + s["residual"].double()
        return acc if op == "dropout_add" else (_normed64(acc, s["weight"].double()), acc)
    if op == "dropout_norm_bwd":
        h, w = leaf("h"), leaf("weight")
        dh, dw = torch.autograd.grad([_normed64(h, w), h * 1.0], [h, w], [s["dout"].double(), s["dres"].double()])
        return dh * _kept64(s, *h.shape), dh, dw
    if op == "rope":
        return [_turned64(s[n].double(), s, case) for n in ("q", "k")]
    if op == "rope_bwd":
        xs = [torch.zeros_like(s[n], dtype=torch.float64, requires_grad=True) for n in ("q", "k")]
        return list(torch.autograd.grad([_turned64(x, s, case) for x in xs], xs, [s[n].double() for n in ("q", "k")]))
    xs, ws = [leaf(n) for n in ("q", "k")], [leaf(n + "_weight") for n in ("q", "k")]
    ys = [_turned64(_normed64(x, w), s, case) for x, w in zip(xs, ws)]
    if op == "norm_rope":
        return ys
    return list(torch.autograd.grad(ys, xs + ws, [s["dq"].double(), s["dk"].double()]))
