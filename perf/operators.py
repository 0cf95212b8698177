"""The training operators of the output head, case by case: how their inputs are made, their plain form in
elementary torch operations, the calls of this package, their definition in 64 bits and the work of one pass.

Three operators, in the order in which a training step of the head meets them:

* ``residual_norm``: the end of a block. With h the residual stream, y the block's output and
  n(x; w) = w x / sqrt(mean(x^2) + eps):  h' = scale h + gate n(y; post),  x = n(h'; pre).
* ``cross_entropy``: z = H W^T, per row loss = lse(z) - z_target + z_loss lse(z)^2, and the gradients of the
  (mean, summed or weighted) loss in H and W. Rows whose target is the ignored index have no loss and no gradient.
* ``adamw``: one step over many tensors, with both moments in 32 bits or in 8 bits (blocks of 256 values that
  share a scale; the second moment is held as its root).
"""
import math
import random

import torch

own = False  # true: run() makes the package's calls; false: the plain forms

BF, F32, F64, F8 = torch.bfloat16, torch.float32, torch.float64, torch.float8_e4m3fn
IGNORE = -100
BLOCK, TOP = 256, 448.0  # values that share a scale in the 8-bit states, and the largest value of their type


def listed():
    return [
        # the smallest training step: the repository's tiny workload
        {"name": "loss step tiny", "op": "loss", "M": 4, "d": 256, "V": 4096, "grad": True, "reduction": "mean", "z_loss": 0.0},
        # evaluation loss of one small batch on the decode shape: forward only
        {"name": "loss eval 16", "op": "loss", "M": 16, "d": 5120, "V": 151936, "grad": False, "reduction": "mean", "z_loss": 0.0},
        # a short sequence: few rows against the whole head, both gradients
        {"name": "loss step 64", "op": "loss", "M": 64, "d": 4096, "V": 151936, "grad": True, "reduction": "mean", "z_loss": 1e-4},
        # a ragged batch with ignored rows and a weight for each row's loss, odd sizes
        {"name": "loss step ragged 509", "op": "loss", "M": 509, "d": 2056, "V": 50257, "grad": True, "reduction": "none", "z_loss": 1e-4},
        # a full training batch on the prefill shape
        {"name": "loss step 4096", "op": "loss", "M": 4096, "d": 6144, "V": 200064, "grad": True, "reduction": "mean", "z_loss": 0.0},
        # decoding: a few rows, latency
        {"name": "norm forward 16", "op": "norm", "M": 16, "d": 5120, "grad": False, "stream": "bf16", "weights": "bf16", "post": True, "gate": "channel", "scale": 1.0},
        # a ragged batch on a 32-bit residual stream with a gate for each token and channel
        {"name": "norm backward ragged 1021", "op": "norm", "M": 1021, "d": 4100, "grad": True, "stream": "fp32", "weights": "fp32", "post": True, "gate": "token", "scale": 0.5},
        # training batches, forward and backward
        {"name": "norm forward 8192", "op": "norm", "M": 8192, "d": 6144, "grad": False, "stream": "bf16", "weights": "bf16", "post": True, "gate": "channel", "scale": 1.0},
        {"name": "norm backward 8192", "op": "norm", "M": 8192, "d": 6144, "grad": True, "stream": "bf16", "weights": "bf16", "post": True, "gate": "channel", "scale": 1.0},
        # many small tensors (an adapter): the cost of a call
        {"name": "adamw many small", "op": "adamw", "vectors": 96, "dim": 250, "matrices": 32, "rows": 17, "params": "fp32", "bits": 32},
        # the decode shape's head and its norms: bf16 weights with 32-bit copies, 32-bit states
        {"name": "adamw head 32", "op": "adamw", "vectors": 3, "dim": 4096, "matrices": 1, "rows": 151936, "params": "bf16", "bits": 32},
        # the same kind of head with 8-bit states
        {"name": "adamw head 8", "op": "adamw", "vectors": 3, "dim": 5120, "matrices": 1, "rows": 151936, "params": "bf16", "bits": 8},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["loss", "loss", "norm", "adamw"])
    if op == "loss":
        # one token to a full batch; hidden sizes are multiples of 8 as the head asks, few of them of 64; vocabularies any size
        return {"op": op, "M": _log(rng, 1, 4096), "d": 40 * _log(rng, 2, 153), "V": _log(rng, 1000, 200064), "grad": rng.random() < 0.75,
                "reduction": rng.choice(["mean", "sum", "none"]), "z_loss": rng.choice([0.0, 1e-4])}
    if op == "norm":
        return {"op": op, "M": _log(rng, 1, 8192), "d": _log(rng, 64, 6144), "grad": rng.random() < 0.5, "stream": rng.choice(["bf16", "fp32"]),
                "weights": rng.choice(["bf16", "fp32"]), "post": rng.random() < 0.75, "gate": rng.choice(["none", "channel", "token"]),
                "scale": rng.choice([1.0, 0.5])}
    dim = _log(rng, 64, 5120)
    return {"op": op, "vectors": _log(rng, 1, 128), "dim": dim, "matrices": _log(rng, 1, 32), "rows": _log(rng, 16, max(17, 16_000_000 // dim)),
            "params": rng.choice(["bf16", "fp32"]), "bits": rng.choice([32, 8])}


# ---------------------------------------------------------------------------------- inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return {"loss": _loss_inputs, "norm": _norm_inputs, "adamw": _adamw_inputs}[case["op"]](case, g)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _loss_inputs(c, g):
    M, d, V = c["M"], c["d"], c["V"]
    W = torch.empty(V, d, dtype=BF, device="cuda")
    for r in range(0, V, 16384):
        n = min(16384, V - r)
        W[r:r + n] = _randn(g, n, d) * d ** -0.5
    t = torch.randint(0, V, (M,), generator=g, device="cuda", dtype=torch.int32)
    # logits on a unit scale; a trained head favours the target by a little for some tokens, by a lot for others
    lift = 9 * torch.rand(M, generator=g, device="cuda")
    H = (_randn(g, M, d) + lift[:, None] * W[t.long()].float()).to(BF)
    if M > 8:  # padding and prompt tokens carry no loss
        t[torch.rand(M, generator=g, device="cuda") < 0.1] = IGNORE
        t[-1] = IGNORE
    s = {"c": c, "H": H, "W": W, "targets": t, "grad": None}
    if c["grad"] and c["reduction"] == "none":  # the weight of each row's loss
        s["grad"] = torch.rand(M, generator=g, device="cuda") / M
    return s


def _norm_inputs(c, g):
    M, d = c["M"], c["d"]
    st, wt = {"bf16": BF, "fp32": F32}[c["stream"]], {"bf16": BF, "fp32": F32}[c["weights"]]
    s = {"c": c, "h": (3 * _randn(g, M, d)).to(st), "y": (0.5 * _randn(g, M, d)).to(BF), "pre": (1 + 0.1 * _randn(g, d)).to(wt), "post": None, "gate": None}
    if c["post"]:
        s["post"] = (1 + 0.1 * _randn(g, d)).to(wt)
    if c["gate"] != "none":
        s["gate"] = (0.5 + 0.1 * _randn(g, d)).to(wt) if c["gate"] == "channel" else (0.5 + 0.1 * _randn(g, M, d)).to(BF)
    if c["grad"]:  # backward: h is then the stream h' that forward left, with the gradients of both outputs
        s["dx"], s["dh"] = (0.01 * _randn(g, M, d)).to(BF), (0.01 * _randn(g, M, d)).to(st)
    return s


def _sizes(c):
    """The tensors' sizes: norm and gate vectors, and matrices; in between one size that no vector width divides."""
    return [c["dim"]] * c["vectors"] + [c["dim"] * c["rows"] + (i % 2) for i in range(c["matrices"])]


def _quantise(x):
    """8-bit codes and scales of x (a multiple of BLOCK values), and zeros where a block's largest value is below 2^-100."""
    b = x.view(-1, BLOCK)
    top = b.abs().amax(1)
    small = top < 2.0 ** -100
    mul = torch.where(small, 0.0, TOP / torch.where(small, 1.0, top))
    return b * mul[:, None], torch.where(small, 0.0, top * (1 / TOP))


def _adamw_inputs(c, g):
    sizes = _sizes(c)
    at, n = [], 0
    for k in sizes:  # every tensor starts at a block of its own in the flat buffers
        at.append(n)
        n += -(-k // BLOCK) * BLOCK
    real = torch.zeros(n, dtype=torch.bool, device="cuda")
    for o, k in zip(at, sizes):
        real[o:o + k] = True
    w = _randn(g, n).mul_(0.02).masked_fill_(~real, 0)
    s = {"c": c, "t": 100, "lr": 1e-3, "b1": 0.9, "b2": 0.95, "eps": 1e-8, "wd": 0.1, "grad_scale": torch.full((1,), 0.75, device="cuda")}
    s["grad"] = _randn(g, n).mul_(1e-3).masked_fill_(~real, 0)
    m, r = _randn(g, n).mul_(1e-3).masked_fill_(~real, 0), _randn(g, n).abs_().mul_(1e-3).masked_fill_(~real, 0)
    if c["params"] == "bf16":
        s["master"], s["p"], s["grad"] = w, w.to(BF), s["grad"].to(BF)
    else:
        s["master"], s["p"] = None, w
    if c["bits"] == 8:
        (m, s["ms"]), (r, s["rs"]) = _quantise(m), _quantise(r)
        s["m"], s["r"] = m.reshape(-1).to(F8), r.reshape(-1).to(F8)
    else:
        s["m"], s["v"] = m, r.mul_(r)
    del w, m, r, real
    if own:  # the handle that a training program keeps: it holds the tensors' addresses and sizes
        import gemm_epilogue_reduction_gb300 as sb

        def views(t, per=1):
            return None if t is None else [t[o // per:o // per + -(-k // per)] for o, k in zip(at, sizes)]

        state = [views(s["m"]), views(s["r"] if c["bits"] == 8 else s["v"])]
        if c["bits"] == 8:
            state += [views(s["ms"], BLOCK), views(s["rs"], BLOCK)]
        s["opt"] = sb.AdamW(views(s["p"]), views(s["grad"]), masters=views(s["master"]), states=list(zip(*state)), lr=s["lr"], betas=(s["b1"], s["b2"]),
                            eps=s["eps"], weight_decay=s["wd"], state_bits=c["bits"], step=s["t"])
    return s


# ---------------------------------------------------------------------------------- one pass
def run(s):
    return {"loss": _loss, "norm": _norm, "adamw": _adamw}[s["c"]["op"]](s)


def _loss(s):
    c, H, W, t = s["c"], s["H"], s["W"], s["targets"]
    zl = c["z_loss"]
    if own:
        import gemm_epilogue_reduction_gb300 as sb
        f = sb.cross_entropy(H, W, t, ignore_index=IGNORE, z_loss=zl, reduction=c["reduction"])
        if not c["grad"]:
            return {"loss": f["loss"], "lse": f["lse"]}
        b = sb.cross_entropy_backward(H, W, t, f["lse"], grad=s["grad"], ignore_index=IGNORE, z_loss=zl, reduction=c["reduction"])
        return {"loss": f["loss"], "lse": f["lse"], "dH": b["dH"], "dW": b["dW"]}
    Hf, Wf = H.float(), W.float()
    z = Hf @ Wf.t()
    top = z.amax(1, keepdim=True)
    lse = top[:, 0] + (z - top).exp().sum(1).log()
    valid = t != IGNORE
    at = torch.where(valid, t, 0).long()[:, None]
    rows = torch.where(valid, lse - z.gather(1, at)[:, 0] + zl * lse * lse, 0.0)
    count = valid.sum().clamp(min=1)
    loss = {"mean": lambda: rows.sum() / count, "sum": lambda: rows.sum(), "none": lambda: rows}[c["reduction"]]()
    out = {"loss": loss.reshape(-1), "lse": lse}
    if c["grad"]:
        g = valid.float()
        if c["reduction"] == "mean":
            g = g / count
        elif c["reduction"] == "none":
            g = g * s["grad"]
        G = (z - lse[:, None]).exp() * (g * (1 + 2 * zl * lse))[:, None]
        G.scatter_add_(1, at, -g[:, None])
        out["dH"], out["dW"] = (G @ Wf).to(BF), (G.t() @ Hf).to(BF)
    return out


def _norm(s, eps=1e-6):
    c, post, gate, pre, scale = s["c"], s["post"], s["gate"], s["pre"], s["c"]["scale"]
    if own:
        import gemm_epilogue_reduction_gb300 as sb
        if c["grad"]:
            b = sb.residual_norm_backward(s["dx"], s["dh"], s["h"], s["y"], pre, post=post, gate=gate, scale=scale, eps=eps)
            return {k: b[k] for k in ("dh", "dy", "dpre", "dpost", "dgate") if b[k] is not None}
        f = sb.residual_norm(s["h"], s["y"], pre, post=post, gate=gate, scale=scale, eps=eps)
        return {"h": f["h"], "x": f["x"]}
    h, y, wpre = s["h"].float(), s["y"].float(), pre.float()
    ry = (y.square().mean(1, keepdim=True) + eps).rsqrt() if c["post"] else None
    u = y * ry * post.float() if c["post"] else y
    gf = gate.float() if gate is not None else None
    if not c["grad"]:
        h = h * scale + (u * gf if gate is not None else u)
        x = h * (h.square().mean(1, keepdim=True) + eps).rsqrt() * wpre
        return {"h": h.to(s["h"].dtype), "x": x.to(BF)}
    dx, rh = s["dx"].float(), (h.square().mean(1, keepdim=True) + eps).rsqrt()
    e = dx * wpre
    dh = s["dh"].float() + rh * (e - h * (rh * rh) * (e * h).mean(1, keepdim=True))
    out = {"dpre": (dx * h * rh).sum(0).to(pre.dtype), "dh": (dh * scale).to(s["h"].dtype)}
    if gate is not None:
        out["dgate"] = (dh * u).sum(0).to(gate.dtype) if c["gate"] == "channel" else (dh * u).to(BF)
        dh = dh * gf
    if c["post"]:
        out["dpost"] = (dh * y * ry).sum(0).to(post.dtype)
        dh = dh * post.float()
        dh = ry * (dh - y * (ry * ry) * (dh * y).mean(1, keepdim=True))
    out["dy"] = dh.to(BF)
    return out


def _adamw(s):
    c = s["c"]
    names = ["p", "master", "m"] + (["r", "ms", "rs"] if c["bits"] == 8 else ["v"])
    if own:
        s["opt"].step(grad_scale=s["grad_scale"])
        return {k: s[k] for k in names if s[k] is not None}
    s["t"] += 1
    b1, b2 = s["b1"], s["b2"]
    w = s["p"] if s["master"] is None else s["master"]
    g = s["grad"].float() * s["grad_scale"]
    if c["bits"] == 8:
        m, r = (s[a].float().view(-1, BLOCK) * s[b][:, None] for a, b in (("m", "ms"), ("r", "rs")))
        m, v = m.view(-1), r.view(-1).square()
    else:
        m, v = s["m"], s["v"]
    m = m * b1 + g * (1 - b1)
    v = v * b2 + g * g * (1 - b2)
    root = v.sqrt()
    step = m / (root * (1 / math.sqrt(1 - b2 ** s["t"])) + s["eps"])
    w.mul_(1 - s["lr"] * s["wd"]).sub_(step * (s["lr"] / (1 - b1 ** s["t"])))
    if s["master"] is not None:
        s["p"].copy_(w)
    if c["bits"] == 8:
        q, scale = _quantise(m)
        s["m"].copy_(q.view(-1)), s["ms"].copy_(scale)
        q, scale = _quantise(root)
        q = torch.where((q > 0) & (q < 2.0 ** -9), 2.0 ** -9, q)  # a root that is there stays there
        s["r"].copy_(q.view(-1)), s["rs"].copy_(scale)
    else:
        s["m"].copy_(m), s["v"].copy_(v)
    return {k: s[k] for k in names if s[k] is not None}


# ---------------------------------------------------------------------------------- definition in 64 bits
def exact(case, seed):
    if case["op"] == "loss" and 6.0 * case["M"] * case["d"] * case["V"] > 8e12:
        return None
    s = prepare(case, seed)
    return {"loss": _loss_exact, "norm": _norm_exact, "adamw": _adamw_exact}[case["op"]](case, s)


def _loss_exact(c, s):
    H, W, t, V, zl = s["H"].to(F64), s["W"], s["targets"].long(), c["V"], c["z_loss"]
    M, step = c["M"], 8192
    lse, target = torch.full((M,), -math.inf, dtype=F64, device="cuda"), torch.zeros(M, dtype=F64, device="cuda")
    for a in range(0, V, step):
        z = H @ W[a:a + step].to(F64).T
        lse = torch.logaddexp(lse, torch.logsumexp(z, 1))
        here = (t >= a) & (t < a + z.shape[1])
        target[here] = z[here, t[here] - a]
    has = t != IGNORE
    loss = torch.where(has, lse - target + zl * lse ** 2, torch.zeros_like(lse))
    weight = has.to(F64)
    total = int(has.sum())
    if c["reduction"] == "mean":
        weight = weight / max(total, 1)
    elif c["reduction"] == "none" and s["grad"] is not None:
        weight = weight * s["grad"].to(F64)
    value = loss if c["reduction"] == "none" else loss.sum().reshape(1) / (max(total, 1) if c["reduction"] == "mean" else 1)
    out = {"loss": value, "lse": lse}
    if c["grad"]:
        dH, dW = torch.zeros_like(H), torch.empty(V, c["d"], dtype=F64, device="cuda")
        for a in range(0, V, step):
            w = W[a:a + step].to(F64)
            p = torch.exp(H @ w.T - lse[:, None])
            p *= (1 + 2 * zl * lse)[:, None]
            here = torch.nonzero((t >= a) & (t < a + w.shape[0]))[:, 0]
            p[here, t[here] - a] -= 1
            p *= weight[:, None]
            dH += p @ w
            dW[a:a + step] = p.T @ H
        out["dH"], out["dW"] = dH, dW
    return out


def _norm_exact(c, s, eps=1e-6):
    wide = {k: v.to(F64) for k, v in s.items() if isinstance(v, torch.Tensor)}
    leaf = {k: v.requires_grad_(c["grad"]) for k, v in wide.items() if k in ("h", "y", "pre", "post", "gate")}

    def norm(x, w):
        return w * x / torch.sqrt(torch.mean(x * x, dim=-1, keepdim=True) + eps)

    u = norm(leaf["y"], leaf["post"]) if c["post"] else leaf["y"]
    branch = u * leaf["gate"] if c["gate"] != "none" else u
    if not c["grad"]:
        h = c["scale"] * leaf["h"] + branch
        return {"h": h, "x": norm(h, leaf["pre"])}
    # the given stream is h' itself: what reaches it from both outputs goes on to the old stream (times scale) and the branch
    up, dpre = torch.autograd.grad(norm(leaf["h"], leaf["pre"]), [leaf["h"], leaf["pre"]], wide["dx"])
    up = up + wide["dh"]
    names = ["y"] + [k for k in ("post", "gate") if k in leaf]
    down = dict(zip(names, torch.autograd.grad(branch, [leaf[k] for k in names], up)))
    return {"dh": up * c["scale"], "dpre": dpre, **{"d" + k: v for k, v in down.items()}}


def _adamw_exact(c, s):
    t = s["t"] + 1
    w = (s["p"] if s["master"] is None else s["master"]).to(F64)
    g = s["grad"].to(F64) * 0.75

    def held(codes, scales):
        return (codes.to(F32).to(F64).view(-1, BLOCK) * scales.to(F64)[:, None]).view(-1)

    m, v = (held(s["m"], s["ms"]), held(s["r"], s["rs"]) ** 2) if c["bits"] == 8 else (s["m"].to(F64), s["v"].to(F64))
    m = s["b1"] * m + (1 - s["b1"]) * g
    v = s["b2"] * v + (1 - s["b2"]) * g ** 2
    del g
    w = w - s["lr"] * s["wd"] * w - s["lr"] * (m / (1 - s["b1"] ** t)) / ((v / (1 - s["b2"] ** t)).sqrt() + s["eps"])
    out = {"p": w}
    if s["master"] is not None:
        out["master"] = w
    if c["bits"] == 32:
        return {**out, "m": m, "v": v}
    for code, scale, x in (("m", "ms", m), ("r", "rs", v.sqrt())):
        x = x.view(-1, BLOCK)
        top = x.abs().amax(1)
        out[scale] = top / TOP
        out[code] = (x / (top / TOP).clamp(min=1e-300)[:, None]).view(-1)
    return out


# ---------------------------------------------------------------------------------- work of one pass
def work(c):
    if c["op"] == "loss":
        M, d, V = c["M"], c["d"], c["V"]
        read = 2 * (M * d + V * d) + 4 * M
        if not c["grad"]:
            return {"bytes": read + 8 * M, "flops": 2.0 * M * d * V}
        # logits, dH and dW: one product each
        return {"bytes": read + 8 * M + 2 * (M * d + V * d), "flops": 6.0 * M * d * V}
    if c["op"] == "norm":
        n, st, wt = c["M"] * c["d"], 2 if c["stream"] == "bf16" else 4, 2 if c["weights"] == "bf16" else 4
        vectors = (1 + c["post"] + (c["gate"] == "channel")) * wt * c["d"]
        token = 2 * n if c["gate"] == "token" else 0
        if not c["grad"]:
            return {"bytes": n * (2 * st + 4) + token + vectors, "flops": 12.0 * n}
        # reads dx, dh, h', y and the gate, writes dh, dy and the gate's gradient
        return {"bytes": n * (3 * st + 6) + 2 * token + 2 * vectors, "flops": 30.0 * n}
    n = sum(_sizes(c))
    weight = 2 + 2 + 8 if c["params"] == "bf16" else 4 + 8  # gradient in, parameter out, its 32-bit value in and out
    states = 16 if c["bits"] == 32 else 4 + 16 / BLOCK
    return {"bytes": n * (weight + states), "flops": 15.0 * n}
