"""The operators at a model's two ends, case by case: how their inputs are made, their plain form in elementary torch
operations, the calls of this package, their definition in 64 bits and the work of one pass.

Four operators, as a step meets them:

* ``embedding``: the tokens' rows of the vocabulary matrix, out_t = scale W[id_t], and its gradient, the sum of the
  tokens' gradients for each row of W, written whole or added to the output head's gradient of the same (tied) matrix.
* ``dropout``: out_i = residual_i + keep_i x_i / (1 - p). Element i draws 16 bits, field i mod 4 of number i / 4 of the
  SplitMix64 stream of a seed, and is dropped where they are below round(65536 p), so no mask is stored. The call is its own gradient.
* ``layer_norm``: h' = h + dropout(y), x = (h' - mean) / sqrt(variance + eps) weight + bias, and its gradients.
* ``verify_drafts``: which of the tokens that a small model drafted the head's distribution p keeps. Draft x of
  distribution q stays where u < p(x) / q(x); the first that does not is replaced by a sample of max(p - q, 0), and where
  all stay a sample of the next row's p follows. Samples are argmax w_j / -log u_rj with 24-bit u_rj, number r V + j of a seed's stream.
"""
import math
import random

import torch

own = False  # true: run() makes the package's calls; false: the plain forms

BF, F32, F64, I32 = torch.bfloat16, torch.float32, torch.float64, torch.int32
TYPES = {"bf16": BF, "fp32": F32}
IGNORE = -100


def listed():
    return [
        # a decode step's tokens on their way in: latency
        {"name": "embed 16", "op": "embed", "M": 16, "d": 5120, "V": 151936, "weights": "bf16", "stream": "bf16", "grad": "none"},
        # a training batch whose embedding is tied to the head: into the gradient that the loss has left
        {"name": "embed grad tied 8192", "op": "embed", "M": 8192, "d": 6144, "V": 200064, "weights": "bf16", "stream": "bf16", "grad": "add"},
        # a batch with a matrix of its own: the whole gradient is written, most of it zeros
        {"name": "embed grad whole 4096", "op": "embed", "M": 4096, "d": 4096, "V": 151936, "weights": "bf16", "stream": "bf16", "grad": "whole"},
        # dropout behind the embedding of a short sequence
        {"name": "dropout 64", "op": "dropout", "M": 64, "d": 4096, "x": "bf16", "out": "bf16", "residual": False, "p": 0.1},
        # a branch's dropout and its sum with the residual stream, a whole batch
        {"name": "dropout residual 8192", "op": "dropout", "M": 8192, "d": 6144, "x": "bf16", "out": "bf16", "residual": True, "p": 0.1},
        # decoding: the norm in front of the head for a few rows, latency
        {"name": "layer norm forward 16", "op": "norm", "M": 16, "d": 5120, "grad": False, "stream": "bf16", "weights": "bf16", "bias": True, "branch": False, "p": 0.0},
        # training batches with the branch's dropout, forward and backward
        {"name": "layer norm forward 8192", "op": "norm", "M": 8192, "d": 6144, "grad": False, "stream": "bf16", "weights": "bf16", "bias": True, "branch": True, "p": 0.1},
        {"name": "layer norm backward 8192", "op": "norm", "M": 8192, "d": 6144, "grad": True, "stream": "bf16", "weights": "bf16", "bias": True, "branch": True, "p": 0.1},
        # a ragged batch on a 32-bit residual stream, an odd width
        {"name": "layer norm backward ragged 1021", "op": "norm", "M": 1021, "d": 4099, "grad": True, "stream": "fp32", "weights": "fp32", "bias": True, "branch": False, "p": 0.0},
        # one user's drafts on the decode shape: latency
        {"name": "verify 1", "op": "verify", "B": 1, "n": 4, "V": 151936, "logits": "bf16", "draft": True, "lse": False, "temperature": 1.0},
        # a batch on an odd vocabulary, with the logsumexp that the head's projection returned
        {"name": "verify lse 32", "op": "verify", "B": 32, "n": 5, "V": 50257, "logits": "bf16", "draft": True, "lse": True, "temperature": 1.0},
        # the largest serving batch, tempered
        {"name": "verify 64", "op": "verify", "B": 64, "n": 8, "V": 151936, "logits": "bf16", "draft": True, "lse": False, "temperature": 0.7},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["embed", "embed", "dropout", "norm", "norm", "verify", "verify"])
    kind = lambda: rng.choice(["bf16", "fp32"])  # noqa: E731
    if op == "embed":
        # one token to a large batch; widths of any size, vocabularies of any size, gradients of at most the largest listed one's bytes
        c = {"op": op, "M": _log(rng, 1, 8192), "d": _log(rng, 64, 6144), "V": _log(rng, 1000, 200064), "weights": kind(), "stream": kind(),
             "grad": rng.choice(["none", "add", "whole"])}
        c["V"] = min(c["V"], int(1.2e9 / (4 * c["d"])))
        return c
    if op == "dropout":
        return {"op": op, "M": _log(rng, 1, 4096), "d": _log(rng, 64, 6144), "x": kind(), "out": kind(), "residual": rng.random() < 0.5, "p": rng.choice([0.1, 0.25, 0.5])}
    if op == "norm":
        branch = rng.random() < 0.6
        return {"op": op, "M": _log(rng, 1, 8192), "d": _log(rng, 64, 6144), "grad": rng.random() < 0.5, "stream": kind(), "weights": kind(),
                "bias": rng.random() < 0.75, "branch": branch, "p": rng.choice([0.0, 0.1, 0.3]) if branch else 0.0}
    return {"op": op, "B": _log(rng, 1, 64), "n": rng.randint(1, 8), "V": _log(rng, 1000, 151936), "logits": rng.choice(["bf16", "bf16", "fp32"]),
            "draft": rng.random() < 0.75, "lse": rng.random() < 0.4, "temperature": rng.choice([1.0, 0.7, 1.3])}


# ---------------------------------------------------------------------------------- inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return {"c": case, "seed": seed * 7919 + 12345, **{"embed": _embed_inputs, "dropout": _dropout_inputs, "norm": _norm_inputs, "verify": _verify_inputs}[case["op"]](case, g)}


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _matrix(g, V, d, kind, scale):
    W = torch.empty(V, d, dtype=kind, device="cuda")
    for r in range(0, V, 16384):
        W[r:r + 16384] = _randn(g, min(16384, V - r), d) * scale
    return W


def _embed_inputs(c, g):
    M, d, V = c["M"], c["d"], c["V"]
    # tokens as in text: the k-th most frequent one with a share of about 1 / (k ln V), at any place of the vocabulary
    rank = ((V + 1.0) ** torch.rand(M, generator=g, device="cuda", dtype=F64) - 1).long().clamp(max=V - 1)
    ids = torch.randperm(V, generator=g, device="cuda")[rank].to(I32)
    if M > 8:  # padding
        ids[torch.rand(M, generator=g, device="cuda") < 0.1] = IGNORE
        ids[-1] = IGNORE
    s = {"ids": ids, "scale": math.sqrt(d)}
    if c["grad"] == "none":
        s["W"] = _matrix(g, V, d, TYPES[c["weights"]], d ** -0.5)
    else:
        s["dout"] = (0.01 * _randn(g, M, d)).to(TYPES[c["stream"]])
        if c["grad"] == "add":
            s["dW"] = _matrix(g, V, d, TYPES[c["weights"]], 0.01)
    return s


def _dropout_inputs(c, g):
    s = {"x": _randn(g, c["M"], c["d"]).to(TYPES[c["x"]]), "residual": None}
    if c["residual"]:
        s["residual"] = (2 * _randn(g, c["M"], c["d"])).to(TYPES[c["out"]])
    return s


def _norm_inputs(c, g):
    M, d, st, wt = c["M"], c["d"], TYPES[c["stream"]], TYPES[c["weights"]]
    # a residual stream has channels of its own level and spread
    level, spread = 0.5 * _randn(g, d), 0.5 + torch.rand(d, generator=g, device="cuda")
    s = {"h": (level + spread * 2 * _randn(g, M, d)).to(st), "weight": (1 + 0.1 * _randn(g, d)).to(wt), "bias": None, "y": None}
    if c["bias"]:
        s["bias"] = (0.1 * _randn(g, d)).to(wt)
    if c["grad"]:  # backward: h is then the stream h' that forward left, with the gradients of both outputs
        s["dx"], s["dh"] = (0.01 * _randn(g, M, d)).to(BF), (0.01 * _randn(g, M, d)).to(st)
    elif c["branch"]:
        s["y"] = (0.5 * _randn(g, M, d)).to(BF)
    return s


def _rows(c):
    """The requests' drafts, no two neighbours alike, some with none; a request has one row more than drafts."""
    return [(5 * b + 4) % (c["n"] + 1) + 1 for b in range(c["B"])]


def _verify_inputs(c, g):
    B, V, T, kind = c["B"], c["V"], c["temperature"], TYPES[c["logits"]]
    rows = _rows(c)
    starts = [0]
    for k in rows:
        starts.append(starts[-1] + k)
    R = starts[-1]
    z, q = torch.empty(R, V, dtype=kind, device="cuda"), torch.empty(R - B, V, dtype=kind, device="cuda") if c["draft"] else None
    drafts = torch.full((R,), -1, dtype=I32, device="cuda")
    lse = torch.empty(R, device="cuda") if c["lse"] else None
    draft_lse = torch.empty(R - B, device="cuda") if c["lse"] and c["draft"] else None
    inv_t = float(1 / torch.tensor(T))
    for b in range(B):
        a, k = starts[b], rows[b]
        # the target's logits: a spread over the vocabulary, and one token that is likely by itself, by a little or by a lot
        zb = 2 * _randn(g, k, V)
        likely = torch.randint(0, V, (k, 1), generator=g, device="cuda")
        level = T * torch.logsumexp(zb / T, 1, keepdim=True) + T * (4 * torch.rand(k, 1, generator=g, device="cuda") - 1)
        zb = zb.scatter_(1, likely, level).to(kind)
        z[a:a + k] = zb
        if c["lse"]:
            lse[a:a + k] = torch.logsumexp(zb.double() * inv_t, 1).float()
        if k == 1:
            continue
        if not c["draft"]:  # tokens looked up in what was written before: mostly the likely one
            other = torch.rand(k - 1, generator=g, device="cuda") < 0.2
            drafts[a:a + k - 1] = torch.where(other, (likely[:-1, 0] + 1) % V, likely[:-1, 0]).to(I32)
            continue
        # the small model knows the logits up to an error, and drafts samples of its own distribution
        qb = (zb[:-1].float() + 0.8 * _randn(g, k - 1, V)).to(kind)
        noise = -torch.log(-torch.log(torch.rand(k - 1, V, generator=g, device="cuda").clamp(1e-7, 1 - 1e-6)))
        drafts[a:a + k - 1] = (qb.float() / T + noise).argmax(1).to(I32)
        q[a - b:a - b + k - 1] = qb
        if c["lse"]:
            draft_lse[a - b:a - b + k - 1] = torch.logsumexp(qb.double() * inv_t, 1).float()
    return {"logits": z, "draft_logits": q, "drafts": drafts, "starts": torch.tensor(starts, dtype=I32, device="cuda"),
            "uniforms": torch.rand(R, generator=g, device="cuda"), "lse": lse, "draft_lse": draft_lse}


# ---------------------------------------------------------------------------------- one pass
def run(s):
    return {"embed": _embed, "dropout": _dropout, "norm": _norm, "verify": _verify}[s["c"]["op"]](s)


def _signed(x):
    return (x + 2 ** 63) % 2 ** 64 - 2 ** 63


def _draws(n, seed):
    """Numbers n (64 bits) of the SplitMix64 stream of `seed`, as signed 64-bit integers."""
    x = n * _signed(0x9E3779B97F4A7C15) + _signed(seed + 0x9E3779B97F4A7C15)
    x = (x ^ ((x >> 30) & (2 ** 34 - 1))) * _signed(0xBF58476D1CE4E5B9)
    x = (x ^ ((x >> 27) & (2 ** 37 - 1))) * _signed(0x94D049BB133111EB)
    return x ^ ((x >> 31) & (2 ** 33 - 1))


def _dropped(x, p, seed):
    """x with the elements dropped that the seed's stream says, the others over the share that is kept."""
    below = round(p * 65536)
    i = torch.arange((x.numel() + 3) // 4, device=x.device)
    fields = torch.stack([_draws(i, seed) >> k & 65535 for k in (0, 16, 32, 48)], 1).view(-1)[:x.numel()]
    return torch.where(fields.view(x.shape) >= below, x.float() * (65536 / (65536 - below)), 0.0)


def _embed(s):
    c, ids = s["c"], s["ids"]
    if own:
        import gemm_epilogue_reduction_gb300 as sb
        if c["grad"] == "none":
            return sb.embedding(ids, s["W"], scale=s["scale"], ignore_index=IGNORE, dtype=TYPES[c["stream"]])
        if c["grad"] == "add":
            return sb.embedding_backward(ids, s["dout"], scale=s["scale"], ignore_index=IGNORE, dW=s["dW"])["dW"]
        return sb.embedding_backward(ids, s["dout"], vocab=c["V"], scale=s["scale"], ignore_index=IGNORE, dtype=TYPES[c["weights"]])["dW"]
    has = (ids != IGNORE)[:, None]
    if c["grad"] == "none":
        return torch.where(has, s["W"][ids.clamp(min=0).long()].float() * s["scale"], 0.0).to(TYPES[c["stream"]])
    dout = torch.where(has, s["dout"].float() * s["scale"], 0.0)
    if c["grad"] == "whole":
        return torch.zeros(c["V"], c["d"], device=ids.device).index_add_(0, ids.clamp(min=0), dout).to(TYPES[c["weights"]])
    # added: the sums stand at each token's first place; every place of a token then writes the same row. Padding goes with some token, as zeros.
    at = torch.where(ids != IGNORE, ids, ids.amax().clamp(min=0)).long()
    place = torch.arange(len(at), device=ids.device)
    first = torch.full((c["V"],), len(at), device=ids.device).scatter_reduce_(0, at, place, "amin")[at]
    sums = torch.zeros_like(dout).index_add_(0, first, dout)
    s["dW"][at] = (s["dW"][at].float() + sums[first]).to(s["dW"].dtype)
    return s["dW"]


def _dropout(s):
    c, x, residual = s["c"], s["x"], s["residual"]
    if own:
        import gemm_epilogue_reduction_gb300 as sb
        return sb.dropout(x, c["p"], seed=s["seed"], residual=residual, dtype=TYPES[c["out"]])
    out = _dropped(x, c["p"], s["seed"])
    return (out if residual is None else residual.float() + out).to(TYPES[c["out"]])


def _norm(s, eps=1e-5):
    c, y, weight, bias = s["c"], s["y"], s["weight"], s["bias"]
    if own:
        import gemm_epilogue_reduction_gb300 as sb
        if c["grad"]:
            b = sb.layer_norm_backward(s["dx"], s["dh"], s["h"], weight, need_dbias=c["bias"], need_dy=c["branch"], p=c["p"], seed=s["seed"], eps=eps)
            return {k: b[k] for k in ("dh", "dy", "dweight", "dbias") if b[k] is not None}
        f = sb.layer_norm(s["h"], weight, bias, y=y, p=c["p"], seed=s["seed"], eps=eps)
        return {"h": f["h"], "x": f["x"]} if c["branch"] else f["x"]
    h, w = s["h"].float(), weight.float()
    if not c["grad"] and c["branch"]:
        h = h + (_dropped(y, c["p"], s["seed"]) if c["p"] else y.float())
    centred = h - h.mean(1, keepdim=True)
    r = (centred.square().mean(1, keepdim=True) + eps).rsqrt()
    unit = centred * r
    if not c["grad"]:
        x = (unit * w + bias.float() if c["bias"] else unit * w).to(BF)
        return {"h": h.to(s["h"].dtype), "x": x} if c["branch"] else x
    dx = s["dx"].float()
    a = dx * w
    dh = s["dh"].float() + r * (a - a.mean(1, keepdim=True) - unit * (a * unit).mean(1, keepdim=True))
    out = {"dh": dh.to(s["h"].dtype), "dweight": (dx * unit).sum(0).to(weight.dtype)}
    if c["bias"]:
        out["dbias"] = dx.sum(0).to(weight.dtype)
    if c["branch"]:
        out["dy"] = (_dropped(dh, c["p"], s["seed"]) if c["p"] else dh).to(BF)
    return out


def _verify(s):
    c, z, q, drafts, starts = s["c"], s["logits"], s["draft_logits"], s["drafts"], s["starts"]
    B, V, R = c["B"], c["V"], z.shape[0]
    if own:
        import gemm_epilogue_reduction_gb300 as sb
        f = sb.verify_drafts(z, drafts, starts, s["uniforms"], draft_logits=q, lse=s["lse"], draft_lse=s["draft_lse"], temperature=c["temperature"], seed=s["seed"])
        return {k: f[k] for k in ("token", "accepted", "token_logprob")}
    inv_t = float(1 / torch.tensor(c["temperature"]))  # rounded to 32 bits
    row = torch.arange(R, device=z.device)
    request = torch.searchsorted(starts[1:].long(), row, right=True)
    last = row + 1 == starts[1:][request]
    lse = s["lse"] if s["lse"] is not None else torch.logsumexp(z.float() * inv_t, 1)
    d = drafts.clamp(min=0).long()
    lp = z.gather(1, d[:, None])[:, 0].float() * inv_t - lse
    ratio, at = lp.exp(), (row - request).clamp(max=max(R - B - 1, 0))
    if q is not None and R > B:
        qlse = s["draft_lse"] if s["draft_lse"] is not None else torch.logsumexp(q.float() * inv_t, 1)
        ratio = (lp - (q[at, d].float() * inv_t - qlse[at])).exp()
    keep = (ratio > s["uniforms"]) & ~last
    # the row that ends each request: its first draft that does not stay, or its last row
    end = torch.full((B,), R, device=z.device).scatter_reduce_(0, request, torch.where(keep, R, row), "amin")
    y = (z[end].float() * inv_t).to(F64)  # 64 bits: p - q, and the sample that is largest by a hair
    p = (y - lse[end].to(F64)[:, None]).exp()
    w, refused = p, ~last[end][:, None]
    column = torch.arange(V, device=z.device)
    if q is None:
        w = torch.where(refused & (column == d[end][:, None]), 0.0, p)
    elif R > B:
        w = torch.where(refused, p - ((q[at[end]].float() * inv_t).to(F64) - qlse[at[end]].to(F64)[:, None]).exp(), p).clamp(min=0.0)
    w = torch.where(w.amax(1, keepdim=True) > 0, w, p)
    u = ((_draws(end[:, None] * V + column, s["seed"]) >> 40) & 0xFFFFFF).to(F64) * 2.0 ** -24
    score = w / -u.log()
    sample = torch.where(score == score.amax(1, keepdim=True), column, V).amin(1)
    mine = end[request]
    token = torch.where(row < mine, drafts, torch.where(row == mine, sample[request], -1).to(I32))
    sampled = (y.gather(1, sample[:, None])[:, 0] - lse[end].to(F64)).float()
    logprob = torch.where(row < mine, lp, torch.where(row == mine, sampled[request], 0.0))
    return {"token": token, "accepted": (end - starts[:-1]).to(I32), "token_logprob": logprob}


# ---------------------------------------------------------------------------------- definition in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"embed": _embed_exact, "dropout": _dropout_exact, "norm": _norm_exact, "verify": _verify_exact}[case["op"]](case, s)


def _stream(count, seed, first=0):
    """`count` numbers of SplitMix64's stream from number `first` on, in four 16-bit parts from the lowest: the additions and products in parts too."""
    mask = 0xFFFF

    def parts(v):
        return [(v >> 16 * k) & mask for k in range(4)]

    def carry(a):
        out, c = [], 0
        for k in range(4):
            v = a[k] + c
            out.append(v & mask)
            c = v >> 16
        return out

    def times(a, b):
        return carry([sum(a[i] * b[k - i] for i in range(k + 1)) for k in range(4)])

    def mix(a, shift):
        low = [*a, 0, 0, 0, 0]
        word, bit = divmod(shift, 16)
        return [a[k] ^ ((low[k + word] >> bit | low[k + word + 1] << (16 - bit)) & mask) for k in range(4)]

    n = torch.arange(first + 1, first + 1 + count, device="cuda")
    x = times(parts(n), parts(0x9E3779B97F4A7C15))
    x = carry([a + b for a, b in zip(x, parts(seed % 2 ** 64))])
    x = times(mix(x, 30), parts(0xBF58476D1CE4E5B9))
    x = times(mix(x, 27), parts(0x94D049BB133111EB))
    return mix(x, 31)


def _factors(shape, p, seed):
    """What dropout multiplies each element by: nothing, or one over the share that is kept."""
    n = math.prod(shape)
    drop = round(p * 2 ** 16)
    kept = torch.stack(_stream(-(-n // 4), seed), -1).reshape(-1)[:n].reshape(shape) >= drop
    return kept.to(F64) * (2 ** 16 / (2 ** 16 - drop))


def _embed_exact(c, s):
    used = torch.nonzero(s["ids"] != IGNORE)[:, 0]
    ids = s["ids"][used].long()
    if c["grad"] == "none":
        out = torch.zeros(c["M"], c["d"], dtype=F64, device="cuda")
        out[used] = s["W"][ids].to(F64) * s["scale"]
        return out
    sums = s["dW"].to(F64) if c["grad"] == "add" else torch.zeros(c["V"], c["d"], dtype=F64, device="cuda")
    return sums.index_add_(0, ids, s["dout"][used].to(F64) * s["scale"])


def _dropout_exact(c, s):
    out = s["x"].to(F64) * _factors(s["x"].shape, c["p"], s["seed"])
    return out if s["residual"] is None else out + s["residual"].to(F64)


def _norm_exact(c, s, eps=1e-5):
    h, weight = s["h"].to(F64), s["weight"].to(F64).requires_grad_(c["grad"])
    bias = s["bias"].to(F64) if c["bias"] else torch.zeros(c["d"], dtype=F64, device="cuda")
    if s["y"] is not None:
        h = h + s["y"].to(F64) * _factors(h.shape, c["p"], s["seed"])
    bias.requires_grad_(c["grad"])
    h.requires_grad_(c["grad"])
    var, mean = torch.var_mean(h, dim=1, correction=0, keepdim=True)
    x = (h - mean) / torch.sqrt(var + eps) * weight + bias
    if not c["grad"]:
        return {"h": h, "x": x} if c["branch"] else x
    up, dweight, dbias = torch.autograd.grad(x, [h, weight, bias], s["dx"].to(F64))
    up = up + s["dh"].to(F64)
    out = {"dh": up, "dweight": dweight}
    if c["bias"]:
        out["dbias"] = dbias
    if c["branch"]:
        out["dy"] = up * _factors(h.shape, c["p"], s["seed"])
    return out


def _verify_exact(c, s):
    z, q, V, inv_t = s["logits"], s["draft_logits"], c["V"], float(1 / torch.tensor(c["temperature"]))
    R = z.shape[0]
    token = torch.full((R,), -1, dtype=I32, device="cuda")
    logprob, accepted = torch.zeros(R, dtype=F64, device="cuda"), []
    drafts, u, begin = s["drafts"].tolist(), s["uniforms"].tolist(), 0

    def logs(row, given):
        t = row.to(F64) * inv_t
        return t - (torch.logsumexp(t, 0) if given is None else given.to(F64))

    for b, k in enumerate(_rows(c)):
        for r in range(begin, begin + k):
            lp = logs(z[r], None if s["lse"] is None else s["lse"][r])
            weight = lp.exp()
            if r < begin + k - 1:
                x = drafts[r]
                if q is None:
                    stays = float(weight[x]) > u[r]
                    weight[x] = 0.0
                else:
                    lq = logs(q[r - b], None if s["draft_lse"] is None else s["draft_lse"][r - b])
                    stays = math.exp(min(700.0, float(lp[x] - lq[x]))) > u[r]
                    weight = torch.relu(weight - lq.exp())
                if stays:
                    token[r], logprob[r] = x, lp[x]
                    continue
                if float(weight.max()) <= 0:
                    weight = lp.exp()
            part = _stream(V, s["seed"], r * V)
            bits = part[3] * 256 + (part[2] >> 8)
            x = int(torch.argmax(weight / -torch.log(bits.to(F64) / 2 ** 24)))
            token[r], logprob[r] = x, lp[x]
            accepted.append(r - begin)
            break
        begin += k
    return {"token": token, "accepted": torch.tensor(accepted, dtype=I32), "token_logprob": logprob}


# ---------------------------------------------------------------------------------- work of one pass
def _distinct(M, V):
    """How many different tokens M tokens are, on average (see _embed_inputs)."""
    k = torch.arange(1, V + 1, dtype=F64)
    return float((1 - (1 - torch.log1p(1 / k) / math.log(V + 1)) ** M).sum())


def work(c):
    size = {"bf16": 2, "fp32": 4}
    if c["op"] == "embed":
        M, d, V, wt, st = c["M"], c["d"], c["V"], size[c["weights"]], size[c["stream"]]
        rows = _distinct(0.9 * M if M > 8 else M, V)
        if c["grad"] == "none":
            return {"bytes": 4 * M + rows * d * wt + M * d * st, "flops": 1.0 * M * d}
        # padding's gradients are not read; added: the tokens' rows in and out
        used = 0.9 * M if M > 8 else M
        return {"bytes": 4 * M + used * d * st + (2 * rows if c["grad"] == "add" else V) * d * wt, "flops": 2.0 * M * d}
    if c["op"] == "dropout":
        n = c["M"] * c["d"]
        return {"bytes": n * (size[c["x"]] + size[c["out"]] * (1 + c["residual"])), "flops": 3.0 * n}
    if c["op"] == "norm":
        n, st, wt = c["M"] * c["d"], size[c["stream"]], size[c["weights"]]
        vectors = (1 + c["bias"]) * wt * c["d"]
        if not c["grad"]:
            return {"bytes": n * (st + 2 + (2 + st) * c["branch"]) + vectors, "flops": 10.0 * n}
        # reads dx, dh and h', writes dh and dy
        return {"bytes": n * (2 + 3 * st + 2 * c["branch"]) + wt * c["d"] + vectors, "flops": 20.0 * n}
    B, V, t, R = c["B"], c["V"], size[c["logits"]], sum(_rows(c))
    if not c["lse"]:  # every row's logsumexp
        return {"bytes": t * V * (R + (R - B) * c["draft"]), "flops": 3.0 * V * (R + (R - B) * c["draft"])}
    # the row that ends each request; the draft's too where it was refused (about three in ten drafts are)
    refused = sum(1 - 0.7 ** (k - 1) for k in _rows(c))
    return {"bytes": t * V * (B + refused * c["draft"]), "flops": 8.0 * V * B}
