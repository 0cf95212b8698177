"""The layer norm with its branch and dropout, and its gradients, against the definition in 64 bits.

Bounds (u = 2^-8 for a rounding to bf16, e = 2^-24 for one in fp32, R = 32e for what a sum over a row
in the kernels' tree of at most 30 steps, or a few roundings in turn, can be off relative to its
magnitudes): the mean is off by m = R·mean|h'|, a centred value c by dc = m + 2e(|h| + |branch|) + e|c|,
the variance by mean(2|c|dc) + R·var, so 1/deviation relatively by rho = mean(|c|dc)/(var + eps) + R.
The outputs' bounds follow by the sum of their terms.  A sum over rows adds (sqrt(rows) + 64)·e + R of
its terms' magnitudes (at most 8 rows in turn, 12 groups, 19 + 8 partials).
"""
import pytest
import torch

import gemm_epilogue_reduction_gb300 as sb
from test_dropout import dropped, factor, kept

gpu = pytest.mark.gpu
U, E = 2.0 ** -8, 2.0 ** -24
R = 32 * E
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gemm_epilogue_reduction_gb300 import build as sbbuild
    sbbuild.build()


def _make(M, d, *, stream=BF, weights=F32, bias=True, branch=True, seed=0, level=0.5):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def rnd(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    return {"h": (level + 2 * rnd(M, d)).to(stream), "y": rnd(M, d).to(BF) if branch else None,
            "weight": (1 + 0.2 * rnd(d)).to(weights), "bias": rnd(d).to(weights) if bias else None,
            "dx": rnd(M, d).to(BF), "dh": rnd(M, d).to(stream)}


def _round(v, t):
    return (U if t is BF else E) * v.abs()


def _stats(h, eps, slack):
    """(c, dc, 1/deviation, rho) of rows h in 64 bits; slack: what the values themselves are off."""
    c = h - h.mean(1, keepdim=True)
    dc = R * h.abs().mean(1, keepdim=True) + slack + slack.mean(1, keepdim=True) + E * c.abs()
    v = (c * c).mean(1, keepdim=True) + eps
    return c, dc, 1 / torch.sqrt(v), (c.abs() * dc).mean(1, keepdim=True) / v + R


def _forward(s, p, seed, eps):
    h, slack = s["h"].double(), 0 * s["h"].double()
    out = {}
    if s["y"] is not None:
        add = dropped(s["y"], p, seed)[0]
        slack = 2 * E * (h.abs() + add.abs())
        h = h + add
        out["h"] = (h, slack + _round(h, s["h"].dtype))
    c, dc, r, rho = _stats(h, eps, slack)
    w = s["weight"].double()
    x, dx = c * r * w, (dc + c.abs() * rho) * r * w.abs()
    if s["bias"] is not None:
        x = x + s["bias"].double()
        dx = dx + E * (x.abs() + s["bias"].double().abs())
    out["x"] = (x, dx + U * x.abs() + 4 * E * x.abs())
    return out


def _backward(s, p, seed, eps, dh, dy):
    h, dx, w = s["h"].double(), s["dx"].double(), s["weight"].double()
    c, dc, r, rho = _stats(h, eps, 0 * h)
    a = dx * w
    ma, mac = a.mean(1, keepdim=True), (a * c).mean(1, keepdim=True)
    t = r * (a - ma) - c * r ** 3 * mac
    dma = R * a.abs().mean(1, keepdim=True)
    dmac = R * (a * c).abs().mean(1, keepdim=True) + (a.abs() * dc).mean(1, keepdim=True)
    off = (rho + 4 * E) * r * (a.abs() + ma.abs()) + r * dma
    off = off + r ** 3 * (dc * mac.abs() + c.abs() * dmac + (3 * rho + 8 * E) * (c * mac).abs())
    if dh:
        t = t + s["dh"].double()
        off = off + 2 * E * s["dh"].double().abs()
    cols = ((h.shape[0] + 1) ** 0.5 + 64) * E + R
    k = dx * c * r
    out = {"dh": (t, off + 2 * E * t.abs() + _round(t, s["h"].dtype))}
    dw = k.sum(0)
    out["dweight"] = (dw, (dx.abs() * r * (dc + c.abs() * (rho + 2 * E))).sum(0) + cols * k.abs().sum(0) +
                      _round(dw, s["weight"].dtype))
    db = dx.sum(0)
    out["dbias"] = (db, cols * dx.abs().sum(0) + _round(db, s["weight"].dtype))
    if dy:
        keep, f = kept(h.numel(), p, seed).view(h.shape), factor(p)
        v = torch.where(keep, t * f, 0.0)
        out["dy"] = (v, torch.where(keep, (off + 4 * E * t.abs()) * f, 0.0) + U * v.abs())
    return out


def _within(got, want, name):
    value, bound = want
    off = (got.double() - value).abs()
    assert torch.isfinite(got).all(), name
    assert (off <= bound * 1.01 + 1e-37).all(), (name, float((off - bound).max()), float(off.max()))


def _check(s, p=0.0, seed=0, eps=1e-5, dh=True):
    f = sb.layer_norm(s["h"], s["weight"], s["bias"], y=s["y"], p=p, seed=seed, eps=eps)
    for k, want in _forward(s, p, seed, eps).items():
        _within(f[k], want, k)
    if s["y"] is None:
        assert f["h"] is s["h"]
    dy = s["y"] is not None
    b = sb.layer_norm_backward(s["dx"], s["dh"] if dh else None, s["h"], s["weight"],
                               need_dbias=s["bias"] is not None, need_dy=dy, p=p, seed=seed, eps=eps)
    want = _backward(s, p, seed, eps, dh, dy)
    for k in ("dh", "dy", "dweight", "dbias"):
        if (k == "dbias" and s["bias"] is None) or (k == "dy" and not dy):
            assert b[k] is None
        else:
            _within(b[k], want[k], k)
    return f, b


SHAPES = [(1, 2), (1, 64), (3, 7), (5, 250), (16, 5120), (33, 96), (2, 4100), (700, 640), (1021, 260),
          (40, 6144), (305, 8192), (7, 8200), (3, 16384), (2, 16383), (9, 1025), (1000, 33), (130, 4099)]


@gpu
@pytest.mark.parametrize("M,d", SHAPES)
@pytest.mark.parametrize("stream,weights", [(BF, BF), (F32, F32), (BF, F32), (F32, BF)])
def test_values_and_gradients(M, d, stream, weights):
    _check(_make(M, d, stream=stream, weights=weights, seed=M + d), p=0.2, seed=77)


@gpu
@pytest.mark.parametrize("M,d", [(1250, 4096), (1251, 3737), (1249, 3585), (650, 8192), (700, 7001), (613, 6143),
                                 (1111, 6137), (153, 7168)])
@pytest.mark.parametrize("stream,branch", [(BF, True), (BF, False), (F32, True), (F32, False)])
def test_blocks_that_fill_an_sm(M, d, stream, branch):
    # two groups of long rows, rows of more than 6144 values; several turns, the last one with a row missing
    _check(_make(M, d, stream=stream, branch=branch, seed=M + d), p=0.2 * branch, seed=5)


@gpu
@pytest.mark.parametrize("M,d", [(1, 5120), (50, 1032), (7, 333), (64, 100), (33, 12)])
@pytest.mark.parametrize("bias", [True, False])
@pytest.mark.parametrize("branch,p", [(False, 0.0), (True, 0.0), (True, 0.5), (True, 1.0)])
@pytest.mark.parametrize("dh", [True, False])
def test_optional_inputs(M, d, bias, branch, p, dh):
    _check(_make(M, d, bias=bias, branch=branch, seed=d), p=p, seed=2 ** 63 + 5, dh=dh)


@gpu
@pytest.mark.parametrize("d", [640, 4099])
@pytest.mark.parametrize("stream", [BF, F32])
def test_a_level_far_from_zero(d, stream):
    """A row's level of a thousand deviations: the variance is summed over centred values."""
    _check(_make(20, d, stream=stream, branch=False, seed=3, level=2000.0))


@gpu
def test_one_value_and_constant_rows():
    s = _make(9, 1, branch=False, seed=4)
    f, b = _check(s)
    assert torch.equal(f["x"], s["bias"].bfloat16().expand(9, 1)) and (b["dweight"] == 0).all()
    # equal values of any size: the mean is theirs but for its rounding, which eps has to outweigh
    h = torch.full((4, 512), 3.0, device="cuda")
    x = sb.layer_norm(h, torch.ones(512, device="cuda"))["x"]
    assert (x == 0).all()


@gpu
def test_the_branch_is_dropped_as_dropout_drops():
    for M, d in ((30, 640), (11, 333), (9, 100)):
        s = _make(M, d, stream=F32, seed=5)
        f = sb.layer_norm(s["h"], s["weight"], s["bias"], y=s["y"], p=0.3, seed=9)
        assert torch.equal(f["h"], sb.dropout(s["y"], 0.3, seed=9, residual=s["h"]))
        b = sb.layer_norm_backward(s["dx"], s["dh"], f["h"], s["weight"], need_dy=True, p=0.3, seed=9)
        assert torch.equal(b["dy"], sb.dropout(b["dh"], 0.3, seed=9, dtype=BF))


@gpu
def test_what_is_not_finite_stays_in_its_row():
    s = _make(6, 264, seed=6)
    s["h"][2, 5], s["h"][4, 0] = float("nan"), float("inf")
    f = sb.layer_norm(s["h"], s["weight"], s["bias"], y=s["y"])
    bad = ~torch.isfinite(f["x"]).all(1)
    assert bad.tolist() == [False, False, True, False, True, False]
    # a dropped infinity has no part in its row
    s = _make(4, 264, seed=7)
    keep = kept(4 * 264, 0.5, 1).view(4, 264)
    s["y"][~keep] = float("inf")
    assert torch.isfinite(sb.layer_norm(s["h"], s["weight"], y=s["y"], p=0.5, seed=1)["x"]).all()


@gpu
def test_in_place_at_the_c_interface():
    s = _make(50, 640, seed=8)
    want, back = _check(s, p=0.1, seed=3)
    h, y = s["h"].clone(), s["y"].clone()
    assert sb.sb_layer_norm_forward(h, y, s["weight"], s["bias"], 50, 640, 0, 1, 0.1, 3, None, 1e-5, h,
                                    y) == sb.SB_OK
    assert torch.equal(h, want["h"]) and torch.equal(y, want["x"])
    dx, dh = s["dx"].clone(), s["dh"].clone()
    n = sb.sb_layer_norm_workspace_bytes(50, 640)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    dw, db = (torch.empty_like(s["weight"]) for _ in range(2))
    assert sb.sb_layer_norm_backward(dx, dh, s["h"], s["weight"], 50, 640, 0, 1, 0.1, 3, None, 1e-5, dh,
                                     dx, dw, db, ws, n) == sb.SB_OK
    for a, k in ((dh, "dh"), (dx, "dy"), (dw, "dweight"), (db, "dbias")):
        assert torch.equal(a, back[k]), k


@gpu
def test_no_rows():
    s = _make(0, 96)
    assert sb.layer_norm(s["h"], s["weight"], s["bias"], y=s["y"])["x"].shape == (0, 96)
    b = sb.layer_norm_backward(s["dx"], s["dh"], s["h"], s["weight"])
    assert (b["dweight"] == 0).all() and (b["dbias"] == 0).all()


@gpu
def test_gradients_against_differences():
    """Directional derivatives of <h', a> + <x, b> in 64 bits by central differences of 1e-4 against
    the gradients, within their bounds (the differences' error is of third order)."""
    M, d, p, seed, eps = 6, 72, 0.25, 5, 1e-5
    s = _make(M, d, stream=F32, seed=8)
    h_out = _forward(s, p, seed, eps)["h"][0].float()
    b = sb.layer_norm_backward(s["dx"], s["dh"], h_out, s["weight"], need_dy=True, p=p, seed=seed, eps=eps)
    bound = _backward(dict(s, h=h_out), p, seed, eps, True, True)

    def value(**new):
        t = {**{k: v.double() for k, v in s.items()}, **new}
        o = _forward(t, p, seed, eps)
        return (o["h"][0] * t["dh"]).sum() + (o["x"][0] * t["dx"]).sum()

    g = torch.Generator(device="cuda").manual_seed(2)
    for k, out in (("h", "dh"), ("y", "dy"), ("weight", "dweight"), ("bias", "dbias")):
        way = torch.randn(s[k].shape, generator=g, device="cuda", dtype=torch.float64)
        slope = (value(**{k: s[k].double() + 1e-4 * way}) - value(**{k: s[k].double() - 1e-4 * way})) / 2e-4
        # 1e-4: the differences' error, and h' rounded to fp32
        assert abs(slope - (b[out].double() * way).sum()) <= (bound[out][1] * way.abs()).sum() + 1e-4, k


@gpu
def test_repeats_streams_and_graphs_give_the_same_bits():
    s = _make(3000, 1032, weights=BF, seed=9)
    f, b = _check(s, p=0.1, seed=4)
    kw = {"p": 0.1, "seed": 4}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())

    def both(**more):
        return (sb.layer_norm(s["h"], s["weight"], s["bias"], y=s["y"], **kw, **more),
                sb.layer_norm_backward(s["dx"], s["dh"], s["h"], s["weight"], need_dy=True, **kw, **more))

    for stream in (None, side, side.cuda_stream):
        for _ in range(5):
            f2, b2 = both(stream=stream)
        torch.cuda.synchronize()
        for x, y in ((f, f2), (b, b2)):
            for k in x:
                if k != "workspace":
                    assert torch.equal(x[k], y[k]), k
    off = torch.zeros(1, dtype=torch.int64, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        f2, b2 = both(seed_offset=off)
    for step in (0, 7):
        off.fill_(step)
        graph.replay()
        kw["seed"] = 4 + step
        f, b = both()
        torch.cuda.synchronize()
        assert torch.equal(f2["x"], f["x"]) and torch.equal(b2["dy"], b["dy"])
        assert torch.equal(b2["dweight"], b["dweight"])


@gpu
def test_offsets_past_32_bits():
    """More than 2^31 values: the last rows, which 32-bit offsets would miss, are as alone (but for
    the draws of their branch, which go by the element's number)."""
    M, d, n = 350_003, 6144, 3
    h = torch.randn(n, d, device="cuda").bfloat16()
    big = torch.zeros(M, d, dtype=BF, device="cuda")
    big[-n:] = h
    w = torch.ones(d, device="cuda")
    x = sb.layer_norm(big, w)["x"]
    assert torch.equal(x[-n:], sb.layer_norm(h, w)["x"]) and (x[:M - n] == 0).all()
    del x
    f = sb.layer_norm(big, w, y=torch.ones_like(big), p=0.5, seed=6)["h"]
    keep = kept(n * d, 0.5, 6, first=(M - n) * d).view(n, d)
    assert torch.equal(f[-n:], (h.float() + torch.where(keep, 2.0, 0.0)).bfloat16())


@gpu
def test_refusals():
    s = _make(4, 64)
    for bad in ({"h": s["h"].half()}, {"weight": s["weight"].half()}, {"bias": s["bias"].bfloat16()},
                {"y": s["y"].float()}, {"seed_offset": torch.zeros(1, device="cuda")}):
        with pytest.raises(TypeError):
            sb.layer_norm(**{"h": s["h"], "weight": s["weight"], **bad})
    for bad in ({"h": s["h"].t()}, {"h": s["h"][0]}, {"weight": s["weight"][:8]}, {"bias": s["bias"][:8]},
                {"y": s["y"][:2]}, {"h": s["h"].cpu()}, {"seed": 2 ** 64}):
        with pytest.raises(ValueError):
            sb.layer_norm(**{"h": s["h"], "weight": s["weight"], **bad})
    for bad in ({"p": 1.5}, {"eps": -1.0}, {"eps": float("nan")}):
        with pytest.raises(sb.SbError):
            sb.layer_norm(s["h"], s["weight"], y=s["y"], **bad)
    with pytest.raises(sb.SbError):
        sb.layer_norm(torch.zeros(2, 16392, device="cuda"), torch.zeros(16392, device="cuda"))
    with pytest.raises(TypeError):
        sb.layer_norm_backward(s["dx"], s["dh"].float(), s["h"], s["weight"])
    with pytest.raises(sb.SbError):
        sb.layer_norm_backward(s["dx"], s["dh"], s["h"], s["weight"],
                               workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))


def test_c_refusals():
    P = 1 << 20

    def fwd(h=P, y=P, weight=P, bias=P, M=4, d=64, st=0, wt=1, p=0.1, off=P, eps=1e-5, ho=P, x=P):
        return sb.sb_layer_norm_forward(h, y, weight, bias, M, d, st, wt, p, 0, off, eps, ho, x, 0)

    def bwd(dx=P, dh=P, h=P, weight=P, M=4, d=64, st=0, wt=1, p=0.1, off=P, eps=1e-5, dho=P, dy=P, dw=P,
            db=P, ws=P, n=1 << 30):
        return sb.sb_layer_norm_backward(dx, dh, h, weight, M, d, st, wt, p, 0, off, eps, dho, dy, dw, db,
                                         ws, n, 0)

    bad, off = sb.SB_ERR_INVALID_ARG, sb.SB_ERR_ALIGNMENT
    for call in (fwd, bwd):
        for kw in ({"h": None}, {"weight": None}, {"M": -1}, {"M": 2 ** 31}, {"d": 0}, {"d": 16385},
                   {"st": 2}, {"wt": -1}, {"p": -0.1}, {"p": 1.1}, {"p": float("nan")}, {"eps": -1.0},
                   {"eps": float("inf")}):
            assert call(**kw) == bad, (call.__name__, kw)
        for kw in ({"h": P + 1}, {"h": P + 2, "st": 1}, {"weight": P + 2}, {"off": P + 4}):
            assert call(**kw) == off, (call.__name__, kw)
    assert fwd(x=None) == bad and fwd(ho=None) == bad
    assert fwd(bias=P + 2) == off and fwd(y=P + 1) == off and fwd(x=P + 1) == off and fwd(ho=P + 1) == off
    for kw in ({"dx": None}, {"dho": None}, {"dw": None}, {"ws": None}):
        assert bwd(**kw) == bad, kw
    for kw in ({"dx": P + 1}, {"dh": P + 1}, {"dho": P + 1}, {"dy": P + 1}, {"dw": P + 2}, {"db": P + 2},
               {"ws": P + 8}):
        assert bwd(**kw) == off, kw
    # outputs over a part of an input (rows of 512 bytes), or over another one than their own
    A, B_, C, D, W_, Z = (P + k * 4096 for k in range(1, 7))
    f = {"h": A, "y": B_, "weight": W_, "bias": Z, "off": P, "ho": C, "x": D}
    for kw in ({"ho": A + 2}, {"x": B_ + 2}, {"x": A}, {"ho": B_}, {"ho": D}, {"x": W_}, {"ho": Z}):
        assert fwd(**{**f, **kw}) == bad, kw
    g = {"dx": A, "dh": B_, "h": C, "weight": W_, "off": P, "dho": D, "dy": Z, "dw": P + 99 * 4096,
         "db": P + 100 * 4096, "ws": P + 101 * 4096}
    for kw in ({"dho": C}, {"dho": A}, {"dho": B_ + 2}, {"dy": A + 2}, {"dy": C}, {"dy": B_}, {"dy": D},
               {"dy": W_}):
        assert bwd(**{**g, **kw}) == bad, kw
    assert sb.sb_layer_norm_workspace_bytes(4, 0) == 0 and sb.sb_layer_norm_workspace_bytes(-1, 64) == 0
