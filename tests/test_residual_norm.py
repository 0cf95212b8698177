"""The fused residual norm and its gradients against the definition in 64 bits.

Bounds (u = 2^-8 for a rounding to bf16, e = 2^-24 for one in fp32): a value that goes through
k fp32 roundings and a root mean square is within r = 32e of its own magnitude plus that of the
terms it is a difference of; sums over rows or columns add at most n·e relative to the sum of
magnitudes, which a tree of partial sums keeps below (sqrt(n) + 64)·e for the n <= 16384 here
(the group's tree over columns, at most ceil(rows / blocks) rows in turn and then a block tree).
Outputs in bf16 add u of the value.
"""
import pytest
import torch

import gemm_epilogue_reduction_gb300 as sb

gpu = pytest.mark.gpu
U, E = 2.0 ** -8, 2.0 ** -24
R = 32 * E


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gemm_epilogue_reduction_gb300 import build as sbbuild
    sbbuild.build()


def _make(M, d, *, stream=torch.bfloat16, weights=torch.float32, post=True, gate="channel", seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def rnd(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    s = {"h": (2 * rnd(M, d)).to(stream), "y": rnd(M, d).to(torch.bfloat16),
         "pre": (1 + 0.2 * rnd(d)).to(weights),
         "post": (1 + 0.2 * rnd(d)).to(weights) if post else None,
         "gate": {None: None, "channel": (0.5 + 0.3 * rnd(d)).to(weights),
                  "token": (0.5 + 0.3 * rnd(M, d)).to(torch.bfloat16)}[gate],
         "dx": rnd(M, d).to(torch.bfloat16), "dh": rnd(M, d).to(stream)}
    return s


def _round(v, t):
    return U * v.abs() if t == torch.bfloat16 else E * v.abs()


def _forward_exact(s, scale, eps):
    h, y, pre = s["h"].double(), s["y"].double(), s["pre"].double()
    u = y
    if s["post"] is not None:
        u = y / torch.sqrt((y * y).mean(1, keepdim=True) + eps) * s["post"].double()
    if s["gate"] is not None:
        u = u * s["gate"].double()
    out = scale * h + u
    mag = (scale * h).abs() + u.abs()
    rms = torch.sqrt((out * out).mean(1, keepdim=True) + eps)
    x = out / rms * pre
    # what an error of R·mag in h' does to x: directly, and through the root mean square
    ex = R * (mag / rms * pre.abs() + x.abs() * (1 + (mag * out.abs()).mean(1, keepdim=True) / rms ** 2))
    return {"h": (out, R * mag + _round(out, s["h"].dtype)), "x": (x, ex + U * x.abs())}


def _backward_exact(s, scale, eps, dh=True):
    h, y, pre, dx = (s[k].double() for k in ("h", "y", "pre", "dx"))
    d = h.shape[1]
    rh = 1 / torch.sqrt((h * h).mean(1, keepdim=True) + eps)
    a = dx * pre
    t = rh * (a - h * rh ** 2 * (a * h).mean(1, keepdim=True))
    tm = rh * (a.abs() + h.abs() * rh ** 2 * (a * h).abs().mean(1, keepdim=True))
    if dh:
        t, tm = t + s["dh"].double(), tm + s["dh"].double().abs()
    cols = ((h.shape[0] + 1) ** 0.5 + 64) * E + R  # a sum over the rows
    out = {"dh": (scale * t, R * abs(scale) * tm + _round(scale * t, s["h"].dtype)),
           "dpre": ((dx * h * rh).sum(0), cols * (dx * h * rh).abs().sum(0))}
    ry = 1 / torch.sqrt((y * y).mean(1, keepdim=True) + eps) if s["post"] is not None else 1.0
    u = y * ry * (s["post"].double() if s["post"] is not None else 1.0)
    if s["gate"] is not None:
        if s["gate"].dim() == 1:
            out["dgate"] = ((t * u).sum(0), cols * (tm * u.abs()).sum(0))
        else:
            out["dgate"] = (t * u, R * tm * u.abs())
        t, tm = t * s["gate"].double(), tm * s["gate"].double().abs()
    if s["post"] is not None:
        out["dpost"] = ((t * y * ry).sum(0), cols * (tm * (y * ry).abs()).sum(0))
        f, fm = t * s["post"].double(), tm * s["post"].double().abs()
        t = ry * (f - y * ry ** 2 * (f * y).mean(1, keepdim=True))
        tm = ry * (fm + y.abs() * ry ** 2 * (fm * y.abs()).mean(1, keepdim=True))
    out["dy"] = (t, R * tm)
    for k, src in (("dpre", "pre"), ("dpost", "post"), ("dgate", "gate"), ("dy", "y")):
        if k in out:
            out[k] = (out[k][0], out[k][1] + _round(out[k][0], s[src].dtype))
    return out


def _within(got, want, name):
    value, bound = want
    off = (got.double() - value).abs()
    assert torch.isfinite(got).all(), name
    assert (off <= bound + 1e-37).all(), (name, float((off - bound).max()), float(off.max()))


def _kw(s):
    return {"post": s["post"], "gate": s["gate"]}


def _check(s, scale=1.0, eps=1e-6, dh=True):
    f = sb.residual_norm(s["h"], s["y"], s["pre"], scale=scale, eps=eps, **_kw(s))
    for k, want in _forward_exact(s, scale, eps).items():
        _within(f[k], want, k)
    b = sb.residual_norm_backward(s["dx"], s["dh"] if dh else None, s["h"], s["y"], s["pre"],
                                  scale=scale, eps=eps, **_kw(s))
    want = _backward_exact(s, scale, eps, dh)
    for k in ("dh", "dy", "dpre", "dpost", "dgate"):
        if k in want:
            _within(b[k], want[k], k)
        else:
            assert b[k] is None
    return f, b


SHAPES = [(1, 1), (1, 64), (3, 7), (5, 250), (16, 5120), (33, 96), (2, 4100), (700, 640),
          (1021, 260), (40, 6144), (305, 8192), (7, 8200), (3, 16384), (2, 16383), (9, 1025)]


@gpu
@pytest.mark.parametrize("M,d", SHAPES)
@pytest.mark.parametrize("stream,weights", [(torch.bfloat16, torch.bfloat16),
                                            (torch.float32, torch.float32),
                                            (torch.bfloat16, torch.float32),
                                            (torch.float32, torch.bfloat16)])
def test_values_and_gradients(M, d, stream, weights):
    _check(_make(M, d, stream=stream, weights=weights, seed=M + d), scale=0.5)


@gpu
@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("gate", [None, "channel", "token"])
@pytest.mark.parametrize("M,d", [(300, 520), (17, 77)])
def test_optional_parts(post, gate, M, d):
    _check(_make(M, d, post=post, gate=gate, seed=3), scale=-1.5, dh=gate != "token")


@gpu
def test_arrays_off_the_wide_alignment():
    """Views that start in the middle of an allocation are read value by value."""
    s = _make(20, 264, seed=5)
    for k, v in list(s.items()):
        room = torch.zeros(v.numel() + 1, dtype=v.dtype, device="cuda")
        s[k] = room[1:].view(v.shape).copy_(v)
    _check(s)


@gpu
def test_rows_do_not_meet():
    """A row of zeros, of infinities or of NaN leaves every other row as it is; a row of zeros
    gives zeros and finite gradients."""
    s = _make(9, 512, gate="token", seed=6)
    clean, back = _check(s)
    s["h"][2], s["y"][2] = 0, 0
    s["h"][4] = float("inf")
    s["y"][5] = float("nan")
    f = sb.residual_norm(s["h"], s["y"], s["pre"], **_kw(s))
    b = sb.residual_norm_backward(s["dx"], s["dh"], s["h"], s["y"], s["pre"], **_kw(s))
    keep = [0, 1, 3, 6, 7, 8]
    for a, c in ((f, clean), (b, back)):
        for k in ("h", "x") if a is f else ("dh", "dy", "dgate"):
            assert torch.equal(a[k][keep], c[k][keep]), k
    assert (f["x"][2] == 0).all() and (f["h"][2] == 0).all()
    for k in ("dh", "dy", "dgate"):
        assert torch.isfinite(b[k][2]).all()


@gpu
def test_outputs_may_replace_inputs():
    s = _make(50, 640, seed=7)
    want, back = _check(s)
    h, y = s["h"].clone(), s["y"].clone()
    st = sb.sb_residual_norm_forward(h, y, s["pre"], s["post"], s["gate"], sb.SB_GATE_CHANNEL, 50,
                                     640, sb.SB_BF16, sb.SB_F32, 1.0, 1e-6, h, y)
    assert st == sb.SB_OK
    assert torch.equal(h, want["h"]) and torch.equal(y, want["x"])
    dx, dh = s["dx"].clone(), s["dh"].clone()
    n = sb.sb_residual_norm_workspace_bytes(50, 640)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    dp, dq, dg = (torch.empty_like(s["pre"]) for _ in range(3))
    st = sb.sb_residual_norm_backward(dx, dh, s["h"], s["y"], s["pre"], s["post"], s["gate"],
                                      sb.SB_GATE_CHANNEL, 50, 640, sb.SB_BF16, sb.SB_F32, 1.0, 1e-6,
                                      dh, dx, dp, dq, dg, ws, n)
    assert st == sb.SB_OK
    for a, k in ((dh, "dh"), (dx, "dy"), (dp, "dpre"), (dq, "dpost"), (dg, "dgate")):
        assert torch.equal(a, back[k]), k


@gpu
def test_no_rows():
    s = _make(0, 96)
    f = sb.residual_norm(s["h"], s["y"], s["pre"], **_kw(s))
    assert f["x"].shape == (0, 96)
    b = sb.residual_norm_backward(s["dx"], s["dh"], s["h"], s["y"], s["pre"], **_kw(s))
    for k in ("dpre", "dpost", "dgate"):
        assert (b[k] == 0).all(), k


@gpu
def test_gradients_against_differences():
    """Directional derivatives of <h', a> + <x, b> in 64 bits by central differences of 1e-4
    against the gradients, within their bounds (the differences' error is of third order)."""
    M, d, scale, eps = 6, 72, 0.7, 1e-6
    s = _make(M, d, stream=torch.float32, seed=8)
    # backward differentiates at the stored h': here it is exactly scale·h + gate·n(y; post)
    with torch.no_grad():
        h_out = _forward_exact(s, scale, eps)["h"][0]
    t = dict(s, h=h_out.float())
    b = sb.residual_norm_backward(s["dx"], s["dh"], t["h"], s["y"], s["pre"], scale=scale, eps=eps,
                                  **_kw(s))
    bound = _backward_exact(t, scale, eps)

    def value(**new):
        o = _forward_exact({**{k: v.double() for k, v in s.items()}, **new}, scale, eps)
        return (o["h"][0] * s["dh"].double()).sum() + (o["x"][0] * s["dx"].double()).sum()

    g = torch.Generator(device="cuda").manual_seed(2)
    for k, out in (("h", "dh"), ("y", "dy"), ("pre", "dpre"), ("post", "dpost"), ("gate", "dgate")):
        way = torch.randn(s[k].shape, generator=g, device="cuda", dtype=torch.float64)
        slope = (value(**{k: s[k].double() + 1e-4 * way}) -
                 value(**{k: s[k].double() - 1e-4 * way})) / 2e-4
        mine = (b[out].double() * way).sum()
        # 1e-4: the differences' error, and h' rounded to fp32
        assert abs(slope - mine) <= (bound[out][1] * way.abs()).sum() + 1e-4, (k, slope, mine)


@gpu
def test_repeats_streams_and_graphs_give_the_same_bits():
    s = _make(3000, 1032, weights=torch.bfloat16, seed=9)
    f, b = _check(s)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (None, side):
        for _ in range(5):
            f2 = sb.residual_norm(s["h"], s["y"], s["pre"], stream=stream, **_kw(s))
            b2 = sb.residual_norm_backward(s["dx"], s["dh"], s["h"], s["y"], s["pre"],
                                           stream=stream, **_kw(s))
        torch.cuda.synchronize()
        for x, y in ((f, f2), (b, b2)):
            for k in x:
                if k != "workspace":
                    assert torch.equal(x[k], y[k]), k
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        f2 = sb.residual_norm(s["h"], s["y"], s["pre"], **_kw(s))
        b2 = sb.residual_norm_backward(s["dx"], s["dh"], s["h"], s["y"], s["pre"], **_kw(s))
    for k in ("h", "y", "dx", "dh"):
        s[k].copy_(s[k].flip(0))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(f2["x"], f["x"].flip(0)) and torch.equal(b2["dy"], b["dy"].flip(0))


@gpu
def test_offsets_past_32_bits():
    """More than 2^31 values: the last rows, which 32-bit offsets would miss, are as alone."""
    M, d, n = 350_003, 6144, 40
    s = {k: torch.zeros(M, d, dtype=torch.bfloat16, device="cuda") for k in ("h", "y", "dx", "dh")}
    small = _make(n, d, weights=torch.bfloat16, seed=10)
    for k in s:
        s[k][M - n:] = small[k]
    kw = _kw(small)
    f = sb.residual_norm(s["h"], s["y"], small["pre"], **kw)
    g = sb.residual_norm(small["h"], small["y"], small["pre"], **kw)
    for k in ("h", "x"):
        assert torch.equal(f[k][M - n:], g[k]) and not f[k][:M - n].any(), k
    b = sb.residual_norm_backward(s["dx"], s["dh"], s["h"], s["y"], small["pre"], **kw)
    c = sb.residual_norm_backward(*(small[k] for k in ("dx", "dh", "h", "y", "pre")), **kw)
    for k in ("dh", "dy"):
        assert torch.equal(b[k][M - n:], c[k]) and not b[k][:M - n].any(), k
    want = _backward_exact(small, 1.0, 1e-6)
    for k in ("dpre", "dpost", "dgate"):
        _within(b[k], want[k], k)


@gpu
def test_python_refusals():
    s = _make(8, 64)
    with pytest.raises(TypeError):
        sb.residual_norm(s["h"].half(), s["y"], s["pre"])
    with pytest.raises(TypeError):
        sb.residual_norm(s["h"], s["y"].float(), s["pre"])
    with pytest.raises(TypeError):
        sb.residual_norm(s["h"], s["y"], s["pre"], post=s["pre"].bfloat16())
    with pytest.raises(ValueError):
        sb.residual_norm(s["h"], s["y"][:4], s["pre"])
    with pytest.raises(ValueError):
        sb.residual_norm(s["h"][:, ::2], s["y"][:, ::2], s["pre"][::2])
    with pytest.raises(ValueError):
        sb.residual_norm(s["h"], s["y"], s["pre"], gate=s["gate"][:32])
    with pytest.raises(ValueError):
        sb.residual_norm(s["h"].cpu(), s["y"], s["pre"])
    with pytest.raises(sb.SbError):
        sb.residual_norm(s["h"], s["y"], s["pre"], eps=-1.0)
    with pytest.raises(sb.SbError):
        big = _make(1, 16385)
        sb.residual_norm(big["h"], big["y"], big["pre"])
    with pytest.raises(TypeError):
        sb.residual_norm_backward(s["dx"], s["dh"].float(), s["h"], s["y"], s["pre"])
    with pytest.raises(sb.SbError):
        sb.residual_norm_backward(s["dx"], s["dh"], s["h"], s["y"], s["pre"],
                                  workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))


def test_c_refusals():
    P = 1 << 20

    def fwd(h=P, y=P, pre=P, post=P, gate=P, kind=1, M=4, d=64, st=0, wt=1, scale=1.0, eps=1e-6,
            ho=P, x=P):
        return sb.sb_residual_norm_forward(h, y, pre, post, gate, kind, M, d, st, wt, scale, eps,
                                           ho, x, 0)

    def bwd(dx=P, dh=P, h=P, y=P, pre=P, post=P, gate=P, kind=1, M=4, d=64, st=0, wt=1, scale=1.0,
            eps=1e-6, dho=P, dy=P, dpre=P, dpost=P, dgate=P, ws=P, n=1 << 30):
        return sb.sb_residual_norm_backward(dx, dh, h, y, pre, post, gate, kind, M, d, st, wt,
                                            scale, eps, dho, dy, dpre, dpost, dgate, ws, n, 0)

    bad, off = sb.SB_ERR_INVALID_ARG, sb.SB_ERR_ALIGNMENT
    for call in (fwd, bwd):
        for kw in ({"h": None}, {"y": None}, {"pre": None}, {"gate": None}, {"kind": 3},
                   {"kind": -1}, {"M": -1}, {"M": 2 ** 31}, {"d": 0}, {"d": 16385}, {"st": 2},
                   {"wt": -1}, {"scale": float("nan")}, {"eps": -1.0}, {"eps": float("inf")}):
            assert call(**kw) == bad, (call.__name__, kw)
        for kw in ({"h": P + 1}, {"h": P + 2, "st": 1}, {"y": P + 1}, {"pre": P + 2},
                   {"post": P + 2}, {"gate": P + 2}):
            assert call(**kw) == off, (call.__name__, kw)
    assert fwd(ho=None) == bad and fwd(x=None) == bad and fwd(x=P + 1) == off
    for kw in ({"dx": None}, {"dho": None}, {"dy": None}, {"dpre": None}, {"dpost": None},
               {"dgate": None}, {"ws": None}):
        assert bwd(**kw) == bad, kw
    for kw in ({"dx": P + 1}, {"dh": P + 1}, {"dho": P + 1}, {"dpre": P + 2}, {"ws": P + 8}):
        assert bwd(**kw) == off, kw
    assert sb.sb_residual_norm_workspace_bytes(4, 0) == 0
    assert sb.sb_residual_norm_workspace_bytes(-1, 64) == 0
