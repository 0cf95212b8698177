"""The head's cross entropy and its gradients against the definition in 64 bits.

Bounds, elementwise and derived from the formats (u = 2^-8 is bf16's largest relative rounding
error, e = 2^-24 that of fp32):
  * a logit is a sum of d products that are exact in fp32; the tensor cores add them in steps of
    16, each step losing at most 2 ulp of the running sum, so |dz| <= ez with
    ez = (d / 16 + 2) * 4e * max_rj sum_i |H_ri W_ji|;
  * lse inherits ez (its weights sum to 1), and its own sum and logarithm add less than
    2^-18 + 4e * |lse| (hardware exponentials of 2^-22 relative error, rescaled a few times);
    a row's loss subtracts the target's logit, within ez again, and adds z_loss * lse^2;
  * G carries exp's relative error (ez for z and for lse each, 2^-18 for the exponential) and
    one rounding to bf16, so relative to its two terms |dG| <= (u + 2 ez + 2^-18)(p' + [j = t]);
  * dH and dW are fp32 sums of products with G (steps as above, folded into the u of G: the
    sums here have at most 1500 steps of 2^-22) and are rounded to bf16 once.
"""
import numpy as np
import pytest
import torch

import gemm_epilogue_reduction_gb300 as sb
from gemm_epilogue_reduction_gb300 import synth

gpu = pytest.mark.gpu
U, E = 2.0 ** -8, 2.0 ** -24
IGN = -100


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gemm_epilogue_reduction_gb300 import build as sbbuild
    sbbuild.build()


def _inputs(M, d, V, seed, ignored=True, lift=6.0):
    H, W = synth.make_hw(M, d, V, seed=seed, device="cuda")
    t = synth.make_targets(M, V, seed=seed + 1, device="cuda")
    # some rows know their target well
    a = lift * torch.arange(M, device="cuda").remainder(4).float() / 4
    H = (H.float() + a[:, None] * W[t.long()].float()).to(torch.bfloat16)
    if ignored and M > 2:
        t[::5] = IGN
    return H, W, t


def _exact(H, W, t, *, reduction, z_loss, grad=None, ignore=IGN, piece=4096):
    """Loss, lse, dH, dW in 64 bits, with the bounds of each as laid out above."""
    H, M, V = H.double(), H.shape[0], W.shape[0]
    valid = t != ignore
    inside = valid & (t >= 0) & (t < V)
    at = torch.where(inside, t, 0).long()
    Hm = torch.where(valid[:, None], H, 0.0)
    W = W.double()
    z = torch.cat([H @ W[a:a + piece].T for a in range(0, V, piece)], 1)
    size = max((H.abs() @ W[a:a + piece].abs().T).max() for a in range(0, V, piece))
    ez = (H.shape[1] / 16 + 2) * 4 * E * float(size)
    lse = torch.logsumexp(z, 1)
    row = torch.where(valid, lse - z.gather(1, at[:, None])[:, 0] + z_loss * lse ** 2, 0.0)
    n = max(int(valid.sum()), 1)
    g = valid.double()
    if reduction == "mean":
        g = g / n
    if grad is not None:
        g = g * grad.double()
    p = torch.where(valid[:, None], torch.exp(z - lse[:, None]), 0.0)
    p = p * (1 + 2 * z_loss * lse * valid)[:, None]
    hot = torch.zeros_like(p)
    hot[torch.arange(M, device=p.device)[inside], at[inside]] = 1.0
    G = (p - hot) * g[:, None]
    mag = (p.abs() + hot) * g.abs()[:, None]
    eg = U + 2 * ez + 2.0 ** -18
    dH, dW = G @ W, G.T @ Hm
    e_lse = ez + 2.0 ** -18 + 4 * E * lse.abs()
    e_row = torch.where(valid, e_lse * (1 + 2 * abs(z_loss) * lse.abs()) + ez +
                        8 * E * (row.abs() + lse.abs()), 0.0)
    if reduction == "none":
        loss, e_loss = row, e_row
    else:
        div = n if reduction == "mean" else 1
        loss, e_loss = row.sum()[None] / div, e_row.sum()[None] / div + 4 * E * abs(row.sum() / div)
    return {"loss": (loss, e_loss), "lse": (lse, e_lse),
            "dH": (dH, eg * (mag @ W.abs()) + U * dH.abs() + 1e-37),
            "dW": (dW, eg * (mag.T @ Hm.abs()) + U * dW.abs() + 1e-37)}


def _within(got, want, name):
    value, bound = want
    off = (got.double() - value).abs()
    assert torch.isfinite(got).all(), name
    worst = (off - bound).argmax()
    assert (off <= bound).all(), (name, float(off.flatten()[worst]), float(bound.flatten()[worst]))


def _run(H, W, t, *, reduction="mean", z_loss=0.0, grad=None, ignore=IGN, **kw):
    f = sb.cross_entropy(H, W, t, ignore_index=ignore, z_loss=z_loss, reduction=reduction)
    b = sb.cross_entropy_backward(H, W, t, f["lse"], grad=grad, ignore_index=ignore,
                                  z_loss=z_loss, reduction=reduction, **kw)
    torch.cuda.synchronize()
    assert sb.device_status(f["workspace"]) == sb.SB_OK
    assert sb.device_status(b["workspace"]) == sb.SB_OK
    return {**f, **b}


def _check(M, d, V, *, reduction="mean", z_loss=0.0, grad=None, seed=0, **kw):
    H, W, t = _inputs(M, d, V, seed)
    got = _run(H, W, t, reduction=reduction, z_loss=z_loss, grad=grad, **kw)
    want = _exact(H, W, t, reduction=reduction, z_loss=z_loss, grad=grad)
    for k in ("loss", "lse", "dH", "dW"):
        _within(got[k], want[k], k)
    return got


SHAPES = [
    (1, 64, 100), (1, 8, 1), (2, 8, 7), (4, 256, 4096), (15, 72, 1000), (16, 5120, 1031),
    (64, 640, 5003), (127, 136, 257), (128, 256, 256), (129, 264, 511), (255, 64, 4099),
    (256, 512, 513), (257, 520, 1000), (300, 1032, 777), (513, 96, 2050), (1025, 200, 300),
]


@gpu
@pytest.mark.parametrize("M,d,V", SHAPES)
@pytest.mark.parametrize("reduction,z_loss", [("mean", 0.0), ("none", 1e-3)])
def test_loss_and_gradients(M, d, V, reduction, z_loss):
    grad = None
    if reduction == "none":  # weights of both signs, some of them zero
        grad = torch.linspace(-1, 2, M, device="cuda")
        grad[::3] = 0
    _check(M, d, V, reduction=reduction, z_loss=z_loss, grad=grad, seed=M + V)


@gpu
@pytest.mark.parametrize("M,d,V,piece", [(300, 136, 2000, 256), (40, 264, 3001, 512),
                                         (600, 72, 1111, 1024), (9, 640, 5000, 2304)])
def test_pieces_of_the_vocabulary(M, d, V, piece):
    """Any piece gives the gradients; the same piece gives the same bits."""
    a = _check(M, d, V, reduction="sum", z_loss=1e-4, seed=V, piece=piece)
    b = _check(M, d, V, reduction="sum", z_loss=1e-4, seed=V, piece=piece)
    for k in ("loss", "lse", "dH", "dW"):
        assert torch.equal(a[k], b[k]), k


@gpu
def test_split_reduction_at_a_wide_vocabulary():
    """Few rows against a long vocabulary: dH's reduction is split over the SMs."""
    _check(3, 512, 50257, seed=5)
    _check(70, 256, 70001, seed=6, reduction="sum")


@gpu
@pytest.mark.parametrize("up", [None, 3.5, 0.0, -2.0])
@pytest.mark.parametrize("reduction", ["mean", "sum"])
def test_incoming_gradient(up, reduction):
    grad = None if up is None else torch.tensor([up], device="cuda")
    _check(50, 128, 600, reduction=reduction, grad=grad, seed=9)


@gpu
@pytest.mark.parametrize("need", [(True, False), (False, True)])
@pytest.mark.parametrize("M,V,piece", [(33, 900, 0), (400, 900, 256), (3, 40000, 0)])
def test_one_gradient_only(need, M, V, piece):
    H, W, t = _inputs(M, 264, V, 3)
    both = _run(H, W, t, piece=piece)
    one = _run(H, W, t, piece=piece, need_dH=need[0], need_dW=need[1])
    want = _exact(H, W, t, reduction="mean", z_loss=0.0)
    for k, asked in zip(("dH", "dW"), need):
        if not asked:
            assert one[k] is None
        else:
            _within(one[k], want[k], k)
            if k == "dW":  # its reduction is never split: the same bits
                assert torch.equal(one[k], both[k])


@gpu
@pytest.mark.parametrize("reduction", ["mean", "sum", "none"])
def test_all_rows_ignored(reduction):
    H, W, t = _inputs(37, 136, 500, 1)
    t[:] = IGN
    got = _run(H, W, t, reduction=reduction, z_loss=0.1)
    for k in ("loss", "dH", "dW"):
        assert (got[k] == 0).all(), k


@gpu
def test_what_ignored_rows_hold_does_not_matter():
    H, W, t = _inputs(140, 136, 700, 1)
    rows = (t == IGN).nonzero()[:, 0]
    clean = _run(H, W, t)
    H[rows[0]] = float("nan")
    H[rows[1]] = float("inf")
    H[rows[2], 5] = -float("inf")
    H[rows[3]] = 3e38
    f = sb.cross_entropy(H, W, t)
    b = sb.cross_entropy_backward(H, W, t, f["lse"])
    assert torch.equal(f["loss"], clean["loss"])
    assert torch.equal(b["dW"], clean["dW"])
    assert torch.equal(b["dH"], clean["dH"])


@gpu
def test_ignore_index_inside_the_vocabulary():
    H, W, t = _inputs(40, 64, 300, 2, ignored=False)
    t[::4] = 0
    got = _run(H, W, t, ignore=0)
    want = _exact(H, W, t, reduction="mean", z_loss=0.0, ignore=0)
    for k in ("loss", "lse", "dH", "dW"):
        _within(got[k], want[k], k)


@gpu
@pytest.mark.parametrize("M", [5, 200])
def test_target_outside_the_vocabulary_is_reported(M):
    H, W, t = _inputs(M, 64, 300, 2, ignored=False)
    for bad in (300, -1, 2 ** 31 - 1, -2 ** 31):
        t2 = t.clone()
        t2[3] = bad
        f = sb.cross_entropy(H, W, t2, reduction="none")
        torch.cuda.synchronize()
        assert sb.device_status(f["workspace"]) == sb.SB_ERR_INVALID_ARG
        assert torch.isnan(f["loss"][3]) and torch.isfinite(f["loss"][[0, 1, 2, 4]]).all()
        b = sb.cross_entropy_backward(H, W, t2, f["lse"], reduction="none")
        assert torch.isfinite(b["dH"]).all() and torch.isfinite(b["dW"]).all()


@gpu
@pytest.mark.parametrize("reduction", ["mean", "sum", "none"])
def test_no_rows(reduction):
    H = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    W = torch.ones(50, 64, dtype=torch.bfloat16, device="cuda")
    t = torch.empty(0, dtype=torch.int32, device="cuda")
    got = _run(H, W, t, reduction=reduction)
    assert (got["loss"] == 0).all() and got["loss"].numel() == (reduction != "none")
    assert got["dH"].shape == (0, 64) and (got["dW"] == 0).all()


@gpu
def test_large_logits():
    """Logits of some hundreds: one column has all the weight."""
    H, W, t = _inputs(60, 256, 900, 4)
    H = H * 64
    got = _run(H, W, t)
    want = _exact(H, W, t, reduction="mean", z_loss=0.0)
    for k in ("loss", "lse"):
        _within(got[k], want[k], k)
    assert torch.isfinite(got["dH"]).all() and torch.isfinite(got["dW"]).all()


@gpu
def test_gradients_against_differences():
    """The directional derivatives of the 64-bit loss, by central differences: their error is of
    the third order in the step (1e-4 squared here), the gradients' the bound of this file."""
    M, d, V, zl = 48, 72, 500, 1e-2
    H, W, t = _inputs(M, d, V, 11)
    got = _run(H, W, t, z_loss=zl)
    want = _exact(H, W, t, reduction="mean", z_loss=zl)

    def loss(h, w):
        return _exact(h, w, t, reduction="mean", z_loss=zl)["loss"][0]

    g = torch.Generator(device="cuda").manual_seed(1)
    step = 1e-4
    for k in range(4):
        dirH = torch.randn(M, d, generator=g, device="cuda", dtype=torch.float64)
        dirW = torch.randn(V, d, generator=g, device="cuda", dtype=torch.float64)
        slope = (loss(H.double() + step * dirH, W) - loss(H.double() - step * dirH, W)) / (2 * step)
        mine = (got["dH"].double() * dirH).sum()
        assert abs(slope - mine) <= (want["dH"][1] * dirH.abs()).sum() + 1e-6, (slope, mine)
        slope = (loss(H, W.double() + step * dirW) - loss(H, W.double() - step * dirW)) / (2 * step)
        mine = (got["dW"].double() * dirW).sum()
        assert abs(slope - mine) <= (want["dW"][1] * dirW.abs()).sum() + 1e-6, (slope, mine)


@gpu
def test_repeats_give_the_same_bits_with_a_used_workspace():
    H, W, t = _inputs(600, 520, 3000, 8)
    f = sb.cross_entropy(H, W, t)
    b = sb.cross_entropy_backward(H, W, t, f["lse"], piece=1024)
    for ws in (f["workspace"], b["workspace"]):
        ws.fill_(0xFF)  # no initialisation is expected
    for _ in range(20):
        f2 = sb.cross_entropy(H, W, t, workspace=f["workspace"])
        b2 = sb.cross_entropy_backward(H, W, t, f2["lse"], piece=1024, workspace=b["workspace"])
        for x, y in ((f, f2), (b, b2)):
            for k in x:
                if k != "workspace":
                    assert torch.equal(x[k], y[k]), k


@gpu
def test_other_stream_and_graph():
    H, W, t = _inputs(100, 264, 2000, 13)
    want = _run(H, W, t)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    f = sb.cross_entropy(H, W, t, stream=side)
    b = sb.cross_entropy_backward(H, W, t, f["lse"], stream=side)
    side.synchronize()
    for k in ("loss", "lse"):
        assert torch.equal(f[k], want[k])
    for k in ("dH", "dW"):
        assert torch.equal(b[k], want[k])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        f = sb.cross_entropy(H, W, t)
        b = sb.cross_entropy_backward(H, W, t, f["lse"])
    H2, W2, t2 = _inputs(100, 264, 2000, 14)
    for a in (0, 1):  # the second replay finds the first one's workspace
        H.copy_(H2), W.copy_(W2), t.copy_(t2)
        graph.replay()
        torch.cuda.synchronize()
        again = _run(H2, W2, t2)
        for x in (f, b):
            for k in x:
                if k != "workspace":
                    assert torch.equal(x[k], again[k]), k


@gpu
def test_weights_written_by_the_kernel_before():
    """An update of W directly before the call on the same stream is what the call reads."""
    H, W, t = _inputs(16, 512, 20000, 15)
    for i in range(5):
        W.mul_(-0.5)
        f = sb.cross_entropy(H, W, t)
        b = sb.cross_entropy_backward(H, W, t, f["lse"])
        W0 = W.clone()
        torch.cuda.synchronize()
        f2 = sb.cross_entropy(H, W0, t)
        b2 = sb.cross_entropy_backward(H, W0, t, f2["lse"])
        assert torch.equal(f["loss"], f2["loss"]) and torch.equal(b["dW"], b2["dW"])
        assert torch.equal(b["dH"], b2["dH"])


@gpu
def test_watchdog_of_the_backward_call():
    H, W, t = _inputs(20, 64, 300, 2)
    f = sb.cross_entropy(H, W, t)
    torch.cuda.synchronize()
    assert sb.sb_debug_configure(True, 200_000_000) == sb.SB_OK
    try:
        b = sb.cross_entropy_backward(H, W, t, f["lse"])
        torch.cuda.synchronize()
        assert sb.device_status(b["workspace"]) == sb.SB_ERR_DEVICE_TIMEOUT
    finally:
        sb.sb_debug_configure(False, 2_000_000_000)
    again = _run(H, W, t)
    want = _exact(H, W, t, reduction="mean", z_loss=0.0)
    _within(again["dW"], want["dW"], "dW")


@gpu
def test_offsets_past_32_bits():
    """A head of more than 2^31 weights: the rows at its end, which 32-bit offsets would miss."""
    M, d, V = 40, 4096, 530_000
    W = torch.zeros(V, d, dtype=torch.bfloat16, device="cuda")
    rows = [0, 1, 255, 262_143, 262_144, 524_288, 524_289, V - 257, V - 256, V - 1]
    g = torch.Generator(device="cuda").manual_seed(1)
    W[rows] = (torch.randn(len(rows), d, generator=g, device="cuda") * d ** -0.5).bfloat16()
    H = torch.randn(M, d, generator=g, device="cuda").bfloat16()
    t = torch.tensor([rows[i % len(rows)] for i in range(M)], dtype=torch.int32, device="cuda")
    got = _run(H, W, t, reduction="sum", piece=0)
    # all other logits are 0: the definition over the rows that are not, the rest counted
    few = W[rows]
    z = H.double() @ few.double().T
    lse = torch.log(torch.exp(z).sum(1) + (V - len(rows)))
    at = torch.arange(M, device="cuda") % len(rows)
    loss = (lse - z[torch.arange(M, device="cuda"), at]).sum()
    assert abs(float(got["loss"]) - float(loss)) <= 1e-5 * float(loss)
    p = torch.exp(z - lse[:, None])
    p[torch.arange(M, device="cuda"), at] -= 1
    want = p.T @ H.double()
    off = (got["dW"][rows].double() - want).norm() / want.norm()
    assert off <= 2.0 ** -7, float(off)
    off = (got["dH"].double() - p @ few.double()).norm() / (p @ few.double()).norm()
    assert off <= 2.0 ** -7, float(off)
    # a row of no target and weight 0: the same small share of H's sum everywhere
    rest = (torch.exp(-lse)[None, :] @ H.double())[0]
    for r in (2, 524_290, V - 2):
        off = (got["dW"][r].double() - rest).norm() / rest.norm()
        assert off <= 2.0 ** -7, (r, float(off))


@gpu
def test_python_refusals():
    H, W, t = _inputs(8, 64, 100, 2)
    lse = torch.zeros(8, device="cuda")
    with pytest.raises(TypeError):
        sb.cross_entropy(H.float(), W, t)
    with pytest.raises(TypeError):
        sb.cross_entropy(H, W, t.long())
    with pytest.raises(ValueError):
        sb.cross_entropy(H, W[:, :32], t)
    with pytest.raises(ValueError):
        sb.cross_entropy(H.t().contiguous().t(), W, t)
    with pytest.raises(ValueError):
        sb.cross_entropy(H, W, t[:7])
    with pytest.raises(ValueError):
        sb.cross_entropy(H.cpu(), W, t)
    with pytest.raises(ValueError):
        sb.cross_entropy(H, W, t, reduction="average")
    with pytest.raises(sb.SbError):
        sb.cross_entropy(H, W, t, z_loss=float("nan"))
    with pytest.raises(sb.SbError):
        sb.cross_entropy(H, W, t, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(sb.SbError):
        sb.cross_entropy_backward(H, W, t, lse, need_dH=False, need_dW=False)
    with pytest.raises(sb.SbError):
        sb.cross_entropy_backward(H, W, t, lse, piece=-1)
    sb.cross_entropy_backward(H, W, t, lse, piece=2 ** 63 - 1)  # one piece
    with pytest.raises(ValueError):
        sb.cross_entropy_backward(H, W, t, lse, grad=torch.ones(8, device="cuda"))
    with pytest.raises(ValueError):
        sb.cross_entropy_backward(H, W, t, lse[:4])


def test_c_refusals():
    """Checked before the device is touched: the C entry points refuse what they cannot do."""
    P, Q = 1 << 20, 256  # an aligned address that nothing reads, a size

    def fwd(H=P, W=P, t=P, M=4, d=64, V=100, ign=IGN, red=2, zl=0.0, loss=P, lse=P, ws=P,
            n=1 << 30):
        return sb.sb_cross_entropy_forward(H, W, t, M, d, V, ign, red, zl, loss, lse, ws, n, 0)

    def bwd(H=P, W=P, t=P, lse=P, g=P, M=4, d=64, V=100, ign=IGN, red=2, zl=0.0, piece=0, dH=P,
            dW=P, ws=P, n=1 << 30):
        return sb.sb_cross_entropy_backward(H, W, t, lse, g, M, d, V, ign, red, zl, piece, dH, dW,
                                            ws, n, 0)

    bad = sb.SB_ERR_INVALID_ARG
    for call in (fwd, bwd):
        for kw in ({"H": None}, {"W": None}, {"t": None}, {"M": -1}, {"d": 0}, {"V": 0},
                   {"V": 2 ** 31}, {"red": 3}, {"red": -1}, {"zl": float("inf")}, {"lse": None},
                   {"ws": None}, {"M": 2 ** 31}):
            assert call(**kw) == bad, (call.__name__, kw)
        for kw in ({"H": P + 2}, {"W": P + 8}, {"d": 60}, {"t": P + 1}, {"lse": P + 2},
                   {"ws": P + 16}):
            assert call(**kw) == sb.SB_ERR_ALIGNMENT, (call.__name__, kw)
    assert fwd(loss=None) == bad and fwd(loss=P + 1) == sb.SB_ERR_ALIGNMENT
    assert fwd(n=Q) == sb.SB_ERR_WORKSPACE_TOO_SMALL
    assert bwd(dH=None, dW=None) == bad and bwd(piece=-256) == bad
    assert bwd(dH=P + 4) == sb.SB_ERR_ALIGNMENT and bwd(g=P + 2) == sb.SB_ERR_ALIGNMENT
    assert sb.sb_cross_entropy_workspace_bytes(4, 60, 100) == 0
    assert sb.sb_cross_entropy_workspace_bytes(-1, 64, 100) == 0
    assert sb.sb_cross_entropy_workspace_bytes(0, 64, 100) == 256
    assert sb.sb_cross_entropy_backward_workspace_bytes(4, 64, 100, -1, True, True) == 0
    assert sb.sb_cross_entropy_backward_workspace_bytes(4, 64, 100, 0, False, False) == 0
    assert (sb.sb_cross_entropy_workspace_bytes(4, 64, 100) ==
            sb.sb_workspace_bytes(4, 100, 1, sb.SB_TOKEN) + 256)
