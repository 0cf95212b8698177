"""The training calls on a side stream that is busy: what they read may be let go of as soon as
they return, and its memory is not handed out again before they have read it."""
import pytest
import torch

import gemm_epilogue_reduction_gb300 as sb
from gemm_epilogue_reduction_gb300 import synth

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


def _busy(stream):
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        torch.cuda._sleep(40_000_000)  # some 20 ms


def _reuse(shapes):
    """Takes and overwrites freed blocks of these sizes on the current stream."""
    return [torch.full(s, 7, dtype=t, device="cuda") for s, t in shapes for _ in range(3)]


@pytest.mark.parametrize("raw", [False, True])
def test_inputs_may_go(raw):
    side = torch.cuda.Stream()
    stream = side.cuda_stream if raw else side
    M, d, V = 64, 1024, 9000
    BF, F32 = torch.bfloat16, torch.float32

    def inputs():
        H, W = synth.make_hw(M, d, V, seed=2, device="cuda")
        return H, W, synth.make_targets(M, V, device="cuda")

    H, W, t = inputs()
    f = sb.cross_entropy(H, W, t)
    want = (f["loss"], sb.cross_entropy_backward(H, W, t, f["lse"])["dW"])
    pre = torch.ones(d, device="cuda")
    n = sb.residual_norm(H, H.flip(0), pre)
    back = sb.residual_norm_backward(H, H.flip(1), n["h"], H.flip(0), pre)
    want += (n["x"], back["dh"], back["dpre"])
    torch.cuda.synchronize()
    keep_h = n["h"].clone()

    _busy(side)
    a, b, c = inputs()
    f = sb.cross_entropy(a, b, c, stream=stream)
    g = sb.cross_entropy_backward(a, b, c, f["lse"], stream=stream)
    y = a.flip(0)
    n = sb.residual_norm(a, y, pre, stream=stream)
    z = a.flip(1)
    k = sb.residual_norm_backward(a, z, keep_h, y, pre, stream=stream)
    del a, b, c, y, z
    junk = _reuse([((M, d), BF), ((V, d), BF), ((M,), torch.int32)])
    torch.cuda.synchronize()
    got = (f["loss"], g["dW"], n["x"], k["dh"], k["dpre"])
    for i, (x, w) in enumerate(zip(got, want)):
        assert torch.equal(x, w), i
    del junk


def test_gradients_of_a_step_may_go():
    n = 300_000
    side = torch.cuda.Stream()
    grads = [torch.randn(n, device="cuda") for _ in range(2)]
    p, q = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
    ref = sb.AdamW([q])
    for g in grads:
        ref.step([g])
    opt = sb.AdamW([p])
    torch.cuda.synchronize()
    _busy(side)
    for g in grads:
        opt.step([g.clone()], stream=side)
        junk = _reuse([((n,), torch.float32)])
        side.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    assert torch.equal(p, q)
    del junk


def test_optimiser_may_go():
    n = 300_000
    side = torch.cuda.Stream()
    g, p, q = torch.randn(n, device="cuda"), torch.zeros(n, device="cuda"), torch.zeros(
        n, device="cuda")
    sb.AdamW([q], [g]).step()
    torch.cuda.synchronize()
    opt = sb.AdamW([p], [g])
    _busy(side)
    opt.step(stream=side)
    del opt
    junk = _reuse([((n,), torch.float32)])
    torch.cuda.synchronize()
    assert torch.equal(p, q)
    del junk


def test_legacy_stream_handle():
    a, pre = torch.ones(4, 256, device="cuda", dtype=torch.bfloat16), torch.ones(256, device="cuda")
    want = sb.residual_norm(a, a, pre)["x"]
    assert torch.equal(sb.residual_norm(a, a, pre, stream=0)["x"], want)
