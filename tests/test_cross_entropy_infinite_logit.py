"""A target whose logit is minus infinity: its loss is infinite, its logsumexp is that of the
others, and its gradient that of a probability of zero."""
import pytest
import torch

import gemm_epilogue_reduction_gb300 as sb
from gemm_epilogue_reduction_gb300 import synth

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


@pytest.mark.parametrize("M", [4, 70, 300])
def test_target_at_minus_infinity(M):
    d, V = 136, 700
    H, W = synth.make_hw(M, d, V, seed=5, device="cuda")
    t = synth.make_targets(M, V, seed=6, device="cuda")
    t[t == 9] = 10
    t[2] = 9
    H[:, 0], W[:, 0] = 0, 0
    H[2, 0], W[9, 0] = 16, -2e38  # the product overflows
    f = sb.cross_entropy(H, W, t, reduction="none")
    z = H.double() @ W.double().T
    z[2, 9] = -float("inf")
    lse = torch.logsumexp(z, 1)
    assert f["loss"][2] == float("inf")
    # the errors of logits of some units: 2^-16
    assert ((f["lse"].double() - lse).abs() <= 2.0 ** -16).all()
    rest = torch.arange(M, device="cuda") != 2
    want = lse - z[torch.arange(M, device="cuda"), t.long()]
    assert ((f["loss"].double() - want).abs() <= 2.0 ** -15)[rest].all()
    b = sb.cross_entropy_backward(H, W, t, f["lse"], reduction="none")
    G = torch.exp(z - lse[:, None])
    G[torch.arange(M, device="cuda"), t.long()] -= 1
    for got, value, size in ((b["dH"], G @ W.double(), G.abs() @ W.double().abs()),
                             (b["dW"], G.T @ H.double(), G.abs().T @ H.double().abs())):
        assert torch.isfinite(got).all()
        # G and the result are rounded to bf16 (2^-9 each), p within 2^-14
        assert ((got.double() - value).abs() <= 2.0 ** -7 * size + 1e-37).all()
