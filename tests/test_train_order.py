"""Training calls directly behind one another on one stream, without a synchronisation: what a call
reads is what the call before it wrote."""
import pytest
import torch

import gemm_epilogue_reduction_gb300 as sb
from gemm_epilogue_reduction_gb300 import synth

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


def test_loss_gradient_directly_after_the_norm():
    """x formed again in place of y (as a program that saves activations' memory does), and the
    gradient of the loss directly behind it: d is a multiple of 8 and not of 16, so neighbouring
    rows share sectors, and long enough to be read without the ring."""
    M, d, V = 200, 16376, 900
    g = torch.Generator(device="cuda").manual_seed(2)
    h, y = (torch.randn(M, d, generator=g, device="cuda").bfloat16() for _ in range(2))
    W = (torch.randn(V, d, generator=g, device="cuda") * d ** -0.5).bfloat16()
    t = synth.make_targets(M, V, device="cuda")
    pre = torch.ones(d, device="cuda")
    x = sb.residual_norm(h, y, pre)["x"]
    lse = sb.cross_entropy(x, W, t)["lse"]
    want = sb.cross_entropy_backward(x, W, t, lse)
    ho = torch.empty_like(h)
    for _ in range(10):
        buf = y.clone()
        assert sb.sb_residual_norm_forward(h, buf, pre, None, None, sb.SB_GATE_NONE, M, d,
                                           sb.SB_BF16, sb.SB_F32, 1.0, 1e-6, ho, buf) == sb.SB_OK
        got = sb.cross_entropy_backward(buf, W, t, lse)
        for k in ("dH", "dW"):
            assert torch.equal(got[k], want[k]), k
