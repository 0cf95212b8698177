"""A projection directly behind an optimizer step on one stream: it loads the weight early, and what
it loads is what the step wrote."""
import pytest
import torch

import gemm_epilogue_reduction_gb300 as sb
from gemm_epilogue_reduction_gb300 import synth

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("M,V,k", [(16, 40000, 4), (300, 20000, 2)])
def test_projection_after_an_optimizer_step(bits, M, V, k):
    """The projection loads the weight early; the step before it has to be done with it."""
    d = 512
    H, W = synth.make_hw(M, d, V, seed=3, device="cuda")
    dW = torch.randn(V, d, device="cuda").bfloat16()
    opt = sb.AdamW([W], [dW], lr=0.05, state_bits=bits)
    ws = torch.empty(sb.sb_workspace_bytes(M, V, k, sb.SB_TOKEN_LOGPROB), dtype=torch.uint8,
                     device="cuda")
    got, weights = [], []
    for i in range(8):
        out, bufs = sb.make_outputs(M, V, k, sb.SB_TOKEN_LOGPROB, workspace=ws)
        opt.step(lr=0.05 * (i + 1))
        assert sb.sb_lmhead_project(H, W, M, d, V, k, sb.SB_TOKEN_LOGPROB, 1.0, 0, out) == sb.SB_OK
        got.append(bufs)
        weights.append(W.clone())
    torch.cuda.synchronize()
    for bufs, w in zip(got, weights):
        want = sb.project(H, w, k, sb.SB_TOKEN_LOGPROB)
        torch.cuda.synchronize()
        for key in ("token", "token_logprob", "lse"):
            assert torch.equal(bufs[key], want[key]), key
