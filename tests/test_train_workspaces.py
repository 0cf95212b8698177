"""A workspace that the caller gives to a training call is checked like the other tensors."""
import pytest
import torch

import gemm_epilogue_reduction_gb300 as sb
from gemm_epilogue_reduction_gb300 import synth

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


def _calls():
    H, W = synth.make_hw(9, 64, 300, seed=1, device="cuda")
    t = synth.make_targets(9, 300, device="cuda")
    lse = sb.cross_entropy(H, W, t)["lse"]
    pre = torch.ones(64, device="cuda")
    return [lambda ws: sb.cross_entropy(H, W, t, workspace=ws),
            lambda ws: sb.cross_entropy_backward(H, W, t, lse, workspace=ws),
            lambda ws: sb.residual_norm_backward(H, None, H, H, pre, workspace=ws)]


@pytest.mark.parametrize("call", range(3))
def test_refusals(call):
    f = _calls()[call]
    n = f(None)["workspace"].numel()
    for ws in (torch.empty(n, dtype=torch.uint8), torch.empty(n, dtype=torch.uint8, pin_memory=True),
               torch.empty(2 * n, dtype=torch.uint8, device="cuda")[::2]):
        with pytest.raises(ValueError, match="workspace"):
            f(ws)
    with pytest.raises(sb.SbError):
        f(torch.empty(n - 1, dtype=torch.uint8, device="cuda"))
    with pytest.raises(sb.SbError):  # not on a boundary that the call needs
        f(torch.empty(n + 8, dtype=torch.uint8, device="cuda")[8:])


@pytest.mark.parametrize("call", range(3))
def test_any_type_counts_by_its_bytes(call):
    f = _calls()[call]
    want = f(None)
    n = want["workspace"].numel()
    got = f(torch.empty((n + 3) // 4, dtype=torch.float32, device="cuda"))
    torch.cuda.synchronize()
    for k, x in want.items():
        if k != "workspace" and x is not None:
            assert torch.equal(got[k], x), k
