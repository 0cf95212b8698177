"""Weights of rows, incoming gradients and logits that are not finite: they show in the results
that the formulas put them in, and nowhere else."""
import pytest
import torch

import gemm_epilogue_reduction_gb300 as sb
from gemm_epilogue_reduction_gb300 import synth

pytestmark = pytest.mark.gpu
IGN = -100
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


def _inputs(M, d=136, V=700):
    H, W = synth.make_hw(M, d, V, seed=3, device="cuda")
    H = torch.where(H == 0, 1.0, H)
    t = synth.make_targets(M, V, seed=4, device="cuda")
    if M > 2:
        t[1::5] = IGN
    return H, W, t


def _grads(H, W, t, grad, reduction):
    f = sb.cross_entropy(H, W, t, reduction=reduction)
    b = sb.cross_entropy_backward(H, W, t, f["lse"], grad=grad, reduction=reduction)
    return b["dH"], b["dW"]


@pytest.mark.parametrize("M", [1, 20, 70, 300])
@pytest.mark.parametrize("others", [0.0, 0.5])
@pytest.mark.parametrize("odd", [NAN, INF, -INF])
def test_weight_of_a_row(M, others, odd):
    H, W, t = _inputs(M)
    r = 2 if M > 2 else 0
    grad = torch.full((M,), others, device="cuda")
    grad[r] = 0
    clean, _ = _grads(H, W, t, grad, "none")
    grad[r] = odd
    dH, dW = _grads(H, W, t, grad, "none")
    assert not torch.isfinite(dH[r]).any()
    rest = torch.arange(M, device="cuda") != r
    assert torch.equal(dH[rest], clean[rest])
    if odd != odd:
        assert torch.isnan(dW).all()
    else:  # G is infinite with the sign of p - [j = t], p > 0
        sign = torch.ones(W.shape[0], 1, device="cuda")
        sign[t[r].long()] = -1
        want = sign * H[r].float()[None, :].sign() * odd
        assert torch.equal(dW.float(), want)


@pytest.mark.parametrize("M", [20, 70, 300])
def test_weight_of_an_ignored_row_does_not_matter(M):
    H, W, t = _inputs(M)
    grad = torch.linspace(0.1, 1, M, device="cuda")
    want = _grads(H, W, t, grad, "none")
    grad[t == IGN] = NAN
    got = _grads(H, W, t, grad, "none")
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("M", [1, 20, 70, 300])
@pytest.mark.parametrize("reduction", ["sum", "mean"])
@pytest.mark.parametrize("odd", [NAN, INF])
def test_incoming_gradient(M, reduction, odd):
    H, W, t = _inputs(M)
    dH, dW = _grads(H, W, t, torch.tensor([odd], device="cuda"), reduction)
    valid = t != IGN
    assert not torch.isfinite(dH[valid]).any()
    assert (dH[~valid] == 0).all()
    assert not torch.isfinite(dW).any()
    t[:] = IGN
    dH, dW = _grads(H, W, t, torch.tensor([odd], device="cuda"), reduction)
    assert (dH == 0).all() and (dW == 0).all()
