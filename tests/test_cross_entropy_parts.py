"""What the second bf16 part of G (up to 32 rows) and the target's fp32 logit are for, on inputs where
their absence is larger than every other error.

G in two bf16 parts is within 2^-16 of its entries, in one part within 2^-9. Sums whose terms nearly
cancel show the difference: with u = 2^-9 of one rounding of the result,
  * dW of two equal rows of H with weights 1 and -(1 - 2^-6): both rows have the same p to the bit, so
    what remains is 2^-6 of the terms, off by the parts' 2^-16 of both terms and by what p is off
    (2 ez + 2^-18, as in test_cross_entropy.py) of the result itself;
  * dH with rows of W in pairs w, -w and small logits: terms p(z) w - p(-z) w, whose p are off by 2 ez +
    2^-18 each.
fp32 sums of n terms add n 2^-23 of the terms (tensor cores: steps of 16, at most 2 ulp lost in each).

The loss of a row whose target's logit z is large and negative is lse - z, and with zeros for all other
rows of W lse is known: the fp32 logit is a sum of d products in chains of at most d / 128 + 9
additions of halves (2^-24 of sum |h w| for each), where the tensor cores lose up to 2 ulp in each of
d / 16 steps, always towards zero.
"""
import math

import pytest
import torch

import gemm_epilogue_reduction_gb300 as sb

pytestmark = pytest.mark.gpu
U, E = 2.0 ** -9, 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


def _ez(H, W):
    size = float((H.double().abs() @ W.double().abs().T).max())
    return (H.shape[1] / 16 + 2) * 4 * E * size


@pytest.mark.parametrize("d,V", [(64, 500), (264, 3001)])
def test_head_gradient_of_rows_that_nearly_cancel(d, V):
    g = torch.Generator(device="cuda").manual_seed(d)
    h = torch.randn(1, d, generator=g, device="cuda").bfloat16()
    H = h.expand(2, d).contiguous()
    W = (torch.randn(V, d, generator=g, device="cuda") * d ** -0.5).bfloat16()
    t = torch.tensor([V // 2, V // 2], dtype=torch.int32, device="cuda")
    grad = torch.tensor([1.0, -(1 - 2.0 ** -6)], device="cuda")
    f = sb.cross_entropy(H, W, t, reduction="none")
    dW = sb.cross_entropy_backward(H, W, t, f["lse"], grad=grad, reduction="none")["dW"]
    G = torch.softmax(h.double() @ W.double().T, 1)[0]
    G[V // 2] -= 1
    want = 2.0 ** -6 * G[:, None] * h.double()
    terms = 2 * G.abs()[:, None] * h.double().abs()
    bound = (U + 2 * _ez(H, W) + 2.0 ** -18) * want.abs() + (2.0 ** -16 + 64 * 2.0 ** -23) * terms
    off = (dW.double() - want).abs()
    assert (off <= bound).all(), float((off / bound).max())
    # one part would be outside: a rounding to bf16 of each of the two terms
    one = (G.float().bfloat16().double() - (G * (1 - 2.0 ** -6)).float().bfloat16().double())
    assert ((one[:, None] * h.double() - want).abs() > bound).any()


@pytest.mark.parametrize("M", [1, 5, 32])
def test_hidden_gradient_of_columns_that_nearly_cancel(M):
    d, pairs = 64, 600
    g = torch.Generator(device="cuda").manual_seed(M)
    H = (torch.randn(M, d, generator=g, device="cuda") * 2.0 ** -6).bfloat16()
    half = (torch.randn(pairs, d, generator=g, device="cuda") * d ** -0.5).bfloat16()
    W = torch.cat([half, -half, torch.zeros(1, d, device="cuda").bfloat16()])
    t = torch.full((M,), 2 * pairs, dtype=torch.int32, device="cuda")  # the row of zeros
    f = sb.cross_entropy(H, W, t, reduction="sum")
    dH = sb.cross_entropy_backward(H, W, t, f["lse"], reduction="sum")["dH"]
    p = torch.softmax(H.double() @ W.double().T, 1)
    p[:, -1] = 0
    want, terms = p @ W.double(), p @ W.double().abs()
    steps = 2 * pairs / 16 + 8
    bound = U * want.abs() + (2.0 ** -16 + 2 * _ez(H, W) + 2.0 ** -18 + steps * 2.0 ** -23) * terms
    off = (dH.double() - want).abs()
    assert (off <= bound).all(), float((off / bound).max())
    one = p.float().bfloat16().double() @ W.double()
    assert ((one - want).abs() > bound).any()


@pytest.mark.parametrize("M", [3, 40])
def test_loss_of_a_negative_logit(M):
    d, V, z = 5120, 1000, -25.0
    g = torch.Generator(device="cuda").manual_seed(M)
    H = (1 + torch.rand(M, d, generator=g, device="cuda")).bfloat16()
    W = torch.zeros(V, d, device="cuda")
    t = torch.arange(M, device="cuda") * 5 + 1
    W[t] = (z / 1.5 / d) * (0.5 + torch.rand(M, d, generator=g, device="cuda"))
    W = W.bfloat16()
    f = sb.cross_entropy(H, W, t.int(), reduction="none")
    zt = (H.double() * W[t].double()).sum(1)
    # the other targets' rows have logits near z too: e^z of a thousand columns
    lse = torch.logsumexp(H.double() @ W.double().T, 1)
    size = (H.double() * W[t].double()).abs().sum(1)
    bound = (d / 128 + 9) * E * size + 2.0 ** -20 + 4 * E * (lse - zt)
    off = (f["loss"].double() - (lse - zt)).abs()
    assert (off <= bound).all(), float((off / bound).max())
    assert math.isfinite(float(f["loss"].sum()))
