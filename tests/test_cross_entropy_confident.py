"""The gradient of targets that the model is sure of, against the definition in 64 bits.

There G_t = p - 1 is the small difference of two numbers near 1, and the rest of the row adds up to
its opposite, so an error in the target's logit that p does not share with lse shows in full.
Bounds, per row with R = 1 - p (e = 2^-24; ez is the tensor cores' error of a logit as in
test_cross_entropy.py; u = 2^-8 the rounding of G and of the result to bf16):
  * an entry that is not the target's is off by (u + 2 ez + 2^-18) p_j;
  * the target's by (u + 2 ez + 2^-18) R for the same reasons, as R is the sum of the others, and
    by the fp32 roundings of numbers near 1 and near lse: the 128 exponentials of the target's
    record and the records' sum, (136 + V / 128) e, and lse with the difference from it, 2 e |lse|;
  * fp32 sums over them (folded into u), and one rounding of the result.
"""
import math

import pytest
import torch

import gemm_epilogue_reduction_gb300 as sb

gpu = pytest.mark.gpu
U, E = 2.0 ** -8, 2.0 ** -24
SHIFTED = 64  # channels that carry the shift of all logits


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gemm_epilogue_reduction_gb300 import build as sbbuild
    sbbuild.build()


def _inputs(M, d, V, shift, device="cuda"):
    """Rows whose targets have 1 - p from 1e-2 to 1e-6; `shift` is added to every logit."""
    g = torch.Generator().manual_seed(M + d)
    H = torch.randn(M, d, generator=g)
    W = torch.randn(V, d, generator=g) * (0.5 / math.sqrt(d))
    t = (torch.arange(M) * 7 + 3) % V
    assert t.unique().numel() == M
    H[:, :SHIFTED] = 8
    rest = H[:, SHIFTED:]
    lift = math.log(V) + 0.125 - torch.linspace(-2, -6, M) * math.log(10)
    W[t, SHIFTED:] = lift[:, None] * rest / rest.square().sum(1, keepdim=True)
    W[:, :SHIFTED] = shift / (8 * SHIFTED)
    return (H.bfloat16().to(device), W.bfloat16().to(device), t.int().to(device))


def _exact(H, W, t, z_loss):
    """dH and dW of the summed loss, R and the bounds of both gradients."""
    M, V, d = H.shape[0], W.shape[0], H.shape[1]
    H, W, r = H.double(), W.double(), torch.arange(H.shape[0], device=H.device)
    z = H @ W.T
    ez = (d / 16 + 2) * 4 * E * float((H.abs() @ W.abs().T).max())
    lse = torch.logsumexp(z, 1)
    p = torch.exp(z - lse[:, None])
    others = p.clone()
    others[r, t.long()] = 0
    R = others.sum(1)
    more = 2 * z_loss * lse  # dlse²
    G = others * (1 + more)[:, None]
    G[r, t.long()] = -R + more * p[r, t.long()]
    eg = U + 2 * ez + 2.0 ** -18
    size = eg * G.abs()
    near_one = (136 + V / 128) * E + 2 * E * lse.abs()
    size[r, t.long()] = eg * (R + (more * p[r, t.long()]).abs()) + near_one
    dH, dW = G @ W, G.T @ H
    return (R, (dH, size @ W.abs() + U * dH.abs() + 1e-37),
            (dW, size.T @ H.abs() + U * dW.abs() + 1e-37))


SHAPES = [(8, 5120, 3000), (40, 5120, 3000), (300, 2056, 2500)]


@pytest.mark.parametrize("M,d,V", SHAPES[:1])
@pytest.mark.parametrize("shift", [0.0, 12.0])
def test_the_bounds_say_something(M, d, V, shift):
    """They are a part of the gradient itself down to 1 - p = 1e-4."""
    R, (dH, bound), _ = _exact(*_inputs(M, d, V, shift, "cpu"), 0.0)
    share = bound.norm(dim=1) / dH.norm(dim=1)
    assert R.max() > 5e-3 and R.min() < 2e-6
    assert (share[R > 1e-3] < 0.06).all() and (share[R > 1e-4] < 0.25).all(), share


@gpu
@pytest.mark.parametrize("M,d,V", SHAPES)
@pytest.mark.parametrize("shift,z_loss", [(0.0, 0.0), (12.0, 0.0), (-20.0, 0.0), (12.0, 1e-4)])
@pytest.mark.parametrize("piece", [0, 512])
def test_gradients(M, d, V, shift, z_loss, piece):
    H, W, t = _inputs(M, d, V, shift)
    f = sb.cross_entropy(H, W, t, z_loss=z_loss, reduction="sum")
    b = sb.cross_entropy_backward(H, W, t, f["lse"], z_loss=z_loss, reduction="sum", piece=piece)
    R, *want = _exact(H, W, t, z_loss)
    for name, (value, bound) in zip(("dH", "dW"), want):
        off = (b[name].double() - value).abs()
        assert (off <= bound).all(), (name, float((off / bound).max()))


@gpu
def test_one_word_has_no_gradient():
    """With a vocabulary of one word p is 1 whatever its logit."""
    g = torch.Generator(device="cuda").manual_seed(1)
    H = torch.randn(50, 5120, generator=g, device="cuda").bfloat16()
    W = torch.randn(1, 5120, generator=g, device="cuda").bfloat16()
    t = torch.zeros(50, dtype=torch.int32, device="cuda")
    f = sb.cross_entropy(H, W, t, reduction="none")
    b = sb.cross_entropy_backward(H, W, t, f["lse"], reduction="none")
    for x in (f["loss"], b["dH"], b["dW"]):
        assert (x == 0).all()
