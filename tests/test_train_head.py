"""The training operators together, as examples/train_head.py runs them: the loss falls, both
state widths learn alike, and one step's gradients are those of the whole tail in 64 bits."""
import os
import sys

import pytest
import torch

import gemm_epilogue_reduction_gb300 as sb

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                "examples"))


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


@pytest.mark.parametrize("bits", [32, 8])
def test_training_lowers_the_loss(bits):
    import train_head
    losses, right = train_head.train(steps=60, tokens=512, d=320, vocab=500, bits=bits, every=0)
    assert all(x == x for x in losses)
    # from a uniform guess (ln 500 = 6.2) the head learns the directions: each label is seen some
    # 57 times, and h + y holds its direction at a length of sqrt(320) against noise of sqrt(2)
    # per channel
    assert losses[0] > 5.5 and losses[-1] < 0.5 * losses[0]
    assert right > 0.5


def test_gradients_of_the_whole_tail():
    """dh, dy and the weights' gradients through norm, head and loss against autograd in 64 bits.
    Between the kernels x and dH are rounded to bf16 (2^-8 relative each, 2^-9 rms), so a
    gradient, as a sum of products with them, is within 2 % of its norm."""
    import train_head
    d, V, M = 264, 700, 90
    tail = train_head.Tail(d, V, bits=32, lr=0.0, seed=3)
    h, y, t = next(train_head.batches(d, V, M, 4))
    norm = {"post": tail.post, "gate": tail.gate}
    f = sb.residual_norm(h, y, tail.pre, **norm)
    ce = sb.cross_entropy(f["x"], tail.W, t, z_loss=1e-4)
    b = sb.cross_entropy_backward(f["x"], tail.W, t, ce["lse"], z_loss=1e-4)
    n = sb.residual_norm_backward(b["dH"], None, f["h"], y, tail.pre, **norm)

    leaf = [x.double().requires_grad_() for x in (h, y, tail.W, tail.pre, tail.post, tail.gate)]
    H, Y, W, pre, post, gate = leaf

    def rms(x):
        return x / torch.sqrt((x * x).mean(1, keepdim=True) + 1e-6)

    x = rms(H + gate * post * rms(Y)) * pre
    z = x @ W.T
    lse = torch.logsumexp(z, 1)
    keep = t >= 0
    rows = lse - z[torch.arange(M, device="cuda"), t.clamp(min=0).long()] + 1e-4 * lse ** 2
    loss = rows[keep].mean()
    value = float(loss.detach())
    assert abs(float(ce["loss"]) - value) <= 2e-2 * value
    grads = torch.autograd.grad(loss, leaf)
    for name, got, want in zip(("dh", "dy", "dW", "dpre", "dpost", "dgate"),
                               (n["dh"], n["dy"], b["dW"], n["dpre"], n["dpost"], n["dgate"]),
                               grads):
        off = (got.double() - want).norm() / want.norm()
        assert off <= 2e-2, (name, float(off))
