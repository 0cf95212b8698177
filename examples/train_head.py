"""Training the tail of a language model: the last residual sum and norm, the output head and its
loss, their gradients, and an AdamW step over head, norms and gate.

    python examples/train_head.py [--steps 60] [--tokens 512] [--d 640] [--vocab 5000] [--bits 8]

The data stand in for what the frozen blocks below would deliver: every token has the residual
stream h and the last block's output y, and its label is the nearest of a set of hidden
directions, so the head has something to learn. Some labels are ignored, as padding is.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gemm_epilogue_reduction_gb300 as sb  # noqa: E402

IGNORE = -100


class Tail:
    """The weights, their 32-bit copies and the optimizer of the model's tail."""

    def __init__(self, d: int, vocab: int, *, bits: int, lr: float, seed: int):
        g = torch.Generator(device="cuda").manual_seed(seed)
        W = torch.randn(vocab, d, generator=g, device="cuda") * d ** -0.5
        ones = torch.ones(d, device="cuda")
        self.copies = [W, ones.clone(), ones.clone(), 0.5 * ones]
        self.W, self.pre, self.post, self.gate = (c.bfloat16() for c in self.copies)
        # the head decays, the vectors do not
        self.opt = sb.AdamW([self.W, self.pre, self.post, self.gate], masters=self.copies, lr=lr,
                            betas=(0.9, 0.95), weight_decay=[0.1, 0.0, 0.0, 0.0], state_bits=bits)

    def step(self, h, y, targets):
        """One training step; returns the loss (on the device) and the gradients that the blocks
        below would go on with."""
        norm = {"post": self.post, "gate": self.gate}
        f = sb.residual_norm(h, y, self.pre, **norm)
        loss = sb.cross_entropy(f["x"], self.W, targets, ignore_index=IGNORE, z_loss=1e-4)
        back = sb.cross_entropy_backward(f["x"], self.W, targets, loss["lse"], ignore_index=IGNORE,
                                         z_loss=1e-4)
        # nothing but the head reads the last residual stream: its own gradient is none
        below = sb.residual_norm_backward(back["dH"], None, f["h"], y, self.pre, **norm)
        self.opt.step([back["dW"], below["dpre"], below["dpost"], below["dgate"]])
        return loss["loss"], below["dh"], below["dy"]

    def tokens(self, h, y):
        """What the trained tail answers with: the most likely token of every row."""
        x = sb.residual_norm(h, y, self.pre, post=self.post, gate=self.gate)["x"]
        return sb.project(x, self.W, 1, sb.SB_TOKEN)["token"]


def batches(d: int, vocab: int, tokens: int, seed: int):
    """Endless (h, y, targets): the label is the best of `vocab` fixed directions for h + y."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    way = torch.randn(vocab, d, generator=g, device="cuda")
    while True:
        label = torch.randint(0, vocab, (tokens,), generator=g, device="cuda")
        mean = 0.5 * way[label]
        h = (mean + torch.randn(tokens, d, generator=g, device="cuda")).bfloat16()
        y = (mean + torch.randn(tokens, d, generator=g, device="cuda")).bfloat16()
        targets = label.int()
        targets[::16] = IGNORE
        yield h, y, targets


def train(steps: int = 60, tokens: int = 512, d: int = 640, vocab: int = 5000, bits: int = 8,
          lr: float = 3e-3, seed: int = 0, every: int = 10):
    """Trains for `steps` steps; returns the losses and the share of right tokens at the end."""
    tail = Tail(d, vocab, bits=bits, lr=lr, seed=seed)
    data = batches(d, vocab, tokens, seed + 1)
    losses = []
    for i in range(steps):
        losses.append(tail.step(*next(data))[0])
        if every and (i + 1) % every == 0:
            print(f"step {i + 1}: loss {losses[-1].item():.4f}", flush=True)
    h, y, targets = next(data)
    right = (tail.tokens(h, y) == targets)[targets != IGNORE].float().mean()
    return [float(x) for x in torch.cat(losses)], float(right)


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, value in (("steps", 60), ("tokens", 512), ("d", 640), ("vocab", 5000), ("bits", 8)):
        ap.add_argument(f"--{name}", type=int, default=value)
    a = ap.parse_args()
    from gemm_epilogue_reduction_gb300 import build
    build.build()
    _, right = train(a.steps, a.tokens, a.d, a.vocab, a.bits)
    print(f"right tokens: {100 * right:.1f} %")
