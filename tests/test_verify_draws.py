"""Samples of verification whose draws are chosen: SplitMix64 is one to one, so there is a seed for every
value of a draw.  A uniform of 0 (one draw in 2^24) gives a score of 0, which wins only where no other column
has any weight: a row with a finite logit always has a sample."""
import numpy as np
import pytest
import torch

import gemm_epilogue_reduction_gb300 as sb
from test_dropout import splitmix

gpu = pytest.mark.gpu
MASK = (1 << 64) - 1
GOLDEN = 0x9E3779B97F4A7C15


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gemm_epilogue_reduction_gb300 import build as sbbuild
    sbbuild.build()


def seed_for(n, value):
    """The seed whose draw n is `value`."""
    def undo(x, k):  # y = x ^ (x >> k)
        y = x
        for _ in range(64 // k + 1):
            y = x ^ (y >> k)
        return y & MASK

    x = undo(value, 31) * pow(0x94D049BB133111EB, -1, 1 << 64) & MASK
    x = undo(x, 27) * pow(0xBF58476D1CE4E5B9, -1, 1 << 64) & MASK
    return (undo(x, 30) - (n + 1) * GOLDEN) & MASK


def test_the_seed_of_a_draw():
    for n, value in ((0, 0), (5, 0), (10 ** 12, 123456789), (7, MASK)):
        assert int(splitmix(np.array([n], dtype=np.uint64), seed_for(n, value))[0]) == value


def _one(z, column, u=0.0, x=0, q=None, T=1.0, row=0, more=0):
    """A request whose draw of `column` in row `row` is 0; rows before it are requests of their own."""
    R, V = row + more + 1, len(z)
    logits = torch.tensor([z] * R, dtype=torch.float32, device="cuda")
    starts = list(range(row + 1)) + [R]
    f = sb.verify_drafts(logits, torch.full((R,), x, dtype=torch.int32, device="cuda"),
                         torch.tensor(starts, dtype=torch.int32, device="cuda"),
                         torch.full((R,), u, device="cuda"), temperature=T, seed=seed_for(row * V + column, 0),
                         draft_logits=None if q is None else torch.tensor([q] * more, dtype=torch.float32, device="cuda"))
    assert sb.device_status(f["workspace"]) == sb.SB_OK
    return int(f["accepted"][-1]), int(f["token"][row]), float(f["token_logprob"][row])


INF = float("inf")


@gpu
@pytest.mark.parametrize("V", [1, 5, 300, 5001])
@pytest.mark.parametrize("row", [0, 3])
def test_the_only_column(V, row):
    """One column with probability, at the front, in the middle and at the end of a row."""
    for j in {0, V // 2, V - 1}:
        z = [-INF] * V
        z[j] = 2.5
        assert _one(z, j, row=row) == (0, j, 0.0)


@gpu
@pytest.mark.parametrize("V", [40, 5001])
def test_a_column_beside_others_too_small_for_fp32(V):
    for j in (0, V // 2, V - 1):
        z = [0.0] * V
        z[j] = 1.0
        assert _one(z, j, T=1e-3) == (0, j, 0.0)


@gpu
def test_the_only_column_of_a_difference():
    """p = (.6, .4), q = (.4, .6), the draft 1 refused: column 0 is all that is left, whatever its draw."""
    p, q = np.log([0.6, 0.4]).tolist(), np.log([0.4, 0.6]).tolist()
    accepted, token, lp = _one(p, 0, u=0.9, x=1, q=q, more=1)
    assert (accepted, token) == (0, 0) and abs(lp - np.log(0.6)) < 1e-6
    # without q: the other one of two columns
    accepted, token, _ = _one(p, 0, u=0.9, x=1, more=1)
    assert (accepted, token) == (0, 0)


@gpu
def test_a_score_of_zero_loses_to_any_other():
    z = [0.0] * 300
    z[7] = 60.0  # all others together: 3e-24
    accepted, token, _ = _one(z, 7)
    bits = splitmix(np.arange(300, dtype=np.uint64), seed_for(7, 0)) >> np.uint64(40)
    score = 1 / -np.log(np.maximum(bits.astype(np.float64), 0.5) * 2.0 ** -24)
    score[7] = 0
    assert accepted == 0 and token == int(np.argmax(score))


@gpu
@pytest.mark.parametrize("V", [7, 1003, 4096])
@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32])
def test_a_difference_that_is_nowhere_positive(V, kind):
    """Equal distributions and a refused draft: the sample is of p itself, the refused column among the others.
    Weights are off by 2^-19 at most, scores by as much again."""
    B, seed = 40, 4
    g = torch.Generator(device="cuda").manual_seed(V)
    z = (2 * torch.randn(2 * B, V, generator=g, device="cuda")).to(kind)
    lse = torch.logsumexp(z.double(), 1).float()
    q = z[::2].contiguous()
    drafts = torch.zeros(2 * B, dtype=torch.int32, device="cuda")
    drafts[::2] = z[::2].float().argmax(1).int()
    f = sb.verify_drafts(z, drafts, torch.arange(0, 2 * B + 1, 2, dtype=torch.int32, device="cuda"),
                         torch.full((2 * B,), 2.0, device="cuda"), draft_logits=q, lse=lse,
                         draft_lse=lse[::2].contiguous(), seed=seed)
    assert (f["accepted"] == 0).all() and (f["token"][1::2] == -1).all()
    sure = again = 0
    for b in range(B):
        r = 2 * b
        y = z[r].double().cpu().numpy()
        bits = (splitmix(np.arange(r * V, (r + 1) * V, dtype=np.uint64), seed) >> np.uint64(40)).astype(np.float64)
        score = np.exp(y - y.max()) / -np.log(bits * 2.0 ** -24)
        best = np.sort(score)[-2:]
        if best[0] < best[1] * (1 - 2.0 ** -17):
            sure += 1
            assert int(f["token"][r]) == int(np.argmax(score)), b
            again += int(f["token"][r]) == int(drafts[r])
            assert abs(float(f["token_logprob"][r]) - (y[int(f["token"][r])] - float(lse[r]))) < 1e-5
    assert sure >= B - 2
    assert V > 7 or again > 0  # (a likely column: p allows it, p without it would not)
