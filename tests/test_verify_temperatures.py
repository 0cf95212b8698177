"""Verification at every temperature that is accepted, against the definition in 64 bits.

The reference takes each row's exponents from its largest logit, (z - max) / T with T = 1 / fp32(1 / T), so
that nothing of the size of z / T is ever rounded.  The kernel's exponents of columns that count (|log p| below
some 100) are sums of two fp32 terms, off by at most 2^-22 of their magnitude, and hold ex2's 2^-22 and the
logarithm of a sum of such terms: a log-probability l is off by D = 2^-21 (|l| + log V + 4), a weight p by D p
(|l| p has its largest value at small |l|; beyond 100 p adds nothing).  A score w / -log u is off by that and by
2^-19.  log p/q is formed in 64 bits but for the two sums' logarithms: off by A = 2^-21 (2 log V + 8) and 2^-50 of
itself.  Where a decision is nearer than that to its border the rest of the request is not compared.
"""
import numpy as np
import pytest
import torch

import gemm_epilogue_reduction_gb300 as sb
from test_dropout import splitmix

gpu = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gemm_epilogue_reduction_gb300 import build as sbbuild
    sbbuild.build()


def _logs(z, inv_t):
    """log p of a row, in 64 bits, what the kernel's may be off by, and the logarithm of the sum in it."""
    y = (z - z.max()) * inv_t
    total = np.log(np.exp(y).sum())
    return y - total, 2.0 ** -21 * (np.abs(y - total) + np.log(len(z)) + 4), total


def _weights(lp, off):
    p = np.exp(lp)
    return p, np.where(lp > -200, off, 0) * p


def _answer(z, q, drafts, u, row, T, seed):
    """One request's rows: the tokens with their log-probabilities, None from where it is ambiguous."""
    inv_t = float(np.float32(1) / np.float32(T))
    V, n, out = z.shape[1], len(drafts), []
    for i in range(n + 1):
        lp, off, total = _logs(z[i], inv_t)
        w, dw = _weights(lp, off)
        if i < n:
            x = drafts[i]
            ratio = lp[x]
            if q is not None:
                lq, qoff, qtotal = _logs(q[i], inv_t)
                ratio = ((z[i, x] - z[i].max()) - (q[i, x] - q[i].max())) * inv_t - (total - qtotal)
            if abs(ratio - np.log(u[i])) <= 2.0 ** -21 * (2 * np.log(V) + 8) + 2.0 ** -50 * abs(ratio):
                return out + [None]
            if ratio > np.log(u[i]):
                out.append((x, lp[x], off[x]))
                continue
            if q is None:
                w[x] = 0
            else:
                v, dv = _weights(lq, qoff)
                w, dw = np.maximum(w - v, 0), dw + dv
        if w.max() <= 0:
            w, dw = _weights(lp, off)
        bits = (splitmix(np.arange((row + i) * V, (row + i + 1) * V, dtype=np.uint64), seed) >>
                np.uint64(40)).astype(np.float64)
        with np.errstate(divide="ignore"):
            t = -np.log(bits * 2.0 ** -24)
        score, low, high = w / t, (w - dw) / t * (1 - 2.0 ** -19), (w + dw) / t * (1 + 2.0 ** -19)
        j = int(np.argmax(score))
        rivals = (high >= low[j]) & (np.arange(V) != j)
        return out + [None if rivals.any() else (j, lp[j], off[j])]


def _make(lengths, V, kind, draft, seed, lowest):
    """Logits in steps of a half, so that several columns share the largest; the drafts are columns that are likely
    under either distribution."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    R, D = sum(n + 1 for n in lengths), sum(lengths)

    def logits(rows):
        x = (torch.round(8 * torch.randn(rows, V, generator=g, device="cuda")) / 2).to(kind)
        if lowest:
            x[:, ::7] = torch.finfo(kind).min
        return x

    z, q = logits(R), logits(D)
    starts = np.concatenate([[0], np.cumsum([n + 1 for n in lengths])])
    at = torch.tensor([int(starts[b]) + i for b, n in enumerate(lengths) for i in range(n)], device="cuda")
    same = torch.rand(D, generator=g, device="cuda") < 0.7  # the draft's largest columns are the target's
    q[same] = z[at[same]]
    drafts = torch.zeros(R, dtype=torch.int32, device="cuda")
    drafts[at] = torch.where(torch.rand(D, generator=g, device="cuda") < 0.8, q.float().argmax(1), 3).int()
    return {"logits": z, "draft_logits": q if draft else None, "drafts": drafts,
            "starts": torch.tensor(starts, dtype=torch.int32, device="cuda"),
            "uniforms": 0.01 + 0.98 * torch.rand(R, generator=g, device="cuda")}


TEMPERATURES = [1e-30, 1e-25, 7e-20, 1e-18, 1e-17, 1e-16, 1e-15, 1e-12, 1e-6, 1e-3, 0.3, 30.0, 1e10, 1e30, 3e37, 3e38]


@gpu
@pytest.mark.parametrize("T", TEMPERATURES)
@pytest.mark.parametrize("kind", [BF, F32])
@pytest.mark.parametrize("draft", [True, False])
@pytest.mark.parametrize("lowest", [False, True])
def test_every_temperature(T, kind, draft, lowest):
    lengths, V = [3, 0, 5, 1] * 6, 1003
    s = _make(lengths, V, kind, draft, 5, lowest)
    f = sb.verify_drafts(**s, temperature=T, seed=31)
    assert sb.device_status(f["workspace"]) == sb.SB_OK
    token, accepted, lp = f["token"].tolist(), f["accepted"].tolist(), f["token_logprob"].tolist()
    z = s["logits"].double().cpu().numpy()
    q = s["draft_logits"].double().cpu().numpy() if draft else None
    drafts, u = s["drafts"].tolist(), s["uniforms"].double().tolist()
    sure = at = row = 0
    for b, n in enumerate(lengths):
        assert token[row + accepted[b]] >= 0 and not np.isnan(lp[row + accepted[b]])
        want = _answer(z[row:row + n + 1], q[at:at + n] if draft else None, drafts[row:row + n], u[row:row + n], row,
                       T, 31)
        for i, w in enumerate(want):
            if w is None:
                break
            assert token[row + i] == w[0], (b, i)
            assert abs(lp[row + i] - w[1]) <= w[2] + 2.0 ** -23 * abs(w[1]), (b, i)
        else:
            sure += 1
            assert accepted[b] == len(want) - 1
        row, at = row + n + 1, at + n
    assert sure >= 0.8 * len(lengths)


@gpu
@pytest.mark.parametrize("T", [1.0, 1e30, 3e37, 3e38])
def test_given_logsumexps_at_high_temperatures(T):
    """T times the logsumexp leaves fp32's range long before the logsumexp does."""
    s = _make([2, 0, 4] * 5, 517, BF, True, 6, False)
    inv_t = float(np.float32(1) / np.float32(T))
    lse = torch.logsumexp(s["logits"].double() * inv_t, 1).float()
    qlse = torch.logsumexp(s["draft_logits"].double() * inv_t, 1).float()
    want = sb.verify_drafts(**s, temperature=T, seed=8)
    got = sb.verify_drafts(**s, temperature=T, seed=8, lse=lse, draft_lse=qlse)
    assert torch.equal(got["accepted"], want["accepted"]) and torch.equal(got["token"], want["token"])
    assert (got["token_logprob"] - want["token_logprob"]).abs().max() <= 2.0 ** -20 * 25
