"""Verification of very many requests, most of them without rows: which draft rows are a request's does not depend on
them, and what they cost does not grow with their square.

Log-probabilities: as in test_verify_starts.py (rows move where there are some in front)."""
import pytest
import torch

import gemm_epilogue_reduction_gb300 as sb
from test_verify import _make
from test_verify_starts import BOUND

gpu = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gemm_epilogue_reduction_gb300 import build as sbbuild
    sbbuild.build()


@gpu
@pytest.mark.parametrize("B,front", [(2047, 0), (2048, 0), (2049, 1), (4096, 0), (8193, 3), (50_001, 1), (1 << 20, 0), (1 << 24, 2)])
@pytest.mark.parametrize("draft", [True, False])
def test_requests_without_rows_in_between(B, front, draft):
    g = torch.Generator(device="cuda").manual_seed(B)
    s = _make([3, 0, 1, 2] * 25, 77, draft=draft, seed=2)
    want = sb.verify_drafts(**s, seed=9)
    at = torch.randperm(B, generator=g, device="cuda")[:100].sort().values  # which requests have rows
    rows = torch.zeros(B, dtype=torch.int32, device="cuda")
    rows[at] = s["starts"][1:] - s["starts"][:-1]
    starts = torch.cat([torch.zeros(1, dtype=torch.int32, device="cuda"), rows.cumsum(0).int()])
    t = dict(s, starts=starts + front)
    if front:
        for k in ("logits", "drafts", "uniforms"):
            t[k] = torch.cat([s[k][:front], s[k]])
    seed = (9 - front * 77 * 0x9E3779B97F4A7C15) % 2 ** 64
    f = sb.verify_drafts(**t, seed=seed)
    assert sb.device_status(f["workspace"]) == sb.SB_OK
    assert torch.equal(f["token"][front:], want["token"]) and torch.equal(f["accepted"][at], want["accepted"])
    assert (f["token_logprob"][front:] - want["token_logprob"]).abs().max() <= BOUND
    assert int(f["accepted"].abs().sum()) == int(want["accepted"].sum())


@gpu
def test_no_draft_rows_at_all():
    """Draft logits without a row: requests of one row each, and one whose draft has no row."""
    B, V = 1 << 23, 5
    R = 1000
    g = torch.Generator(device="cuda").manual_seed(1)
    z = torch.randn(R, V, generator=g, device="cuda")
    starts = torch.full((B + 1,), R, dtype=torch.int32, device="cuda")
    starts[:R - 1] = torch.arange(R - 1, device="cuda")
    s = (z, torch.zeros(R, dtype=torch.int32, device="cuda"), starts, torch.zeros(R, device="cuda"))
    f = sb.verify_drafts(*s, draft_logits=z[:0], seed=3)
    assert sb.device_status(f["workspace"]) == sb.SB_ERR_INVALID_ARG  # rows 998 and 999: a draft
    want = sb.verify_drafts(*s, seed=3)
    assert torch.equal(f["token"][:R - 2], want["token"][:R - 2])
    assert int(f["accepted"][R - 2]) == -1 and int(f["accepted"].abs().sum()) == 1
