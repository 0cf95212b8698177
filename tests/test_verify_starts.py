"""Requests that do not begin in the first row: rows in front of starts[0] belong to no request.  They have no token,
and no draft rows; what follows is as it is without them (the draws go by the row's number, so the seed moves).

Log-probabilities: the rows' sums are cut into other pieces when rows move.  Each side is within
2^-22 (max|y| + |lse| + 4) of the definition (test_verify.py), here 2^-22 (12 + 12 + 4) for logits of deviation 2."""
import pytest
import torch

import gemm_epilogue_reduction_gb300 as sb
from test_verify import _make

gpu = pytest.mark.gpu
GOLDEN = 0x9E3779B97F4A7C15
BOUND = 2 * 2.0 ** -22 * 28


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gemm_epilogue_reduction_gb300 import build as sbbuild
    sbbuild.build()


def _filled(s):
    """The call in memory that held other answers before (what it does not write would show)."""
    R, V = s["logits"].shape
    B, D = s["starts"].shape[0] - 1, -1 if s["draft_logits"] is None else s["draft_logits"].shape[0]
    out = {"token": torch.full((R,), 77, dtype=torch.int32, device="cuda"),
           "accepted": torch.full((B,), 77, dtype=torch.int32, device="cuda"),
           "token_logprob": torch.full((R,), 77.0, device="cuda")}
    n = sb.sb_verify_workspace_bytes(R, D, V)
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    st = sb.sb_verify_drafts(s["logits"], s["draft_logits"], s["drafts"], s["starts"], s["uniforms"], None, None, R, D, B,
                             V, sb.SB_BF16, 1.0, s["seed"], *out.values(), ws, n)
    assert st == sb.SB_OK
    return out, sb.device_status(ws)


def _pushed(s, front):
    """The same requests behind `front` rows that are none's."""
    g = torch.Generator(device="cuda").manual_seed(1)
    V = s["logits"].shape[1]

    def behind(t, first):
        return torch.cat([first, t])

    return {"logits": behind(s["logits"], torch.randn(front, V, generator=g, device="cuda").bfloat16()),
            "draft_logits": s["draft_logits"], "starts": s["starts"] + front,
            "drafts": behind(s["drafts"], torch.zeros(front, dtype=torch.int32, device="cuda")),
            "uniforms": behind(s["uniforms"], torch.zeros(front, device="cuda")),
            "seed": (s["seed"] - front * V * GOLDEN) % 2 ** 64}


@gpu
@pytest.mark.parametrize("front", [1, 2, 7, 700])
@pytest.mark.parametrize("lengths", [[2], [3, 0, 5], [None, 2, None, 4], [1] * 200])
@pytest.mark.parametrize("draft", [True, False])
def test_rows_in_front_of_the_first_request(front, lengths, draft):
    s = {**_make(lengths, 1003, draft=draft, seed=front, behind=3), "seed": 12}
    want, status = _filled(s)
    assert status == sb.SB_OK
    got, status = _filled(_pushed(s, front))
    assert status == sb.SB_OK
    assert torch.equal(got["accepted"], want["accepted"])
    assert torch.equal(got["token"][front:], want["token"])
    assert (got["token_logprob"][front:] - want["token_logprob"]).abs().max() <= BOUND
    assert (got["token"][:front] == -1).all() and (got["token_logprob"][:front] == 0).all()


@gpu
def test_another_draft_row_is_not_taken():
    """More draft rows than drafts: the first ones are the requests'."""
    s = {**_make([2, 3], 333, seed=5), "seed": 3}
    want, _ = _filled(s)
    t = _pushed(s, 4)
    t["draft_logits"] = torch.cat([s["draft_logits"], torch.randn(20, 333, device="cuda").bfloat16()])
    got, status = _filled(t)
    assert status == sb.SB_OK and torch.equal(got["accepted"], want["accepted"])
    assert torch.equal(got["token"][4:], want["token"])
    assert (got["token_logprob"][4:] - want["token_logprob"]).abs().max() <= BOUND


@gpu
def test_requests_that_begin_in_front_of_the_first_are_refused():
    s = {**_make([2, 2, 2], 100, seed=6), "seed": 0}
    for starts, accepted in (([3, 6, 0, 9], [None, -1, -1]), ([6, 9, 0, 3], [-1, -1, -1]), ([9, 0, 3, 9], [-1, -1, -1]),
                             ([4, 4, 4, 4], [0, 0, 0])):
        t = dict(s, starts=torch.tensor(starts, dtype=torch.int32, device="cuda"))
        got, status = _filled(t)
        for have, want in zip(got["accepted"].tolist(), accepted):
            assert want is None or have == want, (starts, got["accepted"].tolist())
        assert status == (sb.SB_OK if accepted == [0, 0, 0] else sb.SB_ERR_INVALID_ARG)
        assert (got["token"][:min(starts[0], 9)] == -1).all()


@gpu
@pytest.mark.parametrize("front", [1, 33, 1000])
def test_greedy(front):
    i32 = torch.int32
    target = torch.tensor([5, 6, 7, 8, 1, 2, 9, 4, 4], dtype=i32, device="cuda")
    drafts = torch.tensor([5, 6, 0, 8, 1, 2, 9, 3, 4], dtype=i32, device="cuda")
    starts = torch.tensor([0, 4, 4, 6, 8], dtype=i32, device="cuda") + front
    first = torch.full((front,), 3, dtype=i32, device="cuda")
    R, token = front + 9, torch.full((front + 9,), 77, dtype=i32, device="cuda")
    accepted = torch.full((4,), 77, dtype=i32, device="cuda")
    assert sb.sb_verify_greedy(torch.cat([first, target]), torch.cat([first, drafts]), starts, R, 4, token,
                               accepted) == sb.SB_OK
    assert (token[:front] == -1).all()
    assert token[front:].tolist() == [5, 6, 7, -1, 1, 2, 9, 4, -1] and accepted.tolist() == [2, 0, 1, 1]
    bad = torch.tensor([front, front + 4, 0, 4, front + 8], dtype=i32, device="cuda")
    f = sb.verify_greedy(torch.cat([first, target]), torch.cat([first, drafts]), bad)
    assert f["accepted"].tolist()[1:3] == [-1, -1] and (f["token"][:front] == -1).all()
