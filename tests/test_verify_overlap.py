"""Verification calls whose outputs lie over other arrays: blocks of a request, and other requests, still read what one
of them writes.  The refused calls are never launched; the one form in place that is allowed is compared."""
import pytest
import torch

import gemm_epilogue_reduction_gb300 as sb

gpu = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gemm_epilogue_reduction_gb300 import build as sbbuild
    sbbuild.build()


R, D, B, V = 8, 6, 2, 512
MB = 1 << 20
# arrays a megabyte apart, with their sizes in bytes
INPUTS = {"z": R * V * 2, "q": D * V * 2, "drafts": R * 4, "starts": (B + 1) * 4, "u": R * 4, "lse": R * 4, "qlse": D * 4}
OUTPUTS = {"token": R * 4, "accepted": B * 4, "lp": R * 4, "ws": 0}
PLACE = {k: (i + 1) * MB for i, k in enumerate([*INPUTS, *OUTPUTS])}


def _call(n=None, **kw):
    """On made-up addresses: only with a workspace that is too small, or refused before that."""
    a = {**PLACE, **kw}
    size = sb.sb_verify_workspace_bytes(R, D, V)
    return sb.sb_verify_drafts(a["z"], a["q"], a["drafts"], a["starts"], a["u"], a["lse"], a["qlse"], R, D, B, V, 0, 1.0, 0,
                               a["token"], a["accepted"], a["lp"], a["ws"], size - 1 if n is None else n, 0)


def test_outputs_over_inputs():
    size = sb.sb_verify_workspace_bytes(R, D, V)
    for out, n in OUTPUTS.items():
        n = n or size
        for name, m in INPUTS.items():
            at, step = PLACE[name], 256 if out == "ws" else 4
            last = at + (m - 1) // step * step  # the array's last place, and the last one in front that reaches it
            first = at - (n - 1) // step * step
            for p in {at, last, first}:
                if out == "token" and name == "drafts" and p == at:
                    continue
                assert _call(**{out: p}) == sb.SB_ERR_INVALID_ARG, (out, name, p - at)


def test_outputs_over_each_other():
    for a in OUTPUTS:
        for b in OUTPUTS:
            if a != b:
                assert _call(**{a: PLACE[b]}) == sb.SB_ERR_INVALID_ARG, (a, b)
    assert _call(ws=PLACE["token"] - 256) == sb.SB_ERR_INVALID_ARG


def test_neighbours_are_not_refused():
    """Arrays that touch: these calls get as far as the workspace's size (or the missing device)."""
    for kw in ({}, {"token": PLACE["drafts"]}, {"token": PLACE["drafts"] + R * 4}, {"token": PLACE["u"] - R * 4},
               {"accepted": PLACE["starts"] + (B + 1) * 4}, {"lp": PLACE["z"] + R * V * 2},
               {"token": PLACE["accepted"] - R * 4}, {"ws": PLACE["q"] + D * V * 2}, {"lse": None, "qlse": None, "lp": None}):
        assert _call(**kw) not in (sb.SB_OK, sb.SB_ERR_INVALID_ARG, sb.SB_ERR_ALIGNMENT), kw
    # memory behind what a call needs is not the workspace's
    size = sb.sb_verify_workspace_bytes(R, D, V)
    assert _call(ws=PLACE["z"] - (size + 255) // 256 * 256) != sb.SB_ERR_INVALID_ARG


def test_greedy_outputs_over_inputs():
    P = {k: (i + 1) * MB for i, k in enumerate(("target", "drafts", "starts", "token", "accepted"))}

    def call(**kw):
        a = {**P, **kw}
        return sb.sb_verify_greedy(a["target"], a["drafts"], a["starts"], R, B, a["token"], a["accepted"], 0)

    for kw in ({"token": P["target"] + 4}, {"token": P["drafts"] - 4}, {"token": P["starts"] + 8},
               {"token": P["starts"] - R * 4 + 4}, {"accepted": P["starts"]}, {"accepted": P["starts"] + 8},
               {"accepted": P["target"] + R * 4 - 4}, {"accepted": P["drafts"]}, {"accepted": P["token"]},
               {"token": P["accepted"] + 4}):
        assert call(**kw) == sb.SB_ERR_INVALID_ARG, kw


@gpu
def test_tokens_over_their_drafts():
    """In place, as often as a race would need to show."""
    g = torch.Generator(device="cuda").manual_seed(0)
    n, v = 400, 5003
    z = (2 * torch.randn(n, v, generator=g, device="cuda")).bfloat16()
    drafts = z.float().argmax(1).int()
    starts = torch.arange(0, n + 1, 5, dtype=torch.int32, device="cuda")
    u = torch.rand(n, generator=g, device="cuda") * 0.2
    want = sb.verify_drafts(z, drafts, starts, u, seed=3)
    size = sb.sb_verify_workspace_bytes(n, -1, v)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    greedy = sb.verify_greedy(want["token"], drafts, starts)
    for _ in range(20):
        t, accepted = drafts.clone(), torch.empty(80, dtype=torch.int32, device="cuda")
        assert sb.sb_verify_drafts(z, None, t, starts, u, None, None, n, -1, 80, v, 0, 1.0, 3, t, accepted, None, ws,
                                   size) == sb.SB_OK
        assert torch.equal(t, want["token"]) and torch.equal(accepted, want["accepted"])
        for target, old in ((want["token"], drafts.clone()), (want["token"].clone(), drafts)):
            t = old if old is not drafts else target
            assert sb.sb_verify_greedy(target, old, starts, n, 80, t, accepted) == sb.SB_OK
            assert torch.equal(t, greedy["token"]) and torch.equal(accepted, greedy["accepted"])
