"""A captured verification step draws other numbers in every replay: seed_offset, a counter on the device, is added to
the seed when the kernels run."""
import pytest
import torch

import gemm_epilogue_reduction_gb300 as sb
from test_verify import _check, _make

gpu = pytest.mark.gpu
NAMES = ("token", "accepted", "token_logprob")


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gemm_epilogue_reduction_gb300 import build as sbbuild
    sbbuild.build()


@gpu
@pytest.mark.parametrize("draft", [True, False])
def test_replays_with_a_counter(draft):
    s = _make([4, 0, 1, 7] * 8, 5003, draft=draft, seed=1)
    step = torch.zeros(1, dtype=torch.int64, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        f = sb.verify_drafts(**s, seed=2 ** 64 - 2, seed_offset=step)
        step += 1
    seen = []
    for k in range(4):  # the sum of seed and counter wraps
        graph.replay()
        torch.cuda.synchronize()
        want = _check(s, seed=(2 ** 64 - 2 + k) % 2 ** 64)
        assert all(torch.equal(f[n], want[n]) for n in NAMES), k
        seen.append(f["token"].clone())
    assert not any(torch.equal(seen[0], x) for x in seen[1:])


@gpu
def test_streams_and_types():
    s = _make([3, 2], 777, seed=2)
    off = torch.tensor([41], device="cuda")
    want = sb.verify_drafts(**s, seed=42)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for kw in ({}, {"stream": side}, {"stream": side.cuda_stream}):
        for o in (off, off.view(torch.uint64)):
            got = sb.verify_drafts(**s, seed=1, seed_offset=o, **kw)
            torch.cuda.synchronize()
            assert all(torch.equal(got[n], want[n]) for n in NAMES)
    with pytest.raises(TypeError):
        sb.verify_drafts(**s, seed_offset=off.int())
    with pytest.raises(ValueError):
        sb.verify_drafts(**s, seed_offset=off.cpu())
    with pytest.raises(ValueError):
        sb.verify_drafts(**s, seed_offset=off.expand(2))


def test_c_refusals():
    MB = 1 << 20
    names = ("z", "q", "drafts", "starts", "u", "lse", "qlse", "off", "token", "accepted", "lp", "ws")
    P = {k: (i + 1) * MB for i, k in enumerate(names)}

    def call(**kw):
        a = {**P, **kw}
        return sb.sb_verify_drafts(a["z"], a["q"], a["drafts"], a["starts"], a["u"], a["lse"], a["qlse"], 8, 6, 2, 512, 0,
                                   1.0, 0, a["token"], a["accepted"], a["lp"], a["ws"], 16, 0, seed_offset=a["off"])

    assert call(off=P["off"] + 4) == sb.SB_ERR_ALIGNMENT
    for out in ("token", "accepted", "lp", "ws"):
        assert call(off=P[out]) == sb.SB_ERR_INVALID_ARG, out
    assert call(token=P["off"] - 7 * 4) == sb.SB_ERR_INVALID_ARG
    for kw in ({}, {"off": None}):
        assert call(**kw) not in (sb.SB_OK, sb.SB_ERR_INVALID_ARG, sb.SB_ERR_ALIGNMENT)
