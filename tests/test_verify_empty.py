"""Verification without requests: the status that the workspace's header holds is this call's."""
import pytest
import torch

import gemm_epilogue_reduction_gb300 as sb
from test_verify import _make

gpu = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gemm_epilogue_reduction_gb300 import build as sbbuild
    sbbuild.build()


@gpu
def test_an_empty_call_has_a_status_of_its_own():
    s = _make([2], 50, seed=3)
    ws = torch.zeros(1 << 16, dtype=torch.uint8, device="cuda")
    sb.verify_drafts(**dict(s, drafts=s["drafts"] * 0 - 1), workspace=ws)
    assert sb.device_status(ws) == sb.SB_ERR_INVALID_ARG
    none = _make([], 50)
    f = sb.verify_drafts(**none, workspace=ws)
    assert f["accepted"].shape == (0,) and f["token"].shape == (0,)
    assert sb.device_status(ws) == sb.SB_OK
