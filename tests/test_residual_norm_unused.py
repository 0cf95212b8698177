"""Arguments of the residual norm that a call does not use may hold anything."""
import pytest
import torch

import gemm_epilogue_reduction_gb300 as sb


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gemm_epilogue_reduction_gb300 import build as sbbuild
    sbbuild.build()


def test_gate_address_without_a_gate():
    P = 1 << 20  # nothing is read: there are no rows
    status = sb.sb_residual_norm_forward(P, P, P, None, 1, sb.SB_GATE_NONE, 0, 64, sb.SB_BF16,
                                         sb.SB_F32, 1.0, 1e-6, P, P, 0)
    assert status not in (sb.SB_ERR_ALIGNMENT, sb.SB_ERR_INVALID_ARG)


@pytest.mark.gpu
def test_unused_addresses():
    M, d = 20, 72
    h, y, dx = (torch.randn(M, d, device="cuda").bfloat16() for _ in range(3))
    pre = torch.randn(d, device="cuda")
    want = sb.residual_norm(h, y, pre)
    back = sb.residual_norm_backward(dx, None, want["h"], y, pre)
    ho, x, dho, dy, dpre = (torch.empty_like(t) for t in (h, y, h, y, pre))
    shape = (sb.SB_GATE_NONE, M, d, sb.SB_BF16, sb.SB_F32, 1.0, 1e-6)
    assert sb.sb_residual_norm_forward(h, y, pre, None, 1, *shape, ho, x) == sb.SB_OK
    n = sb.sb_residual_norm_workspace_bytes(M, d)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    assert sb.sb_residual_norm_backward(dx, None, ho, y, pre, None, 1, *shape, dho, dy, dpre, 3, 1,
                                        ws, n) == sb.SB_OK
    for a, b in ((ho, want["h"]), (x, want["x"]), (dho, back["dh"]), (dy, back["dy"]),
                 (dpre, back["dpre"])):
        assert torch.equal(a, b)
