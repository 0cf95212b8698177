"""The lookup's gradient with a workspace over its inputs, on made-up addresses: none is launched (what is not refused
for its addresses has a workspace that is too small)."""
import pytest

import gemm_epilogue_reduction_gb300 as sb

MB = 1 << 20
IDS, DOUT, DW, WS = (k * MB for k in range(1, 5))


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gemm_epilogue_reduction_gb300 import build as sbbuild
    sbbuild.build()


@pytest.mark.parametrize("M,d,V", [(4, 64, 100), (300, 24, 1000)])
def test_the_workspace_over_an_input(M, d, V):
    size = sb.sb_embedding_backward_workspace_bytes(M, d)

    def call(ws):
        return sb.sb_embedding_backward(IDS, DOUT, M, d, V, -100, 1.0, 0, 0, 1, DW, ws, 256, 0)

    for at, n in ((IDS, 4 * M), (DOUT, 2 * M * d), (DW, 2 * V * d)):
        for ws in {at, at + (n - 1) // 256 * 256, at - (size - 1) // 256 * 256}:
            assert call(ws) == sb.SB_ERR_INVALID_ARG, (at // MB, ws - at)
        behind = (at + n + 255) // 256 * 256
        assert call(behind) not in (sb.SB_OK, sb.SB_ERR_INVALID_ARG, sb.SB_ERR_ALIGNMENT)
