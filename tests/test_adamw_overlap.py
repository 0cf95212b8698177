"""Tensors that share memory are refused: two blocks of a launch would write it."""
import pytest
import torch

import gemm_epilogue_reduction_gb300 as sb

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


def test_overlapping_tensors_are_refused():
    p, q = torch.zeros(512, device="cuda"), torch.zeros(512, device="cuda")
    with pytest.raises(ValueError, match="overlap"):
        sb.AdamW([p, q, p])
    with pytest.raises(ValueError, match="overlap"):
        sb.AdamW([p[:300], p[299:]])
    with pytest.raises(ValueError, match="overlap"):
        sb.AdamW([p], states=[(q, q)])
    with pytest.raises(ValueError, match="overlap"):
        sb.AdamW([p.bfloat16(), q.bfloat16()], masters=[p, p])
    sb.AdamW([p[:256], p[256:], q[:0], q[:0], q])  # neighbours and empty tensors
