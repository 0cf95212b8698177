"""An ignored index that no 32-bit target can equal is refused: cut to 32 bits it would be another."""
import pytest
import torch

import gemm_epilogue_reduction_gb300 as sb
from gemm_epilogue_reduction_gb300 import synth

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


@pytest.mark.parametrize("index", [2 ** 32 + 5, -2 ** 63, 2 ** 31])
def test_refused(index):
    H, W = synth.make_hw(8, 64, 300, seed=1, device="cuda")
    t = torch.full((8,), index & 0x7F, dtype=torch.int32, device="cuda")
    lse = torch.zeros(8, device="cuda")
    with pytest.raises(ValueError, match="ignore_index"):
        sb.cross_entropy(H, W, t, ignore_index=index)
    with pytest.raises(ValueError, match="ignore_index"):
        sb.cross_entropy_backward(H, W, t, lse, ignore_index=index)


@pytest.mark.parametrize("index", [2 ** 31 - 1, -2 ** 31])
def test_the_ends_of_the_range(index):
    H, W = synth.make_hw(8, 64, 300, seed=1, device="cuda")
    t = torch.full((8,), index, dtype=torch.int32, device="cuda")
    assert float(sb.cross_entropy(H, W, t, ignore_index=index)["loss"]) == 0
