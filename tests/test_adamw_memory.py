"""The memory that an AdamW handle's kernel reads and writes is not handed out to others."""
import pytest
import torch

import gemm_epilogue_reduction_gb300 as sb

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


@pytest.mark.parametrize("which", ["param", "master", "state", "gradient"])
def test_memory_is_not_handed_out_while_the_handle_lives(which):
    """A tensor that is given other memory (`.data = ...`) leaves the handle with the old one."""
    n = 1_234_567  # a size of its own in the allocator
    p, w, g = torch.zeros(n, device="cuda").bfloat16(), torch.zeros(n, device="cuda"), torch.ones(
        n, device="cuda")
    m, v = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
    opt = sb.AdamW([p], [g], masters=[w], states=[(m, v)])
    x = {"param": p, "master": w, "state": m, "gradient": g}[which]
    old = x.data_ptr()
    x.data = x.data.clone()
    taken = [torch.empty_like(x) for _ in range(8)]
    assert old not in [a.data_ptr() for a in taken]
    del opt
