"""An AdamW handle steps on the device that its tensors are on, and refuses any other."""
import pytest
import torch

import gemm_epilogue_reduction_gb300 as sb

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


class OtherStream:
    """Stands in for a stream of a second device."""
    cuda_stream = 0
    device_index = 7
    device = torch.device("cuda", 7)


def test_another_current_device():
    p = torch.zeros(100, device="cuda")
    opt = sb.AdamW([p], [torch.ones(100, device="cuda")])
    opt._device = 7  # as if the handle had been made on another device
    with pytest.raises(ValueError, match="device"):
        opt.step()
    assert opt.step_count == 0 and (p == 0).all()


def test_a_stream_of_another_device():
    p = torch.zeros(100, device="cuda")
    opt = sb.AdamW([p], [torch.ones(100, device="cuda")])
    with pytest.raises(ValueError, match="device"):
        opt.step(stream=OtherStream())
    assert opt.step_count == 0 and (p == 0).all()
