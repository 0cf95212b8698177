"""A refused AdamW call leaves the handle as it was."""
import pytest
import torch

import gemm_epilogue_reduction_gb300 as sb

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


def _two(n=300):
    g = torch.Generator(device="cuda").manual_seed(1)
    return [torch.randn(n + i, generator=g, device="cuda") for i in range(2)]


def _bound(opt):
    return [(t.grad, t.grad_type) for t in opt._list]


@pytest.mark.parametrize("bad", ["shape", "type", "device", "contiguity", "count"])
def test_refused_gradients_are_not_bound(bad):
    params, grads = _two(), [x * 0.1 for x in _two()]
    same = [x.clone() for x in params]
    opt = sb.AdamW(params, grads)
    before = _bound(opt)
    new = [g.bfloat16() for g in grads]
    last = {"shape": new[1][:5], "type": new[1].double(), "device": new[1].cpu(),
            "contiguity": torch.zeros(602, device="cuda").bfloat16()[::2]}.get(bad)
    with pytest.raises((ValueError, TypeError)):
        opt.step([new[0]] if bad == "count" else [new[0], last])
    assert _bound(opt) == before
    assert opt.step_count == 0
    opt.step()
    sb.AdamW(same, grads).step()
    assert all(torch.equal(a, b) for a, b in zip(params, same))


def test_refused_arguments_leave_rate_and_gradients():
    params, grads = _two(), _two()
    opt = sb.AdamW(params, grads, lr=0.5)
    before = _bound(opt)
    with pytest.raises(sb.SbError):
        opt.step(lr=-1.0)
    with pytest.raises(TypeError):
        opt.step([g.clone() for g in grads], grad_scale=torch.ones(1, device="cuda").double())
    assert opt.lr == 0.5 and opt.step_count == 0 and _bound(opt) == before
