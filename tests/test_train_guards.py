"""The training entry points write nothing outside the arrays they are given: every output, and a
workspace of exactly the size asked for, lies between guard bytes that have to stay."""
import pytest
import torch

import gemm_epilogue_reduction_gb300 as sb
from gemm_epilogue_reduction_gb300 import synth

pytestmark = pytest.mark.gpu
GUARD = 4096


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


class Guards:
    def __init__(self):
        self.all = []

    def like(self, shape, dtype, fill=None):
        """A tensor between guards (256-byte aligned); `fill`: its values."""
        n = 1
        for k in shape:
            n *= k
        size = n * torch.empty(0, dtype=dtype).element_size()
        room = torch.full((GUARD + size + GUARD,), 0xA5, dtype=torch.uint8, device="cuda")
        t = room[GUARD:GUARD + size].view(dtype).view(shape)
        if fill is not None:
            t.copy_(fill)
        self.all.append((room, size))
        return t

    def check(self):
        torch.cuda.synchronize()
        for i, (room, size) in enumerate(self.all):
            assert (room[:GUARD] == 0xA5).all(), ("before", i)
            assert (room[GUARD + size:] == 0xA5).all(), ("after", i)


@pytest.mark.parametrize("M,d,V,piece", [(1, 8, 1, 0), (3, 72, 777, 256), (33, 264, 1000, 0),
                                         (130, 136, 5001, 512), (300, 520, 3333, 1024),
                                         (513, 104, 257, 0), (40, 1032, 30001, 0)])
@pytest.mark.parametrize("reduction", [sb.SB_REDUCE_NONE, sb.SB_REDUCE_MEAN])
def test_cross_entropy(M, d, V, piece, reduction):
    H, W = synth.make_hw(M, d, V, seed=1, device="cuda")
    t = synth.make_targets(M, V, device="cuda")
    if M > 2:
        t[1] = -100
    g = Guards()
    loss = g.like((M if reduction == sb.SB_REDUCE_NONE else 1,), torch.float32)
    lse = g.like((M,), torch.float32)
    n = sb.sb_cross_entropy_workspace_bytes(M, d, V)
    ws = g.like((n,), torch.uint8)
    assert sb.sb_cross_entropy_forward(H, W, t, M, d, V, -100, reduction, 0.0, loss, lse, ws,
                                       n) == sb.SB_OK
    dH, dW = g.like((M, d), torch.bfloat16), g.like((V, d), torch.bfloat16)
    n = sb.sb_cross_entropy_backward_workspace_bytes(M, d, V, piece, True, True)
    ws = g.like((n,), torch.uint8)
    assert sb.sb_cross_entropy_backward(H, W, t, lse, None, M, d, V, -100, reduction, 0.0, piece,
                                        dH, dW, ws, n) == sb.SB_OK
    g.check()
    want = sb.cross_entropy_backward(H, W, t, lse, reduction=["none", "sum", "mean"][reduction],
                                     piece=piece)
    assert torch.equal(dH, want["dH"]) and torch.equal(dW, want["dW"])


@pytest.mark.parametrize("M,d", [(1, 1), (5, 77), (37, 1028), (400, 640), (160, 6144), (9, 8200)])
@pytest.mark.parametrize("stream", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("kind", [sb.SB_GATE_CHANNEL, sb.SB_GATE_TOKEN])
def test_residual_norm(M, d, stream, kind):
    g = Guards()
    st = sb.SB_F32 if stream == torch.float32 else sb.SB_BF16
    h, dh = (torch.randn(M, d, device="cuda").to(stream) for _ in range(2))
    y, dx = (torch.randn(M, d, device="cuda").bfloat16() for _ in range(2))
    pre, post = (torch.ones(d, device="cuda") for _ in range(2))
    token = kind == sb.SB_GATE_TOKEN
    gate = torch.ones(M, d, device="cuda").bfloat16() if token else torch.ones(d, device="cuda")
    ho, x = g.like((M, d), stream), g.like((M, d), torch.bfloat16)
    assert sb.sb_residual_norm_forward(h, y, pre, post, gate, kind, M, d, st, sb.SB_F32, 1.0, 1e-6,
                                       ho, x) == sb.SB_OK
    n = sb.sb_residual_norm_workspace_bytes(M, d)
    ws = g.like((n,), torch.uint8)
    dho, dy = g.like((M, d), stream), g.like((M, d), torch.bfloat16)
    dpre, dpost = g.like((d,), torch.float32), g.like((d,), torch.float32)
    dgate = g.like((M, d), torch.bfloat16) if token else g.like((d,), torch.float32)
    assert sb.sb_residual_norm_backward(dx, dh, ho, y, pre, post, gate, kind, M, d, st, sb.SB_F32,
                                        1.0, 1e-6, dho, dy, dpre, dpost, dgate, ws, n) == sb.SB_OK
    g.check()


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw(bits):
    g = Guards()
    p, m, st, gr = [], [], [], []
    for k in (1, 255, 256, 257, 1000, 4099):
        p.append(g.like((k,), torch.bfloat16, torch.ones(k, device="cuda")))
        m.append(g.like((k,), torch.float32, torch.ones(k, device="cuda")))
        gr.append(torch.randn(k, device="cuda"))
        blocks = (k + 255) // 256
        if bits == 8:
            z = torch.zeros(k, dtype=torch.uint8, device="cuda")
            codes = [g.like((k,), torch.uint8, z).view(torch.float8_e4m3fn) for _ in range(2)]
            st.append(tuple(codes) + tuple(
                g.like((blocks,), torch.float32, torch.zeros(blocks, device="cuda"))
                for _ in range(2)))
        else:
            st.append(tuple(g.like((k,), torch.float32, torch.zeros(k, device="cuda"))
                            for _ in range(2)))
    sb.AdamW(p, gr, masters=m, states=st, state_bits=bits).step()
    g.check()
    assert all(torch.isfinite(x).all() for x in p + m)
