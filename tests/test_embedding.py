"""The embedding lookup and its gradient against their formulas.

Forward is one product in fp32 and one rounding: the same bits as torch's.  Backward sums the n rows
of a token in fp32, in whatever fixed order: the sum is off by at most n·e of the magnitudes' sum
(e = 2^-24), the scale and the old value add 2e of theirs, the rounding to bf16 adds 2^-8 of the
result.  Gradients that are whole numbers below 2^24 have no roundings in fp32: there the bits are
compared.
"""
import pytest
import torch

import gemm_epilogue_reduction_gb300 as sb

gpu = pytest.mark.gpu
BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64
U, E = 2.0 ** -8, 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gemm_epilogue_reduction_gb300 import build as sbbuild
    sbbuild.build()


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _ids(M, V, seed, kind="zipf"):
    g = _gen(seed)
    if kind == "same":
        return torch.full((M,), V - 1, dtype=torch.int32, device="cuda")
    if kind == "all":
        return (torch.randperm(max(M, V), generator=g, device="cuda")[:M] % V).int()
    r = torch.rand(M, generator=g, device="cuda", dtype=F64)
    ids = ((V + 1.0) ** r - 1).long().clamp(max=V - 1).int()
    if kind == "padded" and M:
        ids[torch.rand(M, generator=g, device="cuda") < 0.3] = -100
        ids[-1] = -100
    return ids


def _bits(a, b):
    return torch.equal(a.view(torch.int16 if a.dtype is BF else torch.int32),
                       b.view(torch.int16 if b.dtype is BF else torch.int32))


@gpu
@pytest.mark.parametrize("M,d,V", [(1, 1, 1), (1, 5120, 1000), (5, 7, 3), (33, 64, 500), (16, 5120, 999),
                                   (100, 2056, 777), (257, 4100, 50), (40, 12296, 30), (3, 65540, 5),
                                   (2, 131075, 4), (0, 64, 10)])
@pytest.mark.parametrize("weights", [BF, F32])
@pytest.mark.parametrize("out", [BF, F32])
def test_lookup(M, d, V, weights, out):
    W = torch.randn(V, d, generator=_gen(1), device="cuda").to(weights)
    ids = _ids(M, V, 2, "padded")
    for scale in (1.0, 11.3):
        got = sb.embedding(ids, W, scale=scale, dtype=out)
        want = W[ids.clamp(min=0).long()].float() * scale
        want[ids == -100] = 0
        assert _bits(got, want.to(out))
    assert sb.embedding(ids, W).dtype is weights


@gpu
@pytest.mark.parametrize("d", [9, 10, 15, 31, 257, 1021, 2046, 4099])
@pytest.mark.parametrize("weights", [BF, F32])
@pytest.mark.parametrize("out", [BF, F32])
def test_lookup_of_odd_rows(d, weights, out):
    # every place of a row of W against every place of a row of the output; what lies around both stays
    # unread and unwritten
    V, M = 13, 13 * 8 + 5
    W = torch.randn(V * d, generator=_gen(1), device="cuda").to(weights).view(V, d)
    ids = (torch.arange(M, device="cuda") * 5 + torch.arange(M, device="cuda") // 13).remainder(V).int()
    ids[7], ids[20], ids[-2] = -100, V, V - 1
    room = torch.full((M * d + 64,), 7.0, dtype=out, device="cuda")
    got = room[32:32 + M * d].view(M, d)
    want = W[ids.clamp(0, V - 1).long()].float() * 1.7
    want[7], want[20] = 0, float("nan")
    kind = {BF: 0, F32: 1}
    assert sb.sb_embedding_forward(ids.data_ptr(), W.data_ptr(), M, d, V, -100, 1.7, kind[weights], kind[out],
                                   got.data_ptr(), torch.cuda.current_stream().cuda_stream) == sb.SB_OK
    keep = torch.arange(M, device="cuda") != 20
    assert _bits(got[keep], want[keep].to(out)) and got[20].isnan().all()
    assert (room[:32] == 7).all() and (room[32 + M * d:] == 7).all()


@gpu
def test_lookup_of_ids_outside():
    W = torch.randn(10, 24, device="cuda").bfloat16()
    ids = torch.tensor([3, -1, 10, 2 ** 31 - 1, -2 ** 31, 9, 4], dtype=torch.int32, device="cuda")
    out = sb.embedding(ids, W, ignore_index=4)
    assert torch.equal(out[[0, 5]], W[[3, 9]]) and out[1:5].isnan().all() and (out[6] == 0).all()
    # infinities and NaN of the matrix stay in their rows
    W[3, 5], W[9, 0] = float("inf"), float("nan")
    out = sb.embedding(ids, W, ignore_index=4)
    assert out[0, 5] == float("inf") and out[5, 0].isnan() and (out[6] == 0).all()


def _sums(ids, dout, V, scale, ignore=-100):
    """(sum, sum of magnitudes, count) of every row of W in 64 bits."""
    used = (ids != ignore) & (ids >= 0) & (ids < V)
    at, d = ids[used].long(), dout[used].to(F64) * scale
    out = torch.zeros(V, dout.shape[1], dtype=F64, device="cuda")
    mag, n = out.clone(), torch.zeros(V, 1, dtype=F64, device="cuda")
    n.index_add_(0, at, torch.ones(len(at), 1, dtype=F64, device="cuda"))
    return out.index_add_(0, at, d), mag.index_add_(0, at, d.abs()), n


SHAPES = [(1, 1, 1), (1, 5120, 300), (2, 3, 5), (31, 64, 40), (32, 72, 9), (33, 68, 9), (64, 1032, 3),
          (100, 257, 1000), (500, 640, 100), (1021, 4100, 60), (65, 72, 4), (4097, 4104, 90), (4097, 96, 2000), (8192, 40, 333),
          (8193, 40, 333), (20000, 33, 4000), (30011, 8, 7),
          (70001, 8, 500)]


@gpu
@pytest.mark.parametrize("M,d,V", SHAPES)
@pytest.mark.parametrize("kind", ["zipf", "same", "all", "padded"])
@pytest.mark.parametrize("grad,weights", [(BF, BF), (F32, F32), (BF, F32), (F32, BF)])
def test_gradient(M, d, V, kind, grad, weights):
    ids = _ids(M, V, M + d, kind)
    g = _gen(M)
    # whole numbers: every order of fp32 sums gives the same
    whole = torch.randint(-8, 9, (M, d), generator=g, device="cuda").to(grad)
    exact, mag, n = _sums(ids, whole, V, 2.0)
    got = sb.embedding_backward(ids, whole, vocab=V, scale=2.0, dtype=weights)["dW"]
    assert _bits(got, exact.float().to(weights) + 0.0)
    old = torch.randint(-8, 9, (V, d), generator=g, device="cuda").to(weights)
    new = old.clone()
    assert sb.embedding_backward(ids, whole, dW=new, scale=2.0)["dW"] is new
    assert _bits(torch.where(n > 0, new, 0) + 0.0, torch.where(n > 0, (exact + old.double()).float().to(weights), 0) + 0.0)
    assert _bits(torch.where(n > 0, 0, new), torch.where(n > 0, 0, old))
    # and any numbers, within the bound above
    dout = torch.randn(M, d, generator=g, device="cuda").to(grad)
    exact, mag, n = _sums(ids, dout, V, 0.7)
    u = U if weights is BF else E
    old = torch.randn(V, d, generator=g, device="cuda").to(weights)
    for start in (None, old):
        new = None if start is None else start.clone()
        got = sb.embedding_backward(ids, dout, vocab=V if new is None else None, dW=new, scale=0.7,
                                    dtype=weights)["dW"]
        want = exact if start is None else exact + torch.where(n > 0, start.double(), 0.0)
        size = mag if start is None else mag + start.double().abs()
        if start is not None:
            got = torch.where(n > 0, got, 0)
        # (0.7 itself is rounded to fp32: one e more)
        bound = (n + 4) * E * size * 1.01 + u * want.abs() * 1.01
        assert ((got.double() - want).abs() <= bound).all()


@gpu
@pytest.mark.parametrize("d", [129, 247, 249, 255, 993, 1022, 1983, 4099])
@pytest.mark.parametrize("M,V", [(50, 40), (333, 61), (2500, 17)])
@pytest.mark.parametrize("grad,weights", [(BF, BF), (F32, F32), (BF, F32), (F32, BF)])
def test_gradient_of_odd_rows(M, d, V, grad, weights):
    # whole numbers: no rounding in fp32 (sums below 2500·16 + 64), one to bf16 at the end; runs of one token,
    # inside a piece and over several, rows at every place of a vector, what lies around dW unwritten
    g = _gen(M + d)
    ids = _ids(M, V, M, "padded")
    dout = torch.randint(-8, 9, (M, d), generator=g, device="cuda").to(grad)
    room = torch.full((V * d + 64,), 3.0, dtype=weights, device="cuda")
    dW = room[32:32 + V * d].view(V, d)
    for add in (False, True):
        dW.copy_(torch.randint(-32, 33, (V, d), generator=g, device="cuda"))
        old = dW.double() * add
        sums, _, _ = _sums(ids, dout, V, 2.0)
        if add:
            sb.embedding_backward(ids, dout, dW=dW, scale=2.0)
        else:
            ws = torch.empty(sb.sb_embedding_backward_workspace_bytes(M, d), dtype=torch.uint8, device="cuda")
            kind = {BF: 0, F32: 1}
            assert sb.sb_embedding_backward(
                ids.data_ptr(), dout.data_ptr(), M, d, V, -100, 2.0, kind[grad], kind[weights], 0, dW.data_ptr(),
                ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream) == sb.SB_OK
        assert torch.equal(dW, (sums + old).to(weights))
        assert (room[:32] == 3).all() and (room[32 + V * d:] == 3).all()


@gpu
def test_gradient_ignores_what_has_no_row():
    V, d = 20, 40
    ids = torch.tensor([5, -7, 20, 2 ** 31 - 1, -2 ** 31, 3, 5, 3], dtype=torch.int32, device="cuda")
    dout = torch.ones(8, d, device="cuda")
    dout[1:5] = float("nan")  # of tokens without a row: not looked at
    dout[[5, 7]] = float("inf")
    dW = sb.embedding_backward(ids, dout, vocab=V, ignore_index=3)["dW"]
    want = torch.zeros(V, d, device="cuda")
    want[5] = 2
    assert torch.equal(dW, want)
    # not a number stays in its token's row
    dout[0, 7] = float("nan")
    dW = sb.embedding_backward(ids, dout, vocab=V, ignore_index=3)["dW"]
    assert dW[5, 7].isnan() and dW.isnan().sum() == 1
    # every token without a row
    assert (sb.embedding_backward(torch.full_like(ids, -100), dout, vocab=V)["dW"] == 0).all()


@gpu
def test_no_tokens():
    ids, dout = torch.empty(0, dtype=torch.int32, device="cuda"), torch.empty(0, 72, device="cuda")
    assert (sb.embedding_backward(ids, dout, vocab=33)["dW"] == 0).all()
    dW = torch.randn(33, 72, device="cuda")
    old = dW.clone()
    sb.embedding_backward(ids, dout, dW=dW)
    assert torch.equal(dW, old)
    assert sb.embedding(ids, dW).shape == (0, 72)


@gpu
def test_arrays_that_are_not_on_16_bytes():
    """The same values from addresses that take no wide loads, and zeros up to both ends."""
    M, d, V = 300, 64, 45
    ids = _ids(M, V, 3)

    def off(x):
        room = torch.full((x.numel() + 9,), 7, dtype=x.dtype, device="cuda")
        room[1:1 + x.numel()] = x.reshape(-1)
        return room, room[1:1 + x.numel()].view(x.shape)

    for t in (BF, F32):
        W, dout = torch.randn(V, d, device="cuda").to(t), torch.randn(M, d, device="cuda").to(t)
        assert torch.equal(sb.embedding(ids, off(W)[1]), sb.embedding(ids, W))
        want = sb.embedding_backward(ids, dout, vocab=V)["dW"]
        room, dW = off(torch.ones(V, d, device="cuda").to(t))
        n = sb.sb_embedding_backward_workspace_bytes(M, d)
        ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        kind = sb.SB_F32 if t is F32 else sb.SB_BF16
        assert sb.sb_embedding_backward(ids, off(dout)[1], M, d, V, -100, 1.0, kind, kind, 0, dW, ws,
                                        n) == sb.SB_OK
        torch.cuda.synchronize()
        # one thread's columns are added in the same order whatever their number
        assert torch.equal(dW, want) and room[0] == 7 and (room[1 + V * d:] == 7).all()


@gpu
def test_gradient_against_differences():
    """<embedding(ids, W), a> is linear in W: its slope along any direction is that of the gradient."""
    M, d, V = 40, 24, 11
    ids, g = _ids(M, V, 4, "padded"), _gen(4)
    a = torch.randn(M, d, generator=g, device="cuda")
    W, way = (torch.randn(V, d, generator=g, device="cuda") for _ in range(2))
    dW = sb.embedding_backward(ids, a, vocab=V, scale=3.0)["dW"]

    def value(W):
        return (sb.embedding(ids, W, scale=3.0).double() * a.double()).sum()

    slope = (value(W + way) - value(W - way)) / 2
    # the sums W ± way and the products are rounded: 3e each, twice
    bound = 8 * E * (3 * (W.abs() + way.abs())[ids.clamp(min=0).long()].double() * a.double().abs()).sum()
    assert abs(slope - (dW.double() * way.double()).sum()) <= bound


@gpu
def test_repeats_streams_and_graphs_give_the_same_bits():
    M, d, V = 9000, 520, 1000
    ids, dout = _ids(M, V, 5, "padded"), torch.randn(M, d, device="cuda").bfloat16()
    W = torch.randn(V, d, device="cuda").bfloat16()
    want, rows = sb.embedding_backward(ids, dout, vocab=V)["dW"], sb.embedding(ids, W)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (None, side, side.cuda_stream):
        for _ in range(5):
            got = sb.embedding_backward(ids, dout, vocab=V, stream=stream)["dW"]
            out = sb.embedding(ids, W, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(got, want) and torch.equal(out, rows)
    graph = torch.cuda.CUDAGraph()
    acc = torch.zeros(V, d, device="cuda")
    with torch.cuda.graph(graph):
        got = sb.embedding_backward(ids, dout, vocab=V)["dW"]
        sb.embedding_backward(ids, dout, dW=acc)
        out = sb.embedding(ids, W)
    other = _ids(M, V, 6)
    for x in (other, ids):
        want, rows = sb.embedding_backward(x, dout, vocab=V)["dW"], sb.embedding(x, W)
        sums = sb.embedding_backward(x, dout, vocab=V, dtype=F32)["dW"]
        ids.copy_(x)
        acc.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want) and torch.equal(out, rows) and torch.equal(acc, sums)


@gpu
def test_offsets_past_32_bits():
    """A matrix of more than 2^32 values: its last rows, which 32-bit offsets would miss."""
    V, d = 700_001, 6144
    W = torch.zeros(V, d, dtype=BF, device="cuda")
    W[-3:] = torch.randn(3, d, device="cuda").bfloat16()
    ids = torch.tensor([V - 1, V - 3, 0, V - 2, V - 1], dtype=torch.int32, device="cuda")
    assert torch.equal(sb.embedding(ids, W), W[ids.long()])
    dout = torch.ones(5, d, device="cuda", dtype=BF)
    sb.embedding_backward(ids, dout, dW=W.zero_())
    assert (W[-1] == 2).all() and (W[[0, V - 2, V - 3]] == 1).all() and (W[1:V - 3] == 0).all()
    W.fill_(3)
    del W
    dW = sb.embedding_backward(ids, dout, vocab=V)["dW"]
    assert (dW[-1] == 2).all() and (dW[[0, V - 2, V - 3]] == 1).all() and (dW[1:V - 3] == 0).all()


@gpu
def test_refusals():
    ids = torch.zeros(4, dtype=torch.int32, device="cuda")
    W, dout = torch.zeros(5, 16, device="cuda"), torch.zeros(4, 16, device="cuda")
    for bad in ({"ids": ids.long()}, {"W": W.half()}, {"dtype": torch.float16}):
        with pytest.raises(TypeError):
            sb.embedding(**{"ids": ids, "W": W, **bad})
    for bad in ({"ids": ids.cpu()}, {"W": W.t()}, {"W": W[:, ::2]}, {"W": W[0]}, {"ids": ids[None]},
                {"ignore_index": 2 ** 31}, {"ids": torch.zeros(8, dtype=torch.int32, device="cuda")[::2]}):
        with pytest.raises(ValueError):
            sb.embedding(**{"ids": ids, "W": W, **bad})
    for bad in ({}, {"vocab": 5, "dW": W}, {"vocab": 0}, {"dW": W[:, :8]}, {"dW": W[:, :8].contiguous()},
                {"dW": W, "dtype": BF}, {"vocab": 5, "dout": dout[:3]}, {"dW": W.cpu()},
                {"vocab": 5, "workspace": torch.empty(9999, dtype=torch.uint8)}):
        with pytest.raises(ValueError):
            sb.embedding_backward(**{"ids": ids, "dout": dout, **bad})
    with pytest.raises(TypeError):
        sb.embedding_backward(ids, dout.half(), vocab=5)
    with pytest.raises(sb.SbError):
        sb.embedding(ids, W, scale=float("inf"))
    with pytest.raises(sb.SbError):
        sb.embedding_backward(ids, dout, vocab=5, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))


def test_c_refusals():
    P = 1 << 20

    def fwd(ids=P, W=P, M=4, d=64, V=100, scale=1.0, wt=0, ot=0, out=P):
        return sb.sb_embedding_forward(ids, W, M, d, V, -100, scale, wt, ot, out, 0)

    def bwd(ids=P, dout=P, M=4, d=64, V=100, scale=1.0, gt=0, wt=0, add=0, dW=P, ws=P, n=1 << 30):
        return sb.sb_embedding_backward(ids, dout, M, d, V, -100, scale, gt, wt, add, dW, ws, n, 0)

    bad, off = sb.SB_ERR_INVALID_ARG, sb.SB_ERR_ALIGNMENT
    for call in (fwd, bwd):
        for kw in ({"ids": None}, {"M": -1}, {"M": 2 ** 31}, {"d": 0}, {"d": 2 ** 23}, {"V": 0},
                   {"V": 2 ** 31 - 1}, {"scale": float("nan")}, {"wt": 2}, {"wt": -1}):
            assert call(**kw) == bad, (call.__name__, kw)
        assert call(ids=P + 2) == off
    for kw in ({"W": None}, {"out": None}, {"ot": 2}):
        assert fwd(**kw) == bad, kw
    for kw in ({"W": P + 1}, {"W": P + 2, "wt": 1}, {"out": P + 1}, {"out": P + 2, "ot": 1}):
        assert fwd(**kw) == off, kw
    for kw in ({"dout": None}, {"dW": None}, {"ws": None}, {"gt": 2}, {"add": 2}, {"add": -1}):
        assert bwd(**kw) == bad, kw
    for kw in ({"dout": P + 1}, {"dout": P + 2, "gt": 1}, {"dW": P + 1}, {"dW": P + 2, "wt": 1},
               {"ws": P + 128}):
        assert bwd(**kw) == off, kw
    # outputs over the inputs' memory (arrays of bf16: W 12,800 bytes, out and dout 512)
    far = P + (1 << 18)
    assert fwd(ids=far, out=P + 12798) == bad and fwd(ids=P + 12800 + 508, out=P + 12800) == bad
    assert bwd(ids=far, ws=2 * far, dout=P + 12798, dW=P) == bad and bwd(ids=far, ws=2 * far, dout=P, dW=P) == bad
    assert bwd(ids=far, ws=far + 4096, dout=far - 4096, dW=P, n=64) in (sb.SB_ERR_WORKSPACE_TOO_SMALL,
                                                                     sb.SB_ERR_UNSUPPORTED, sb.SB_ERR_CUDA)
    assert sb.sb_embedding_backward_workspace_bytes(-1, 64) == 0
    assert sb.sb_embedding_backward_workspace_bytes(4, 0) == 0
    assert sb.sb_embedding_backward_workspace_bytes(0, 64) > 0
