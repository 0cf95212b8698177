"""Dropout against SplitMix64 in whole numbers: which elements are dropped has to be equal.

What is kept is x·65536/(65536 - t), formed exactly in 64 bits from the fp32 factor (24 by 24 bits):
without a residual one rounding to fp32 and one to the result's type, the same bits.  With one the
sum is a fused multiply-add: off by one rounding to fp32 of the result, and one to its type.
"""
import numpy as np
import pytest
import torch

import gemm_epilogue_reduction_gb300 as sb

gpu = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
MASK = (1 << 64) - 1


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gemm_epilogue_reduction_gb300 import build as sbbuild
    sbbuild.build()


def splitmix(n, seed):
    """Draws n (array) of the seed's stream."""
    with np.errstate(over="ignore"):
        x = np.uint64(seed & MASK) + (n.astype(np.uint64) + np.uint64(1)) * np.uint64(0x9E3779B97F4A7C15)
        x = (x ^ (x >> np.uint64(30))) * np.uint64(0xBF58476D1CE4E5B9)
        x = (x ^ (x >> np.uint64(27))) * np.uint64(0x94D049BB133111EB)
        return x ^ (x >> np.uint64(31))


def threshold(p):
    return int(np.rint(np.float64(np.float32(p)) * 65536))


def kept(count, p, seed, first=0):
    """Whether elements first .. first + count - 1 stay."""
    i = np.arange(first, first + count, dtype=np.uint64)
    field = (splitmix(i // np.uint64(4), seed) >> (np.uint64(16) * (i % np.uint64(4)))) & np.uint64(65535)
    return torch.from_numpy(field.astype(np.int64) >= threshold(p)).cuda()


def factor(p):
    t = threshold(p)
    return float(np.float32(65536 / (65536 - t))) if t < 65536 else 0.0


def dropped(x, p, seed):
    keep = kept(x.numel(), p, seed).view(x.shape)
    return torch.where(keep, x.double() * factor(p), 0.0), keep


def test_the_reference_is_the_published_generator():
    golden = [int(line.split()[-1], 16) for line in
              open(__file__.replace("test_dropout.py", "golden/splitmix64_seed0.txt"))
              if line.strip() and not line.startswith("#")]
    assert [int(v) for v in splitmix(np.arange(len(golden)), 0)] == golden


@gpu
@pytest.mark.parametrize("shape", [(1,), (3,), (4,), (5,), (8,), (257,), (33, 7), (64, 4096), (1021, 33),
                                   (8191,), (8193,), (3, 5, 77)])
@pytest.mark.parametrize("xt", [BF, F32])
@pytest.mark.parametrize("ot", [BF, F32])
@pytest.mark.parametrize("p,seed", [(0.1, 1), (0.5, 2 ** 64 - 1), (0.999, -5), (0.0, 3), (1.0, 4), (1e-6, 5)])
def test_values(shape, xt, ot, p, seed):
    g = torch.Generator(device="cuda").manual_seed(7)
    x = torch.randn(*shape, generator=g, device="cuda").to(xt)
    want, keep = dropped(x, p, seed)
    got = sb.dropout(x, p, seed=seed, dtype=ot)
    assert got.dtype is ot and torch.equal(got, want.float().to(ot))
    res = (2 * torch.randn(*shape, generator=g, device="cuda")).to(ot)
    got = sb.dropout(x, p, seed=seed, residual=res)
    assert torch.equal(got[~keep], res[~keep])
    want = want + res.double()
    u = 2.0 ** -24 + (2.0 ** -8 if ot is BF else 0)
    assert ((got.double() - want).abs() <= u * want.abs() * 1.01).all()


@gpu
def test_it_is_its_own_gradient_and_drops_the_share_asked_for():
    n, p = 1 << 22, 0.1
    x = torch.ones(n, device="cuda")
    out = sb.dropout(x, p, seed=11)
    back = sb.dropout(torch.full_like(x, 3.0), p, seed=11)
    assert torch.equal(back, 3.0 * out)
    # a share of t / 65536, within five deviations of n draws
    share, t = float((out == 0).double().mean()), threshold(p) / 65536
    assert abs(share - t) < 5 * (t * (1 - t) / n) ** 0.5
    # another seed, another mask: both drop an element with probability t²
    other = sb.dropout(x, p, seed=12)
    both = float(((out == 0) & (other == 0)).double().mean())
    assert abs(both - t * t) < 5 * (t * t / n) ** 0.5


@gpu
def test_what_is_dropped_leaves_no_trace():
    x = torch.full((4096,), float("nan"), device="cuda")
    x[::2] = float("inf")
    keep = kept(4096, 0.5, 9)
    out = sb.dropout(x, 0.5, seed=9, residual=torch.ones_like(x))
    assert (out[~keep] == 1).all() and torch.equal(out[keep].isnan(), x[keep].isnan())
    assert (sb.dropout(x, 1.0, seed=9) == 0).all()


@gpu
def test_in_place_and_unaligned():
    x = torch.randn(10_000, device="cuda").bfloat16()
    res = torch.randn(10_000, device="cuda").bfloat16()
    want, both = sb.dropout(x, 0.3, seed=5), sb.dropout(x, 0.3, seed=5, residual=res)
    for shift in (0, 1, 3):
        room = torch.zeros(10_020, device="cuda", dtype=BF)
        y = room[shift:shift + 10_000]
        y.copy_(x)
        assert torch.equal(sb.dropout(y, 0.3, seed=5), want)
        assert sb.sb_dropout(y, None, 10_000, 0, 0, 0.3, 5, None, y) == sb.SB_OK
        assert torch.equal(y, want) and (room[shift + 10_000:] == 0).all()
        y.copy_(res)
        assert sb.sb_dropout(x, y, 10_000, 0, 0, 0.3, 5, None, y) == sb.SB_OK
        assert torch.equal(y, both)


@gpu
def test_the_offset_is_read_when_the_kernel_runs():
    x = torch.randn(5000, device="cuda")
    off = torch.tensor([41], device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    assert torch.equal(sb.dropout(x, 0.2, seed=1, seed_offset=off, stream=side), sb.dropout(x, 0.2, seed=42))
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        out = sb.dropout(x, 0.2, seed=2 ** 64 - 1, seed_offset=off)
        off += 1
    for step in (41, 42, 43):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, sb.dropout(x, 0.2, seed=step - 1))


@gpu
def test_offsets_past_32_bits():
    n = (1 << 32) + 4099
    x = torch.ones(n, dtype=BF, device="cuda")
    out = sb.dropout(x, 0.5, seed=3)
    for first, count in ((0, 100), ((1 << 31) - 50, 100), ((1 << 32) - 50, 4149)):
        want = torch.where(kept(count, 0.5, 3, first), 2.0, 0.0)
        assert torch.equal(out[first:first + count].float(), want)


@gpu
def test_refusals():
    x = torch.zeros(4, 8, device="cuda")
    for bad in ({"x": x.half()}, {"dtype": torch.float16}, {"residual": x.half()},
                {"seed_offset": torch.zeros(1, device="cuda")}):
        with pytest.raises(TypeError):
            sb.dropout(**{"x": x, "p": 0.1, "seed": 0, **bad})
    for bad in ({"x": x.t()}, {"x": x.cpu()}, {"residual": x[:2]}, {"residual": x, "dtype": BF},
                {"seed": 2 ** 64}, {"seed": -2 ** 63 - 1}, {"seed_offset": torch.zeros(1, dtype=torch.int64)},
                {"seed_offset": torch.zeros(2, dtype=torch.int64, device="cuda")}):
        with pytest.raises(ValueError):
            sb.dropout(**{"x": x, "p": 0.1, "seed": 0, **bad})
    for p in (-0.1, 1.1, float("nan")):
        with pytest.raises(sb.SbError):
            sb.dropout(x, p, seed=0)
    assert sb.dropout(x[:0], 0.1, seed=0).shape == (0, 8)


def test_c_refusals():
    P = 1 << 20

    def call(x=P, res=P, n=4, xt=0, ot=0, p=0.1, off=P, out=P):
        return sb.sb_dropout(x, res, n, xt, ot, p, 0, off, out, 0)

    for kw in ({"x": None}, {"out": None}, {"n": -1}, {"n": 2 ** 43}, {"xt": 2}, {"ot": -1}, {"p": -0.5},
               {"p": 1.5}, {"p": float("nan")}):
        assert call(**kw) == sb.SB_ERR_INVALID_ARG, kw
    for kw in ({"x": P + 1}, {"x": P + 2, "xt": 1}, {"res": P + 1}, {"out": P + 2, "ot": 1}, {"off": P + 4}):
        assert call(**kw) == sb.SB_ERR_ALIGNMENT, kw
    # out over a part of x (4 bf16 or fp32 values) or of the residual, or over x of another type
    far = P + 4096
    for kw in ({"out": P + 4, "res": far}, {"x": far, "out": P + 2}, {"ot": 1, "out": P, "res": far},
               {"xt": 1, "out": P + 12, "res": far}):
        assert call(**{"off": 2 * far, **kw}) == sb.SB_ERR_INVALID_ARG, kw
