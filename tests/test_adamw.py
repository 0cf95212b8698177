"""The AdamW step over many tensors.

Against the formulas in elementary fp32 operations on the same device, which the kernel follows
operation by operation in all that the states keep: the moments' bits are equal (values, codes and
scales). The reciprocal, and the square root in 32 bits, are approximations within 2^-22, so the
update is within 2^-20 of the formulas' and a weight within that plus one rounding (2^-23 of the
weight). Every step is compared from the state that the kernel had before it.

Against the 64-bit definition: ten fp32 roundings between input and output, so |m|, |v| and the
update are within 16·2^-24 (the update: and 2^-20) of the magnitudes they are sums of, a rounding
to bf16 adds 2^-8 and one to E4M3 2^-4 of the value plus the spacing of its smallest numbers
(2^-10 of a code), relative to the block's scale.
"""
import math

import pytest
import torch

import gemm_epilogue_reduction_gb300 as sb

gpu = pytest.mark.gpu
BF, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
E = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gemm_epilogue_reduction_gb300 import build as sbbuild
    sbbuild.build()


def _pad(x):
    out = torch.zeros(-(-x.numel() // 256) * 256, dtype=x.dtype, device=x.device)
    out[:x.numel()] = x.reshape(-1)
    return out


def _codes(x, root):
    """E4M3 codes and scales of a block format tensor, as sb.h describes them."""
    b = _pad(x).view(-1, 256)
    top = b.abs().amax(1)
    small = top < 2.0 ** -100
    mul = torch.where(small, 0.0, 448.0 / torch.where(small, 1.0, top))
    q = b * mul[:, None]
    if root:
        q = torch.where((q > 0) & (q < 2.0 ** -9), 2.0 ** -9, q)
    return q.to(F8).view(-1)[:x.numel()], torch.where(small, 0.0, top * (1 / 448.0))


def _values(codes, scale):
    return (_pad(codes.float()).view(-1, 256) * scale[:, None]).view(-1)[:codes.numel()]


def _make(sizes, *, param=BF, master=True, grad=BF, bits=32, seed=0, offset=0):
    """Parameters, gradients, masters and states (offset: values into an allocation)."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def place(v):
        room = torch.zeros(v.numel() + offset, dtype=v.dtype, device="cuda")
        room[offset:].view(torch.uint8 if v.dtype == F8 else v.dtype).copy_(
            v.view(torch.uint8) if v.dtype == F8 else v)
        return room[offset:]

    p, gr, ma, st = [], [], [], []
    for k in sizes:
        w = 0.02 * torch.randn(k, generator=g, device="cuda")
        p.append(place(w.to(param)))
        ma.append(place(w) if master and param == BF else None)
        gr.append(place((1e-3 * torch.randn(k, generator=g, device="cuda")).to(grad)))
        m = 1e-3 * torch.randn(k, generator=g, device="cuda")
        r = 1e-3 * torch.randn(k, generator=g, device="cuda").abs()
        if bits == 8:
            (a, sa), (b, sb_) = _codes(m, False), _codes(r, True)
            st.append((place(a), place(b), sa, sb_))
        else:
            st.append((place(m), place(r * r)))
    return p, gr, ma, st


def _step(p, g, w, state, *, lr, b1, b2, eps, wd, t, gs, bits):
    """One tensor's step in elementary operations; returns (fp32 weight, state)."""
    x = (p if w is None else w).float()
    g = g.float() if gs is None else g.float() * gs
    m, v = (state if bits == 32 else (_values(state[0], state[2]), _values(state[1], state[3])))
    if bits == 8:
        v = v * v
    m = m * b1 + g * (1 - b1)
    v = v * b2 + g * g * (1 - b2)
    root = v.sqrt()
    upd = m / (root * (1 / math.sqrt(1 - b2 ** t)) + eps)
    x = x * (1 - lr * wd) - upd * (lr / (1 - b1 ** t))
    if bits == 32:
        state = (m, v)
    else:
        (a, sa), (b, sb_) = _codes(m, False), _codes(root, True)
        state = (a, b, sa, sb_)
    return x, state


def _equal(a, b, name):
    if a.dtype == F8:
        a, b = a.view(torch.uint8), b.view(torch.uint8)
    assert torch.equal(a, b), (name, int((a != b).sum()), a.numel())


HYPER = {"lr": 1e-2, "b1": 0.9, "b2": 0.95, "eps": 1e-8}


def _near(got, want, old, name):
    """A weight (or its bf16 rounding) against the formulas' fp32 one, from the old weight."""
    off = (got.double() - want.double()).abs()
    bound = 2.0 ** -20 * (want.double() - old.double()).abs() + 2.0 ** -22 * want.double().abs()
    if got.dtype == BF:
        bound = bound + 2.0 ** -8 * want.double().abs()
    assert (off <= bound + 1e-45).all(), (name, float((off - bound).max()))


def _check_state(got, want, bits, name):
    for k in range(4 if bits == 8 else 2):
        _equal(got[k], want[k], (name, k))


def _compare(sizes, *, bits, steps=3, gs=None, wd=0.1, start=0, offset=0, **kw):
    p, g, w, st = _make(sizes, bits=bits, offset=offset, **kw)
    opt = sb.AdamW(p, g, lr=HYPER["lr"], betas=(HYPER["b1"], HYPER["b2"]), eps=HYPER["eps"],
                   weight_decay=wd, state_bits=bits, masters=w, states=st, step=start)
    decay = wd if isinstance(wd, list) else [wd] * len(sizes)
    for t in range(start + 1, start + steps + 1):
        old = [(a if b is None else b).clone() for a, b in zip(p, w)]
        want = [_step(a, gr, b, s, t=t, wd=d, gs=gs, bits=bits, **HYPER)
                for a, gr, b, s, d in zip(p, g, w, st, decay)]
        opt.step(grad_scale=gs)
        for i, (x, state) in enumerate(want):
            if w[i] is not None:
                _near(w[i], x, old[i], f"master {i}")
                _equal(p[i], w[i].to(BF), f"param {i}")
            else:
                _near(p[i], x, old[i], f"param {i}")
            _check_state(st[i], state, bits, f"state {i}")
    torch.cuda.synchronize()
    assert opt.step_count == start + steps


SIZES = [1, 255, 256, 257, 0, 7, 2048, 2049, 5120, 4096 * 33 + 5]


@gpu
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("param,master,grad", [(BF, True, BF), (BF, False, BF), (F32, False, F32),
                                               (BF, True, F32), (F32, False, BF)])
def test_steps_follow_the_formulas(bits, param, master, grad):
    _compare(SIZES, bits=bits, param=param, master=master, grad=grad)


@gpu
@pytest.mark.parametrize("bits", [32, 8])
def test_grad_scale_late_steps_and_a_decay_for_each(bits):
    gs = torch.tensor([0.37], device="cuda")
    _compare([300, 512, 1000], bits=bits, gs=gs, wd=[0.0, 0.5, 0.01], start=12345)


@gpu
@pytest.mark.parametrize("bits", [32, 8])
def test_arrays_off_the_wide_alignment(bits):
    _compare([300, 512, 4097], bits=bits, offset=1)


@gpu
@pytest.mark.parametrize("bits", [32, 8])
def test_more_tensors_than_one_launch_takes(bits):
    _compare([(37 * i) % 700 for i in range(800)], bits=bits, steps=2)


@gpu
def test_mixed_types_in_one_list():
    a = _make([500], param=BF, grad=F32, seed=1)
    b = _make([600], param=F32, grad=BF, seed=2)
    p, g, w, st = (x + y for x, y in zip(a, b))
    old = [w[0].clone(), p[1].clone()]
    want = [_step(p[i], g[i], w[i], st[i], t=1, wd=0.1, gs=None, bits=32, **HYPER)
            for i in range(2)]
    sb.AdamW(p, g, lr=HYPER["lr"], betas=(HYPER["b1"], HYPER["b2"]), eps=HYPER["eps"],
             weight_decay=0.1, masters=w, states=st).step()
    for got, (x, state), o, s in zip((w[0], p[1]), want, old, st):
        _near(got, x, o, "weight")
        _check_state(s, state, 32, "state")
    _equal(p[0], w[0].to(BF), "param")


@gpu
def test_against_the_definition_in_64_bits():
    n, t = 70000, 5
    for bits in (32, 8):
        p, g, w, st = _make([n], bits=bits, seed=3)
        w0, g0 = w[0].double(), g[0].double()
        if bits == 8:
            m, v = _values(st[0][0], st[0][2]).double(), _values(st[0][1], st[0][3]).double() ** 2
        else:
            m, v = st[0][0].double(), st[0][1].double()
        sb.AdamW(p, g, lr=1e-2, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.1, state_bits=bits,
                 masters=w, states=st, step=t - 1).step()
        m, mm = 0.9 * m + 0.1 * g0, 0.9 * m.abs() + 0.1 * g0.abs()
        v = 0.95 * v + 0.05 * g0 ** 2
        den = (v / (1 - 0.95 ** t)).sqrt() + 1e-8
        rate = 1e-2 / (1 - 0.9 ** t)
        x = w0 * (1 - 1e-3) - rate * m / den
        off = (w[0].double() - x).abs()
        assert (off <= 16 * E * (w0.abs() + rate * mm / den) + 2.0 ** -20 * rate * mm / den).all()
        assert ((p[0].double() - x).abs() <= off + 2.0 ** -8 * x.abs()).all()
        if bits == 32:
            assert ((st[0][0].double() - m).abs() <= 16 * E * mm).all()
            assert ((st[0][1].double() - v).abs() <= 16 * E * v).all()
        else:
            for code, scale, value in ((st[0][0], st[0][2], m), (st[0][1], st[0][3], v.sqrt())):
                s = scale.double().repeat_interleave(256)[:n]
                held = _values(code, scale).double()
                assert ((held - value).abs() <= 2.0 ** -4 * value.abs() + 2.0 ** -9 * s).all()


@gpu
def test_blocks_of_zeros_tiny_and_huge_values():
    """8 bits: an all-zero block, one whose magnitudes span the whole format, one below 2^-100
    and one with a single large gradient; roots that are there stay above zero."""
    n = 256 * 5
    p, g, w, st = _make([n], bits=8, param=F32, grad=F32, seed=4)
    m, r = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
    g[0][:256] = 0
    m[256:512] = torch.logspace(-12, 3, 256, device="cuda")
    r[256:512] = torch.logspace(-9, 2, 256, device="cuda")
    g[0][512:768] = 1e-32
    g[0][768:1024] = 0
    g[0][800] = 1e4
    (a, sa), (b, sb_) = _codes(m, False), _codes(r, True)
    st = [(a, b, sa, sb_)]
    old = p[0].clone()
    want, state = _step(p[0], g[0], None, st[0], t=1, wd=0.1, gs=None, bits=8, **HYPER)
    sb.AdamW(p, g, lr=HYPER["lr"], betas=(HYPER["b1"], HYPER["b2"]), eps=HYPER["eps"],
             weight_decay=0.1, state_bits=8, states=st).step()
    _near(p[0], want, old, "param")
    _check_state(st[0], state, 8, "state")
    assert torch.isfinite(p[0]).all()
    assert (_values(st[0][1], st[0][3])[256:512] > 0).all()


@gpu
def test_a_nan_gradient_stays_where_it_is():
    for bits in (32, 8):
        p, g, w, st = _make([1024], bits=bits, seed=5)
        g[0][700] = float("nan")
        sb.AdamW(p, g, masters=w, states=st, state_bits=bits).step()
        bad = torch.isnan(p[0])
        assert bad[700] and int(bad.sum()) == 1


@gpu
def test_new_gradients_streams_and_graphs():
    for bits in (32, 8):
        p, g, w, st = _make([3000, 77], bits=bits, seed=6)
        p2, _, w2, st2 = _make([3000, 77], bits=bits, seed=6)
        opt = sb.AdamW(p, masters=w, states=st, state_bits=bits)
        with pytest.raises(ValueError):
            opt.step()
        opt.step(g)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        opt.step([2 * x for x in g], lr=0.5, stream=side)  # made and used on two streams:
        torch.cuda.synchronize()                           # kept alive by the handle until here
        ref = sb.AdamW(p2, [x.clone() for x in g], masters=w2, states=st2, state_bits=bits)
        ref.step()
        ref.step([2 * x for x in g], lr=0.5)
        for a, b in zip(p + w, p2 + w2):
            _equal(a, b, "after two steps")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):  # the step number is the captured one
            opt.step(g)
        graph.replay()
        ref.step(g)
        torch.cuda.synchronize()
        for a, b in zip(p + w, p2 + w2):
            _equal(a, b, "after a replay")


@gpu
def test_offsets_past_32_bits():
    """A tensor of more than 2^31 values: its ends and its middle step as short tensors do."""
    n, k = 2 ** 31 + 1000, 512
    p, g = (torch.zeros(n, dtype=BF, device="cuda") for _ in range(2))
    st = [(torch.zeros(n, dtype=torch.uint8, device="cuda").view(F8),
           torch.zeros(n, dtype=torch.uint8, device="cuda").view(F8),
           torch.zeros((n + 255) // 256, device="cuda"), torch.zeros((n + 255) // 256, device="cuda"))]
    at = [0, 2 ** 30, 2 ** 31 - 256, n // 256 * 256 - 256]  # the last one ends inside a block
    sp, sg, _, sst = _make([min(k, n - a) for a in at], bits=8, master=False, seed=7)
    for a, x, y, s in zip(at, sp, sg, sst):
        p[a:a + x.numel()], g[a:a + x.numel()] = x, y
        for j, per in ((0, 1), (1, 1), (2, 256), (3, 256)):
            to = st[0][j].view(torch.uint8) if j < 2 else st[0][j]
            to[a // per:a // per + s[j].numel()] = s[j].view(torch.uint8) if j < 2 else s[j]
    sb.AdamW([p], [g], states=st, state_bits=8).step()
    sb.AdamW(sp, sg, states=sst, state_bits=8).step()
    for a, x, s in zip(at, sp, sst):
        _equal(p[a:a + x.numel()], x, a)
        for j, per in ((0, 1), (1, 1), (2, 256), (3, 256)):
            _equal(st[0][j][a // per:a // per + s[j].numel()], s[j], (a, j))


@gpu
def test_python_refusals():
    p, g, w, st = _make([64, 65])
    with pytest.raises(ValueError):
        sb.AdamW(p, g, state_bits=16)
    with pytest.raises(ValueError):
        sb.AdamW(p, g[:1])
    with pytest.raises(ValueError):
        sb.AdamW(p, [g[0], g[0]])
    with pytest.raises(TypeError):
        sb.AdamW([x.half() for x in p], g)
    with pytest.raises(TypeError):
        sb.AdamW([x.float() for x in p], g, masters=w)
    with pytest.raises(ValueError):
        sb.AdamW([torch.zeros(8, 8, device="cuda").t()[1:]], None)
    with pytest.raises(ValueError):
        sb.AdamW(p, g, states=[s[:1] for s in st])
    with pytest.raises(ValueError):
        sb.AdamW(p, g, weight_decay=[0.1])
    opt = sb.AdamW(p, g, lr=-1.0)
    with pytest.raises(sb.SbError):
        opt.step()
    with pytest.raises(TypeError):
        sb.AdamW(p, g).step(grad_scale=torch.ones(1, device="cuda", dtype=torch.float64))
    with pytest.raises(ValueError):
        sb.AdamW([x.cpu() for x in p], g)


def test_c_refusals():
    P = 1 << 20

    def call(count=1, lr=1e-3, b1=0.9, b2=0.99, eps=1e-8, step=1, bits=32, gs=None, lst=True, **kw):
        f = {"param": P, "grad": P, "master": None, "exp_avg": P, "exp_avg_sq": P, "scale": P,
             "scale_sq": P, "n": 4, "weight_decay": 0.0, "param_type": 0, "grad_type": 0, **kw}
        arr = (sb.sb_adamw_tensor * 1)(sb.sb_adamw_tensor(**f))
        return sb.sb_adamw_step(arr if lst else None, count, lr, b1, b2, eps, step, bits, gs, 0)

    bad, off, nan = sb.SB_ERR_INVALID_ARG, sb.SB_ERR_ALIGNMENT, float("nan")
    for kw in ({"count": -1}, {"lst": False}, {"lr": -1.0}, {"lr": nan}, {"lr": float("inf")},
               {"b1": 1.0}, {"b1": -0.1}, {"b2": nan}, {"eps": -1e-8}, {"eps": nan}, {"step": 0},
               {"bits": 16}, {"param": None}, {"grad": None}, {"exp_avg": None},
               {"exp_avg_sq": None}, {"bits": 8, "scale": None}, {"bits": 8, "scale_sq": None},
               {"n": -1}, {"param_type": 2}, {"grad_type": -1}, {"weight_decay": -0.5},
               {"weight_decay": nan}, {"param_type": 1, "master": P}):
        assert call(**kw) == bad, kw
    for kw in ({"param": P + 1}, {"param": P + 2, "param_type": 1}, {"grad": P + 1},
               {"master": P + 2}, {"exp_avg": P + 2}, {"exp_avg_sq": P + 1},
               {"bits": 8, "scale": P + 2}, {"gs": P + 2}):
        assert call(**kw) == off, kw


def test_the_descriptor_has_the_c_layout(tmp_path):
    """sb_adamw_tensor as a C compiler lays it out is what the binding passes."""
    import ctypes
    import os
    import subprocess
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    names = [n for n, _ in sb.sb_adamw_tensor._fields_]
    lines = "".join(f'printf("%zu ", offsetof(sb_adamw_tensor, {n}));' for n in names)
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include "sb.h"\nint main(void) {' + lines +
                   'printf("%zu", sizeof(sb_adamw_tensor)); return 0; }\n')
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c11", "-Wall", "-Werror", "-I", os.path.join(root, "include"),
                    str(src), "-o", str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True,
                                          check=True).stdout.split()]
    want = [getattr(sb.sb_adamw_tensor, n).offset for n in names]
    assert got == want + [ctypes.sizeof(sb.sb_adamw_tensor)]
