"""The layer norm's value-by-value mode (arrays off 16 bytes, rows of up to eight values) with many rows to a group of
threads, and calls in place where neighbouring rows share 16-byte vectors.  Bounds as in test_layer_norm.py."""
import pytest
import torch

import gemm_epilogue_reduction_gb300 as sb
from test_layer_norm import BF, F32, _check, _make

gpu = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gemm_epilogue_reduction_gb300 import build as sbbuild
    sbbuild.build()


def _off(t):
    """The same values one element behind an allocation's start."""
    v = torch.empty(t.numel() + 1, dtype=t.dtype, device=t.device)[1:].view(t.shape)
    assert v.is_contiguous() and v.data_ptr() % 16
    return v.copy_(t)


@gpu
@pytest.mark.parametrize("M,d", [(5000, 7), (2500, 333), (700, 4099), (2000, 640), (311, 6144), (160, 16384), (4000, 8)])
@pytest.mark.parametrize("stream", [BF, F32])
@pytest.mark.parametrize("name", ["h", "y", "dx", "dh"])
def test_addresses_off_16_bytes(M, d, stream, name):
    s = _make(M, d, stream=stream, seed=M + d)
    aligned = _check(s, p=0.3, seed=21)
    moved = _check(dict(s, **{name: _off(s[name])}), p=0.3, seed=21)
    # what is dropped does not depend on the mode
    assert torch.equal(aligned[0]["h"], moved[0]["h"])
    assert torch.equal(aligned[1]["dy"] == 0, moved[1]["dy"] == 0) or stream is BF


@gpu
@pytest.mark.parametrize("d", [1, 2, 3, 5, 7, 8])
@pytest.mark.parametrize("branch,p", [(False, 0.0), (True, 0.4)])
def test_many_short_rows(d, branch, p):
    _check(_make(9001, d, stream=F32, branch=branch, seed=d), p=p, seed=2)


@gpu
def test_weights_off_16_bytes():
    for weights in (BF, F32):
        s = _make(400, 1032, weights=weights, seed=3)
        want = _check(s, p=0.1, seed=1)
        got = _check(dict(s, weight=_off(s["weight"]), bias=_off(s["bias"])), p=0.1, seed=1)
        assert torch.equal(got[0]["x"], want[0]["x"]) and torch.equal(got[1]["dweight"], want[1]["dweight"])


@gpu
@pytest.mark.parametrize("M,d", [(3000, 333), (2000, 1030), (700, 4099), (500, 6143), (300, 8199)])
@pytest.mark.parametrize("kind", [0, 1])
def test_in_place_where_rows_share_vectors(M, d, kind):
    s = _make(M, d, stream=(BF, F32)[kind], seed=d)
    f = sb.layer_norm(s["h"], s["weight"], s["bias"], y=s["y"], p=0.2, seed=6)
    b = sb.layer_norm_backward(s["dx"], s["dh"], s["h"], s["weight"], need_dy=True, p=0.2, seed=6)
    n = sb.sb_layer_norm_workspace_bytes(M, d)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    dw, db = (torch.empty_like(s["weight"]) for _ in range(2))
    for _ in range(3):
        h, y = s["h"].clone(), s["y"].clone()
        assert sb.sb_layer_norm_forward(h, y, s["weight"], s["bias"], M, d, kind, 1, 0.2, 6, None, 1e-5, h, y) == sb.SB_OK
        assert torch.equal(h, f["h"]) and torch.equal(y, f["x"])
        dx, dh = s["dx"].clone(), s["dh"].clone()
        assert sb.sb_layer_norm_backward(dx, dh, s["h"], s["weight"], M, d, kind, 1, 0.2, 6, None, 1e-5, dh, dx, dw, db, ws,
                                         n) == sb.SB_OK
        for a, k in ((dh, "dh"), (dx, "dy"), (dw, "dweight"), (db, "dbias")):
            assert torch.equal(a, b[k]), k
