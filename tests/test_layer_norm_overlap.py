"""Layer norm calls whose outputs lie over other arrays, on made-up addresses: none is launched (what is not refused for
its addresses has a workspace that is too small)."""
import pytest

import gemm_epilogue_reduction_gb300 as sb


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gemm_epilogue_reduction_gb300 import build as sbbuild
    sbbuild.build()


M, D = 4, 64
MB = 1 << 20
ROWS, VECTOR = M * D * 2, D * 4  # bf16 streams, fp32 weights


def _places(*names):
    return {k: (i + 1) * MB for i, k in enumerate(names)}


def _around(at, size, n, step):
    """Where an array of n bytes would have to start to share the first or the last place of one of `size` bytes."""
    return {at, at + (size - 1) // step * step, at - (n - 1) // step * step}


def test_forward_over_the_seed_offset():
    P = _places("h", "y", "weight", "bias", "off", "ho", "x")

    def call(**kw):
        a = {**P, **kw}
        return sb.sb_layer_norm_forward(a["h"], a["y"], a["weight"], a["bias"], M, D, 0, 1, 0.1, 0, a["off"], 1e-5, a["ho"],
                                        a["x"], 0)

    for out in ("ho", "x"):
        for at in _around(P["off"], 8, ROWS, 16):
            assert call(**{out: at}) == sb.SB_ERR_INVALID_ARG, (out, at - P["off"])


def _backward(outputs):
    P = _places("dx", "dh", "h", "weight", "off", "dho", "dy", "dw", "db", "ws")
    size = M * 2 * D * 4  # of the workspace, with a block to a row
    SIZE = {"dx": ROWS, "dh": ROWS, "h": ROWS, "weight": VECTOR, "off": 8, "dho": ROWS, "dy": ROWS, "dw": VECTOR,
            "db": VECTOR, "ws": size}

    def call(n=0, **kw):
        a = {**P, **kw}
        return sb.sb_layer_norm_backward(a["dx"], a["dh"], a["h"], a["weight"], M, D, 0, 1, 0.1, 0, a["off"], 1e-5, a["dho"],
                                         a["dy"], a["dw"], a["db"], a["ws"], n, 0)

    for out in outputs:
        for other in P:
            if other == out or (other == "ws" and "ws" not in outputs):
                continue
            for at in _around(P[other], SIZE[other], SIZE[out], 256 if out == "ws" else 16):
                if at == P[other] and (out, other) in (("dho", "dh"), ("dy", "dx")):
                    continue
                assert call(**{out: at}) == sb.SB_ERR_INVALID_ARG, (out, other, at - P[other])
    # neighbours, and what is allowed in place, get as far as the workspace's size (or the missing device)
    for kw in ({"dho": P["dh"]}, {"dy": P["dx"]}, {"dw": P["db"] - VECTOR}, {"dho": P["h"] + ROWS},
               {"dh": None, "dy": None, "db": None, "off": None}):
        assert call(**kw) not in (sb.SB_OK, sb.SB_ERR_INVALID_ARG, sb.SB_ERR_ALIGNMENT), kw


def test_backward_outputs():
    _backward(("dho", "dy", "dw", "db"))


@pytest.mark.gpu
def test_backward_workspace():
    """(Without a device its size is not known.)"""
    assert sb.sb_layer_norm_workspace_bytes(M, D) == M * 2 * D * 4
    _backward(("dho", "dy", "dw", "db", "ws"))
