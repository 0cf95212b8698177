"""The layer norm's gradients where a row's deviation is far from 1: x does not depend on the row's scale, and the
gradient goes by its inverse, so every term stays in fp32's range.  Definition in 64 bits; bounds as in
test_layer_norm.py, whose reference takes no power of the deviation either once the rows are scaled back."""
import pytest
import torch

import gemm_epilogue_reduction_gb300 as sb
from test_layer_norm import BF, F32, _backward, _make, _within

gpu = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gemm_epilogue_reduction_gb300 import build as sbbuild
    sbbuild.build()


@gpu
@pytest.mark.parametrize("scale,eps", [(1e15, 1e-5), (1e16, 0.0), (1e-14, 0.0), (1e-17, 0.0), (1e8, 1e-5), (1.0, 1e-5)])
@pytest.mark.parametrize("M,d", [(5, 640), (3, 333), (2, 7), (4, 8192), (2, 12000)])
@pytest.mark.parametrize("stream", [BF, F32])
def test_gradients_of_scaled_rows(scale, eps, M, d, stream):
    """The gradient of rows h·scale is that of h over the scale (eps aside, which is 1e-5 / scale^2 there)."""
    s = _make(M, d, stream=stream, branch=False, seed=d)
    s["h"] = (s["h"].double() * scale).to(stream)
    b = sb.layer_norm_backward(s["dx"], None, s["h"], s["weight"], eps=eps)
    plain = dict(s, h=s["h"].double() / scale)
    want = _backward(plain, 0.0, 0, eps / scale ** 2, False, False)
    # what is stored is rounded to the stream's type at the gradient's own size
    _within(b["dh"].double() * scale, (want["dh"][0], want["dh"][1] + 2.0 ** -8 * want["dh"][0].abs() * (stream is BF)), "dh")
    _within(b["dweight"], want["dweight"], "dweight")
    _within(b["dbias"], want["dbias"], "dbias")
