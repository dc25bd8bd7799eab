"""What is not finite, or nearly so, on its way through the 4-bit layer."""
import numpy as np
import pytest

from mokutil import ROOT  # noqa: F401
from test_gpu_w4 import layer_case

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import mixture_experts_layer_build_amd as mok  # noqa: E402


@pytest.mark.parametrize("how", ["sym128", "zero64", "mxfp4"])
@pytest.mark.parametrize("T", [3, 12])
@pytest.mark.parametrize("limit", [0.0, 0.5, 7.0])
def test_a_limit_keeps_what_is_no_number(how, T, limit):
    """min(g, L) and clamp(u, -L, L) of a NaN are NaN: a token with one, or (int4) with an infinity, and one that chose
    an expert with a NaN scale get a row of NaN, the others what they got without."""
    x, rw, ids, ws, _ = layer_case(20, T, 256, 128, 8, 2, 128, how)
    ids[:] = ids % 6
    clean = mok.forward_w4(x, rw, ids, ws, swiglu_limit=limit)
    assert torch.isfinite(clean).all()
    x[0, 3] = float("nan")
    lost = [0]
    if how != "mxfp4":
        x[1, 200] = float("-inf")
        lost.append(1)
    got = mok.forward_w4(x, rw, ids, ws, swiglu_limit=limit)
    kept = [t for t in range(T) if t not in lost]
    assert torch.isnan(got[lost]).all() and torch.equal(got[kept], clean[kept])
    for name in ("routed_gate", "routed_up"):
        x, rw, ids, ws, _ = layer_case(20, T, 256, 128, 8, 2, 128, how)
        ids[:] = ids % 6
        ids[2, 0] = 7
        scale = ws[name + "_scale"]
        scale[7, 5, 0] = 255 if how == "mxfp4" else float("nan")
        got = mok.forward_w4(x, rw, ids, ws, swiglu_limit=limit)
        kept = [t for t in range(T) if t != 2]
        assert torch.isnan(got[2]).all() and torch.equal(got[kept], clean[kept])
