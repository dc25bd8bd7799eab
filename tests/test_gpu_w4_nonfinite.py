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


@pytest.mark.parametrize("T", [1, 4, 20])
@pytest.mark.parametrize("kind", ["routed", "shared"])
def test_h_beyond_the_largest_bf16(T, kind):
    """MXFP4, h of one column: x^2 1.5 2^96 with x = 209 2^8, fp32's 0.99978 2^128, which rounds to no bf16, and an
    infinity. Both come out as h times the weight, 2^-100 (1 and -6 of it), the first rounded once: h is exact, since
    silu(g) is g at these sizes. (x = 2^127 makes g = 2^175 and u 1.5 times that.)"""
    H, I = 128, 128
    ws, n = {}, 1 if kind == "routed" else 0
    codes = {"gate": np.zeros((I, H), np.uint8), "up": np.zeros((I, H), np.uint8), "down": np.zeros((H, I), np.uint8)}
    codes["gate"][70, 5], codes["up"][70, 5] = 2, 3   # 1 and 1.5
    codes["down"][::2, 70], codes["down"][1::2, 70] = 2, 15  # 1 and -6
    scale = {"gate": 48, "up": 48, "down": -100}

    def put(name, c, s):
        ws[name] = torch.from_numpy(c[..., 0::2] | c[..., 1::2] << 4).cuda()
        ws[name + "_scale"] = torch.full(c.shape[:-1] + (c.shape[-1] // 32,), s + 127, dtype=torch.uint8).cuda()

    for name, c in codes.items():
        put("routed_" + name, (c if kind == "routed" else 0 * c)[None], scale[name])
        if kind == "shared":
            put("shared_" + name, c, scale[name])
    x = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
    x[:, 5] = 209 * 2.0 ** 8
    if T > 1:
        x[1, 5] = 2.0 ** 127
        x[2, 5] = 1
    got = mok.forward_w4(x, torch.ones(T, 1, device="cuda"), torch.zeros(T, 1, dtype=torch.int64, device="cuda"), ws)
    w = np.where(np.arange(H) % 2, -6.0, 1.0) * 2.0 ** -100
    h = 209.0 ** 2 * 2.0 ** 16 * 1.5 * 2.0 ** 96
    assert np.float32(h) == h and 255.5 * 2.0 ** 120 < h < 2.0 ** 128
    got = got.cpu().double().numpy()
    for t in range(T):
        if t == 1:
            assert np.array_equal(got[t], np.inf * w)
        else:
            want = w * (1.5 * 2.0 ** 96 if t == 2 else h)
            assert (np.abs(got[t] - want) <= 2.0 ** -8 * np.abs(want)).all()


def test_an_infinite_limit_is_none():
    """As in MoKConfig, which takes 0 and +inf for no limit; what MoKConfig refuses is refused."""
    mok.create_workspace(mok.MoKConfig(256, 128, 8, 2, 16, swiglu_limit=float("inf")))
    x, rw, ids, ws, _ = layer_case(30, 5, 256, 128, 8, 2, 0, "sym128")
    want = mok.forward_w4(x, rw, ids, ws)
    for limit in (float("inf"), np.inf, 1e39):
        assert torch.equal(mok.forward_w4(x, rw, ids, ws, swiglu_limit=limit), want)
    assert not torch.equal(mok.forward_w4(x, rw, ids, ws, swiglu_limit=0.01), want)
    for limit in (float("-inf"), float("nan"), -1e39):
        with pytest.raises(mok.MokError):
            mok.forward_w4(x, rw, ids, ws, swiglu_limit=limit)
