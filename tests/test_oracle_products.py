"""Pins of oracle/products.py against something other than itself."""
import numpy as np
import pytest

from mokutil import ROOT  # noqa: F401
from oracle import moe as omoe
from oracle import products as op


def test_grouped_brute_force_and_gradients():
    rng = np.random.default_rng(0)
    x, w, off = rng.normal(size=(9, 5)), rng.normal(size=(4, 3, 5)), [1, 3, 3, 7, 8]
    y = op.grouped(x, w, off)
    for r in range(9):
        e = next((e for e in range(4) if off[e] <= r < off[e + 1]), None)
        for n in range(3):
            want = 0.0 if e is None else sum(w[e, n, k] * x[r, k] for k in range(5))
            assert abs(y[r, n] - want) < 1e-12
    # differences of a loss that is linear in y (so the quotient is exact but for rounding)
    dy = rng.normal(size=(9, 3))
    dx, dw = op.grouped_backward(dy, x, w, off)
    d = 1e-3
    for at in np.ndindex(*x.shape):
        xp = x.copy()
        xp[at] += d
        assert abs(((op.grouped(xp, w, off) - y) * dy).sum() / d - dx[at]) < 1e-9
    for at in np.ndindex(*w.shape):
        wp = w.copy()
        wp[at] += d
        assert abs(((op.grouped(x, wp, off) - y) * dy).sum() / d - dw[at]) < 1e-9


def test_bf16_against_torch():
    torch = pytest.importorskip("torch")
    v = np.concatenate([np.random.default_rng(1).normal(size=5000), [1.00390625, 1.01171875, 0.0, -2.0 ** -130]])
    v = v.astype(np.float32)
    assert np.array_equal(op.bf16(v), torch.from_numpy(v).to(torch.bfloat16).double().numpy())


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zero", [False, True])
def test_int4_is_within_half_a_step(group, zero):
    rng = np.random.default_rng(group)
    w = op.bf16(rng.normal(size=(3, 256)) * np.exp(rng.normal(size=(3, 1))))
    w[1, :group] = 0
    codes, scale, z = op.quantize(w, "int4", group, zero)
    assert codes.min() >= 0 and codes.max() <= 15
    v = op.values(codes, scale, z)
    step = np.repeat(scale, group, -1)
    # half a step; at the ends of the range a step more: the scale is rounded to bf16 and, with a zero point, so is it
    assert np.all(np.abs(v - w) <= (1.01 if zero else 0.54) * step)
    assert np.all(v[1, :group] == 0)
    assert np.array_equal(op.unpack(op.pack(codes)), codes)


def test_int4_by_hand():
    w = np.zeros((1, 32))
    w[0, :4] = [7.0, -7.0, 3.5, 2.5]      # amax 7: scale 1; ties to even
    codes, scale, _ = op.quantize(w, "int4", 32)
    assert scale[0, 0] == 1.0 and list(codes[0, :5]) == [15, 1, 12, 10, 8]
    w[0, :4] = [10.0, -5.0, 0.5, 1.5]     # range 15: scale 1, zero 5
    codes, scale, zero = op.quantize(w, "int4", 32, True)
    assert scale[0, 0] == 1.0 and zero[0, 0] == 5 and list(codes[0, :5]) == [15, 0, 5, 7, 5]


def test_mxfp4_nearest_by_brute_force():
    rng = np.random.default_rng(5)
    w = op.bf16(rng.normal(size=(8, 64)))
    w[0, :32] = np.concatenate([np.arange(0, 8, 0.25)])  # every tie at scale 1: amax 7.75, X = 0
    codes, scale, _ = op.quantize(w, "mxfp4", 32)
    assert scale[0, 0] == 127
    assert [op.E2M1[c] for c in codes[0, :32]] == [0, 0, .5, 1, 1, 1, 1.5, 2, 2, 2, 2, 3, 3, 3, 4, 4, 4, 4, 4, 4, 4, 6,
                                                   6, 6, 6, 6, 6, 6, 6, 6, 6, 6]
    v = op.values(codes, scale, mxfp4=True)
    s = np.repeat(np.exp2(scale.astype(float) - 127), 32, -1)
    best = np.abs(np.abs(w / s)[..., None] - op.E2M1).min(-1) * s
    assert np.allclose(np.abs(v - w), best, rtol=0, atol=1e-12)
    amax = np.abs(w).reshape(8, 2, 32).max(-1)
    assert np.all((amax >= 4 * np.exp2(scale - 127.0)) & (amax < 8 * np.exp2(scale - 127.0)))
    assert op.quantize(np.zeros((1, 32)), "mxfp4", 32)[1][0, 0] == 0


@pytest.mark.parametrize("limit", [0.0, 0.4])
def test_layer_is_the_layers_forward(limit):
    rng = np.random.default_rng(9)
    T, H, I, E, k = 5, 6, 4, 7, 3
    x, w = rng.normal(size=(T, H)), rng.random((T, k))
    ids = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int64)
    ids[2, 1], ids[3] = -1, -1
    g, u, d = rng.normal(size=(E, I, H)), rng.normal(size=(E, I, H)), rng.normal(size=(E, H, I))
    s = rng.normal(size=(3, H)), rng.normal(size=(3, H)), rng.normal(size=(H, 3))
    want = omoe.forward(x, ids, w, g, u, d, *s, swiglu_limit=limit)
    assert np.allclose(op.layer(x, w, ids, g, u, d, s, limit), want, rtol=1e-12, atol=1e-12)
