"""Pins of oracle/ops.py: gradients against central differences, the AdamW
formula against torch's own optimizer in float64, the router against brute
force, the 8-bit states' code table and scale rule against closed forms."""
import numpy as np
import pytest

from mokutil import ROOT  # noqa: F401
from oracle import ops as oops

torch = pytest.importorskip("torch")


def differences(f, x, h):
    g = np.zeros_like(x)
    it = np.nditer(x, flags=["multi_index"])
    for _ in it:
        i = it.multi_index
        a, b = x.copy(), x.copy()
        a[i] += h
        b[i] -= h
        g[i] = (f(a) - f(b)) / (2 * h)
    return g


def test_rms_norm_gradient_against_differences():
    rng = np.random.default_rng(1)
    s, w, dy, dsum = rng.standard_normal((3, 7)), rng.standard_normal(7), rng.standard_normal((3, 7)), \
        rng.standard_normal((3, 7))

    def loss(s, w):
        y, t, _ = oops.rms_norm(s, w)
        return (y * dy).sum() + (t * dsum).sum()

    _, _, rstd = oops.rms_norm(s, w)
    ds, dw = oops.rms_norm_backward(dy, s, rstd, w, dsum)
    # central differences: error h^2 f''' / 6 + 1e-16 / h, about 1e-9 at h = 1e-5
    np.testing.assert_allclose(ds, differences(lambda t: loss(t, w), s, 1e-5), atol=1e-7)
    np.testing.assert_allclose(dw, differences(lambda t: loss(s, t), w, 1e-5), atol=1e-7)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_router_gradient_against_differences(scoring, renorm):
    rng = np.random.default_rng(2)
    T, E, k = 4, 6, 2
    # differences on a float64 copy of the router's smooth part: ids and counts are constants
    l = rng.standard_normal((T, E)).astype(np.float32)
    mask = np.array([1, 1, 0, 1])
    dw, dl = rng.standard_normal((T, k)), np.array([0.7, 0.3])
    _, ids, counts, _ = oops.router(l, k, scoring, renorm, 1.5, mask=mask)

    def loss(x):
        tot = 0.0
        for t in range(T):
            if not mask[t]:
                continue
            s = np.exp(x[t]) / np.exp(x[t]).sum() if scoring == "softmax" else 1 / (1 + np.exp(-x[t]))
            w = s[ids[t]]
            if renorm:
                w = w / w.sum()
            n = counts[E]
            tot += (w * 1.5 * dw[t]).sum() + dl[0] * E / k / n / n * (counts[:E] * s / s.sum()).sum()
            if scoring == "softmax":
                tot += dl[1] * np.log(np.exp(x[t]).sum()) ** 2 / n
        return tot

    got = oops.router_backward(dw, l, ids, scoring, renorm, 1.5, mask=mask, counts=counts, d_losses=dl)
    np.testing.assert_allclose(got, differences(loss, l.astype(np.float64), 1e-5), atol=1e-7)


def test_router_against_torch_topk_and_its_rules():
    rng = np.random.default_rng(3)
    l = rng.standard_normal((20, 9)).astype(np.float32)
    w, ids, counts, losses = oops.router(l, 3)
    v, i = torch.topk(torch.from_numpy(l), 3, dim=1)
    np.testing.assert_array_equal(ids, i.numpy())
    np.testing.assert_allclose(w, torch.softmax(v.double(), 1).numpy(), rtol=1e-12)
    assert counts[:9].sum() == 60 and counts[9] == 20
    p = torch.softmax(torch.from_numpy(l).double(), 1).numpy()
    np.testing.assert_allclose(losses[0], 9 / 3 * (counts[:9] / 20 * p.mean(0)).sum(), rtol=1e-12)
    # ties to the lowest id; -inf never chosen; a NaN row has no order; a masked row nothing
    l[0] = 1.0
    l[1, 2:] = -np.inf
    l[2] = -np.inf
    l[3, 5] = np.nan
    l[4] = np.nan
    mask = np.ones(20)
    mask[4] = 0
    w, ids, counts, _ = oops.router(l, 3, mask=mask)
    assert ids[0].tolist() == [0, 1, 2] and set(ids[1, :2]) == {0, 1} and ids[1, 2] == -1 and w[1, 2] == 0
    assert (ids[2] == -1).all() and (w[2] == 0).all()
    assert (ids[3] == -1).all() and np.isnan(w[3]).all()
    assert (ids[4] == -1).all() and (w[4] == 0).all()
    assert counts[9] == 18


def test_adamw_against_torch():
    rng = np.random.default_rng(4)
    p0 = rng.standard_normal(50)
    p = torch.nn.Parameter(torch.from_numpy(p0.copy()))
    opt = torch.optim.AdamW([p], lr=1e-2, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.1)
    q, m, v = p0.copy(), np.zeros(50), np.zeros(50)
    for step in range(1, 6):
        g = rng.standard_normal(50)
        p.grad = torch.from_numpy(g.copy())
        opt.step()
        q, m, v = oops.adamw(q, g, m, v, step, 1e-2, 0.9, 0.95, 1e-8, 0.1)
    np.testing.assert_allclose(q, p.detach().numpy(), rtol=1e-10)


def test_codes_and_scales():
    codes = np.arange(256, dtype=np.uint8)
    codes[0x7F] = codes[0xFF] = 0  # the NaN codes are never written
    want = torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(oops.decode8(codes, np.full(8, 127)), want)
    np.testing.assert_array_equal(oops.decode8(codes, np.full(8, 130)), want * 8)
    for a, x in ((448.0, 0), (448.0001, 1), (449.0, 1), (224.0, -1), (0.0, -127), (448 * 2.0 ** 5, 5), (256.0, 0)):
        assert oops.state_exponent([0.0, -a, a / 3])[0] == x, a


def test_uniforms_are_spread_evenly_and_independent():
    n = 1 << 18
    for seed in (1, 12345, 0xFFFFFFFF):
        u = oops.uniforms(n, seed)
        # mean 1/2, variance 1/12: the mean's standard deviation is 0.289 / 512 = 5.6e-4, five of them 2.8e-3
        assert abs(u.mean() - 0.5) < 2.8e-3
        h = np.histogram(u, 64, (0, 1))[0]  # 4096 each, standard deviation 64, six of them
        assert np.abs(h - n / 64).max() < 6 * 64
        for lag in (1, 2, 32):  # correlation of n pairs: standard deviation 1 / 512, five of them
            assert abs(np.corrcoef(u[:-lag], u[lag:])[0, 1]) < 5 / 512
    a, b = oops.uniforms(n, 0xD1B54A35), oops.uniforms(n, 2 * 0xD1B54A35 & 0xFFFFFFFF)  # seeds of successive steps
    assert abs(np.corrcoef(a, b)[0, 1]) < 5 / 512
