"""How exactly the 4-bit layer holds h between its two products.

Each x has one column that is not zero, so g and u are exact (a code's value times x), and only two columns of h are
not zero (the others' rows of the up projection are zeros), so an output is h1 w1 + h2 w2: over all tokens and rows
some of them leave little of each other, and there h's last bits show.

Tolerance: 2^-8 of the value for the rounding to bf16, and of |h1 w1| + |h2 w2|
  h in fp32: exp(-g) by a product with log2 e and the hardware's exp2, (1.5 |g| + 2) 2^-24, then an addition, a
    division and a product, 2^-24 each: (1.5 |g| + 5) 2^-24; |g| <= 4 here: 11
  MXFP4: h in parts that add up to it, exact products, six sums of at most 2^-23 each: 12
  int4: the sums are those of (16 + code) h and of (16 + 8) h, at most 31 scale |h| each, six terms in both, the
    product and the difference: 14 * 2^-23 * 31 scale (|h1| + |h2|)."""
import numpy as np
import pytest

from mokutil import ROOT  # noqa: F401
from oracle import products as op
from test_gpu_w4 import check_layer, layer_case

torch = pytest.importorskip("torch")
import mixture_experts_layer_build_amd as mok  # noqa: E402

FORMATS = {"sym128": 128, "sym64": 64, "sym32": 32, "zero32": 32, "mxfp4": 32}
EPS = 2.0 ** -24


def case(seed, how, T, H, I):
    """x, and codes of gate, up and down; every scale is 2^-3."""
    rng = np.random.default_rng(seed)
    mx = how == "mxfp4"
    none = 0 if mx else 8
    x = np.zeros((T, H))
    x[np.arange(T), rng.integers(0, H, T)] = rng.choice([-1, 1], T) * op.bf16(rng.uniform(1, 4, T))
    codes = lambda *shape: rng.integers(0, 16, shape)  # noqa: E731
    gate, up, down = codes(I, H), np.full((I, H), none), codes(H, I)
    up[[3, I - 51]] = codes(2, H)
    return x, gate, up, down


def values(c, how):
    if how == "mxfp4":
        return np.where(c > 7, -1.0, 1.0) * op.E2M1[c & 7] / 8
    return (c - 8) / 8


def want_of(x, gate, up, down, how, split=lambda h: h):
    """(output, its bound) with h as `split` leaves it."""
    g, u, d = x @ values(gate, how).T, x @ values(up, how).T, values(down, how)
    assert np.abs(g).max() <= 4
    h = split(g / (1 + np.exp(-g)) * u)
    y, mags = h @ d.T, np.abs(h) @ np.abs(d).T
    sums = 12 * EPS * mags if how == "mxfp4" else 14 * 2 * EPS * 31 / 8 * np.abs(h).sum(1, keepdims=True)
    return y, 2.0 ** -8 * np.abs(y) + (1 + 2.0 ** -8) * (11 * EPS * mags + sums)


def parts(n):
    """h as n bf16 that add up to it."""
    def split(h):
        rest, out = h.astype(np.float32), np.zeros(h.shape)
        for _ in range(n):
            p = op.bf16(rest)
            rest, out = (rest - p).astype(np.float32), out + p
        return out
    return split


SIZES = [(200, 512, 128), (200, 256, 384), (16, 1024, 128), (64, 1024, 256), (5, 2048, 384), (2, 2048, 128)]


@pytest.mark.parametrize("how", FORMATS)
def test_the_bound_tells_the_parts_of_h(how):
    """One bf16 fails it and, in MXFP4 with many tokens, two do; three pass."""
    for T, H, I in SIZES:
        c = case(T + I, how, T, H, I)
        y, lim = want_of(*c, how)
        far = [(np.abs(op.bf16(want_of(*c, how, parts(n))[0]) - y) > lim).sum() for n in (1, 2, 3)]
        assert far[0] > 0 and far[2] == 0
        assert how != "mxfp4" or far[1] > 0 or T < 200


@pytest.mark.gpu
@pytest.mark.parametrize("how", FORMATS)
@pytest.mark.parametrize("T,H,I", SIZES)
@pytest.mark.parametrize("kind", ["routed", "shared"])
def test_layer_holds_h(how, T, H, I, kind):
    c = case(T + I, how, T, H, I)
    y, lim = want_of(*c, how)
    mx, group = how == "mxfp4", FORMATS[how]
    ws = {}

    def put(name, codes):
        shape = codes.shape[:-1] + (codes.shape[-1] // group,)
        ws[name] = torch.from_numpy(op.pack(codes)).cuda()
        ws[name + "_scale"] = (torch.full(shape, 124, dtype=torch.uint8) if mx else
                               torch.full(shape, 2.0 ** -3, dtype=torch.bfloat16)).cuda()
        if how == "zero32":
            ws[name + "_zero"] = torch.full(shape, 8, dtype=torch.uint8).cuda()

    none = 0 if mx else 8
    for name, codes in zip(("gate", "up", "down"), c[1:]):
        put("routed_" + name, (codes if kind == "routed" else np.full(codes.shape, none))[None])
        if kind == "shared":
            put("shared_" + name, codes)
    x = torch.from_numpy(c[0]).to(torch.bfloat16).cuda()
    got = mok.forward_w4(x, torch.ones(T, 1, device="cuda"), torch.zeros(T, 1, dtype=torch.int64, device="cuda"), ws)
    bad = np.abs(got.cpu().double().numpy() - y) > lim
    assert not bad.any(), f"{bad.sum()} of {bad.size} off"


@pytest.mark.gpu
@pytest.mark.parametrize("how", ["sym128", "zero64", "sym32", "mxfp4"])
@pytest.mark.parametrize("T,k", [(5, 3), (5, 1), (4, 4), (6, 2), (5, 4), (6, 1), (3, 5)])
def test_layer_at_the_limits_of_the_rows_of_h(how, T, k):
    """Five tokens' parts fill a row tile; a token that is not finite, or chose an expert that is not, keeps it."""
    x, rw, ids, ws, vs = layer_case(T + k, T, 256, 128, 7, k, 128 if T % 2 else 0, how)
    ids[T - 1, 0] = -1
    if k > 1:
        ids[0, 0] = ids[0, 1] = 3
    check_layer(x, rw, ids, ws, vs, how)
    ids[ids == 6] = 2
    ids[1, 0] = 6
    clean = mok.forward_w4(x, rw, ids, ws)
    x[0, 3] = float("nan")
    if how != "mxfp4":
        ws["routed_down_scale"][6] = float("nan")
    else:
        ws["routed_down_scale"][6] = 255
    got = mok.forward_w4(x, rw, ids, ws)
    assert torch.isnan(got[1]).all() and torch.isnan(got[0]).all() and torch.equal(got[2:], clean[2:])


@pytest.mark.gpu
@pytest.mark.parametrize("T,k", [(1, 8), (5, 3), (12, 8)])
def test_decoding_captured_and_replayed(T, k):
    """Two graphs of the layer, replayed in turn between eager calls on new inputs."""
    x, rw, ids, ws, _ = layer_case(40 + T, T, 256, 128, 16, k, 128, "zero64")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        mok.forward_w4(x, rw, ids, ws)
    torch.cuda.current_stream().wait_stream(s)
    graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    out = []
    for g in graphs:
        with torch.cuda.graph(g):
            out.append(mok.forward_w4(x, rw, ids, ws, swiglu_limit=2.0))
    for seed in (50, 51, 52):
        new = layer_case(seed, T, 256, 128, 16, k, 128, "zero64")[:3]
        for to, of in zip((x, rw, ids), new):
            to.copy_(of)
        graphs[seed % 2].replay()
        want = mok.forward_w4(*new, ws, swiglu_limit=2.0)
        graphs[1 - seed % 2].replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0], want) and torch.equal(out[1], want)
