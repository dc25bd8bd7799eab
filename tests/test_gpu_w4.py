"""4-bit weights: the quantizer and its inverse bit for bit, and the products
with them against float64.

Tolerance of a product, per element: 2^-8 of the value for the rounding to bf16
(half a step), and for the fp32 sums 8 sqrt(n) 2^-24 of the sum of magnitudes,
n terms (each of n roundings is at most 2^-24 of a partial sum, their signs are
independent, 8 standard deviations). int4 sums are those of (128 + code) x, less
(128 + zero) sum x: their magnitudes are up to 271 scale |x|."""
import numpy as np
import pytest

from mokutil import ROOT  # noqa: F401
from oracle import products as op

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import mixture_experts_layer_build_amd as mok  # noqa: E402

FORMATS = {"sym128": ("int4", 128, False), "sym64": ("int4", 64, False), "sym32": ("int4", 32, False),
           "zero128": ("int4", 128, True), "zero64": ("int4", 64, True), "zero32": ("int4", 32, True),
           "mxfp4": ("mxfp4", 32, False)}


def normal(seed, *shape, std=1.0, dtype=torch.bfloat16):
    gen = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=gen) * std).to(dtype)


def f64(t):
    return None if t is None else t.detach().cpu().double().numpy()


def w4(w, how):
    """(codes, scale, zero) on the GPU and the values in float64."""
    form, group, zero = FORMATS[how]
    c, s, z = op.quantize(f64(w), form, group, zero)
    v = op.values(c, s, z, form == "mxfp4")
    scale = torch.from_numpy(s) if form == "mxfp4" else torch.from_numpy(s).to(torch.bfloat16)
    return (torch.from_numpy(op.pack(c)).cuda(), scale.cuda(),
            None if z is None else torch.from_numpy(z.astype(np.uint8)).cuda()), v


def mags_of(x, v, scale, how):
    """Bound of the sums' magnitudes for the products x v^T."""
    form, group, _ = FORMATS[how]
    per = np.abs(v) if form == "mxfp4" else 271 * np.repeat(f64(scale), group, -1)
    return np.abs(x) @ per.T


def close(got, want, lim, what=""):
    got = f64(got)
    assert got.shape == want.shape
    bad = ~(np.abs(got - want) <= lim)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, first at {np.argwhere(bad)[0]}"


# ---- quantizer ----

@pytest.mark.parametrize("how", FORMATS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_quantize_and_back(how, dtype):
    form, group, zero = FORMATS[how]
    w = normal(1, 5, 7, 384, dtype=dtype) * torch.exp2(torch.arange(5 * 7).view(5, 7, 1) % 23 - 11).to(dtype)
    w[0, 0, :group] = 0
    w[0, 1, :group] = -0.0
    w[0, 2, :group] = w[0, 2, :group].abs()
    w[0, 3, :group] = -w[0, 3, :group].abs()
    w[0, 4, 0:384:3] = 0
    w[1, 0, :8] = torch.tensor([7, -7, 3.5, 2.5, 1.5, 0.5, -0.5, -3.5], dtype=dtype)
    codes, scale, z = mok.w4_quantize(w.cuda(), form, group, zero)
    wc, ws, wz = op.quantize(f64(w), form, group, zero)
    assert codes.shape == (5, 7, 192) and scale.shape == (5, 7, 384 // group)
    assert np.array_equal(f64(scale), ws.astype(np.float64))
    assert np.array_equal(op.unpack(codes.cpu().numpy()), wc)
    assert z is None if wz is None else np.array_equal(z.cpu().numpy(), wz)
    back = mok.w4_dequantize(codes, scale, z)
    assert back.dtype == torch.bfloat16 and back.shape == w.shape
    assert np.array_equal(f64(back), op.bf16(op.values(wc, ws, wz, form == "mxfp4").astype(np.float32)))


@pytest.mark.parametrize("how", ["sym128", "zero32", "mxfp4"])
def test_quantize_strided_rows_and_extremes(how):
    form, group, zero = FORMATS[how]
    wide = normal(2, 9, 512, dtype=torch.float32)
    wide[3] *= 2.0 ** -120
    wide[4] *= 2.0 ** 100
    wide[5] = 2.0 ** -149
    got = mok.w4_quantize(wide.cuda()[:, 128:384], form, group, zero)
    want = mok.w4_quantize(wide[:, 128:384].contiguous().cuda(), form, group, zero)
    assert all((a is None and b is None) or torch.equal(a, b) for a, b in zip(got, want))
    wc, ws, _ = op.quantize(f64(wide[:, 128:384]), form, group, zero)
    assert np.array_equal(f64(got[1]), ws.astype(np.float64)) and np.array_equal(op.unpack(got[0].cpu().numpy()), wc)


def test_quantize_nothing():
    for shape in ((0, 64), (3, 0, 64)):
        codes, scale, z = mok.w4_quantize(torch.empty(shape, dtype=torch.bfloat16, device="cuda"), "mxfp4")
        assert codes.shape == shape[:-1] + (32,) and scale.shape == shape[:-1] + (2,)
        assert mok.w4_dequantize(codes, scale).shape == shape


def test_every_code_and_scale_of_mxfp4():
    codes = torch.arange(256, dtype=torch.uint8).repeat(255)[:255 * 16].view(255, 16).cuda()
    scale = torch.arange(255, dtype=torch.uint8).view(255, 1).cuda()
    want = op.values(op.unpack(codes.cpu().numpy()), scale.cpu().numpy(), mxfp4=True)
    # (values below 2^-133 are below bf16's smallest; those above its largest are infinite)
    w32 = torch.from_numpy(want).to(torch.float32).to(torch.bfloat16)
    assert torch.equal(mok.w4_dequantize(codes, scale).cpu(), w32)


# ---- product ----

@pytest.mark.parametrize("how", FORMATS)
@pytest.mark.parametrize("T,n,k", [(1, 16, 128), (1, 1, 128), (3, 50, 384), (16, 64, 1024), (17, 33, 256),
                                   (64, 48, 512), (65, 31, 640), (130, 16, 2048)])
def test_product(how, T, n, k):
    x = normal(T + n, T, k).cuda()
    q, v = w4(normal(k, n, k, std=0.05), how)
    X = f64(x)
    want = X @ v.T
    lim = 2.0 ** -8 * np.abs(want) + 8 * k ** 0.5 * 2.0 ** -24 * mags_of(X, v, q[1], how)
    close(mok.w4_matmul(x, *q), want, lim)


@pytest.mark.parametrize("how,k", [("sym32", 32), ("sym32", 160), ("zero32", 1568), ("sym64", 192), ("zero64", 64),
                                   ("mxfp4", 32), ("mxfp4", 96), ("mxfp4", 1568)])
@pytest.mark.parametrize("T", [1, 20])
def test_widths_that_end_inside_a_chunk(how, k, T):
    q, v = w4(normal(k, 37, k, std=0.05), how)
    x = normal(T, T, k)
    X = f64(x)
    want = X @ v.T
    lim = 2.0 ** -8 * np.abs(want) + 8 * k ** 0.5 * 2.0 ** -24 * mags_of(X, v, q[1], how)
    close(mok.w4_matmul(x.cuda(), *q), want, lim)


def test_product_layout():
    """One x and one weight that are not zero, everywhere: the columns' order is the codes'."""
    for how in FORMATS:
        q, v = w4(torch.eye(256).to(torch.bfloat16), how)
        x = torch.eye(256).to(torch.bfloat16).cuda()
        assert np.array_equal(f64(mok.w4_matmul(x, *q)), op.bf16(v.T.astype(np.float32))), how


def test_product_shapes_strides_and_special_rows():
    q, v = w4(normal(3, 40, 256, std=0.05), "zero64")
    x = normal(4, 2, 3, 256).cuda()
    y = mok.w4_matmul(x, *q)
    assert y.shape == (2, 3, 40) and torch.equal(y.view(6, 40), mok.w4_matmul(x.view(6, 256), *q))
    assert mok.w4_matmul(x[:0], *q).shape == (0, 3, 40)
    wide = torch.full((6, 512), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, 128:384] = x.view(6, 256)
    assert torch.equal(mok.w4_matmul(wide[:, 128:384], *q), y.view(6, 40))
    bad = x.view(6, 256).clone()
    bad[2, 7], bad[4, 9] = float("nan"), float("inf")
    got = mok.w4_matmul(bad, *q)
    good = [0, 1, 3, 5]
    assert torch.equal(got[good], y.view(6, 40)[good]) and not torch.isfinite(got[[2, 4]].float()).any()
    with pytest.raises(mok.MokError):
        mok.w4_matmul(wide[:, 1:257], *q)


def test_rows_do_not_depend_on_the_batch():
    """A row of x gives the same bits alone and among others of its own kernel (up to 16 rows; more)."""
    q, _ = w4(normal(5, 80, 1024, std=0.05), "sym128")
    x = normal(6, 150, 1024).cuda()
    one = torch.cat([mok.w4_matmul(x[i:i + 1], *q) for i in range(16)])
    assert torch.equal(one, mok.w4_matmul(x[:16], *q))
    assert torch.equal(mok.w4_matmul(x, *q)[:64], mok.w4_matmul(x[:64], *q))


# ---- layer ----

def layer_case(seed, T, H, I, E, k, Is, how, std=0.05):
    ws, vs = {}, {}
    shapes = dict(routed_gate=(E, I, H), routed_up=(E, I, H), routed_down=(E, H, I))
    if Is:
        shapes.update(shared_gate=(Is, H), shared_up=(Is, H), shared_down=(H, Is))
    for i, (name, shape) in enumerate(shapes.items()):
        q, vs[name] = w4(normal(seed + i, *shape, std=std), how)
        ws[name], ws[name + "_scale"] = q[0], q[1]
        if q[2] is not None:
            ws[name + "_zero"] = q[2]
    rng = np.random.default_rng(seed)
    ids = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int64) if T else np.zeros((0, k), np.int64)
    rw = rng.random((T, k)).astype(np.float32)
    return normal(seed + 9, T, H).cuda(), torch.from_numpy(rw).cuda(), torch.from_numpy(ids).cuda(), ws, vs


def check_layer(x, rw, ids, ws, vs, how, limit=0.0, got=None):
    """h is off by 2^-8 of itself (its rounding to bf16) and by what g's and u's sums are off, which reach it times at
    most 1.1 |u| and |silu(g)|."""
    X, RW, ID = f64(x), f64(rw), ids.cpu().numpy()
    want, lim = np.zeros(X.shape), np.zeros(X.shape)

    def add(rows, kind, e, weight):
        def part(name):
            v, s = vs[kind + name], ws[kind + name + "_scale"]
            return (v, s) if e is None else (v[e], s[e])
        (g, sg), (u, su), (d, sd) = part("gate"), part("up"), part("down")
        xr = X[rows]
        n = 8 * X.shape[1] ** 0.5 * 2.0 ** -24
        G, U = xr @ g.T, xr @ u.T
        y, h = op.mlp(xr, g, u, d, limit)
        eh = (2.0 ** -8 + 2.0 ** -18) * np.abs(h) + n * (1.1 * np.abs(U) * mags_of(xr, g, sg, how) +
                                                        (np.abs(G) + 0.3) * mags_of(xr, u, su, how))
        want[rows] += weight * y
        lim[rows] += np.abs(weight) * (eh @ np.abs(d).T + 8 * h.shape[1] ** 0.5 * 2.0 ** -24 *
                                       mags_of(np.abs(h) + eh, d, sd, how))

    if "shared_gate" in ws:
        add(np.arange(X.shape[0]), "shared_", None, 1.0)
    for t in range(X.shape[0]):
        for j in range(ID.shape[1]):
            if 0 <= ID[t, j] < ws["routed_gate"].shape[0]:
                add(np.array([t]), "routed_", int(ID[t, j]), RW[t, j])
    got = mok.forward_w4(x, rw, ids, ws, swiglu_limit=limit) if got is None else got
    close(got, want, 2.0 ** -8 * np.abs(want) + (1 + 2.0 ** -7) * lim)


@pytest.mark.parametrize("how", FORMATS)
@pytest.mark.parametrize("T,H,I,E,k,Is", [(1, 256, 128, 8, 2, 0), (1, 384, 256, 16, 4, 128), (5, 256, 384, 8, 3, 256),
                                          (16, 128, 128, 4, 4, 0), (19, 256, 128, 40, 8, 384), (70, 128, 256, 6, 2, 128)])
def test_layer(how, T, H, I, E, k, Is):
    check_layer(*layer_case(T + H, T, H, I, E, k, Is, how), how)


@pytest.mark.parametrize("how", ["sym32", "mxfp4"])
def test_layer_widths_of_32(how):
    check_layer(*layer_case(3, 9, 160, 96, 5, 2, 32, how), how)
    check_layer(*layer_case(4, 21, 32, 32, 3, 1, 224, how), how)


@pytest.mark.parametrize("limit", [0.3, 5.0])
def test_layer_limit(limit):
    check_layer(*layer_case(5, 6, 256, 128, 8, 2, 128, "sym64", std=0.1), "sym64", limit=limit)


@pytest.mark.parametrize("T", [3, 33])
def test_layer_choices_that_are_none_and_choices_twice(T):
    x, rw, ids, ws, vs = layer_case(6, T, 256, 128, 8, 4, 0, "zero64")
    ids[0] = -1                     # a token without a choice: zeros
    ids[1, 1], ids[1, 3] = -1, 8    # outside the experts
    ids[2, 0] = ids[2, 2] = ids[2, 3] = 5
    ids[T - 1, 1] = 1 << 40
    rw[1, 1] = float("nan")         # (no choice: its weight is not read)
    check_layer(x, rw.nan_to_num(0.0), ids, ws, vs, "zero64")
    got = mok.forward_w4(x, rw, ids, ws)
    assert not got[0].any()
    check_layer(x, rw.nan_to_num(0.0), ids, ws, vs, "zero64", got=got)


def test_layer_every_token_one_expert_and_none_at_all():
    x, rw, ids, ws, vs = layer_case(7, 50, 128, 128, 4, 1, 128, "mxfp4")
    ids.fill_(2)
    check_layer(x, rw, ids, ws, vs, "mxfp4")
    ids.fill_(-1)
    check_layer(x, rw, ids, ws, vs, "mxfp4")
    none = {n: t for n, t in ws.items() if n.startswith("routed")}
    assert not mok.forward_w4(x, rw, ids, none).any()
    assert mok.forward_w4(x[:0], rw[:0], ids[:0], ws).shape == (0, 128)


def test_layer_tokens_do_not_mix():
    """What is not finite in one token, or in an expert that one token chose, reaches no other token."""
    x, rw, ids, ws, vs = layer_case(8, 12, 256, 128, 8, 2, 0, "sym128")
    ids[:] = ids % 7
    ids[4, 1] = 7
    clean = mok.forward_w4(x, rw, ids, ws)
    others = [t for t in range(12) if t not in (4, 9)]
    ws["routed_down_scale"][7] = float("nan")
    ws["routed_gate_scale"][7] = float("inf")
    x[9, 3] = float("nan")
    got = mok.forward_w4(x, rw, ids, ws)
    assert torch.equal(got[others], clean[others])
    assert torch.isnan(got[4]).any() and torch.isnan(got[9]).all()


@pytest.mark.parametrize("T,E,k", [(64, 300, 8), (128, 1024, 64), (8192, 4, 1), (100, 64, 64)])
def test_layer_limits(T, E, k):
    """More experts than a byte numbers, 64 choices, the most tokens: a few tokens against float64."""
    x, rw, ids, ws, vs = layer_case(10, T, 128, 32, E, k, 32, "sym32")
    got = mok.forward_w4(x, rw, ids, ws)
    some = [0, 1, T // 2, T - 1]
    check_layer(x[some], rw[some], ids[some], ws, vs, "sym32", got=got[some])


def test_layer_out_and_repeats():
    x, rw, ids, ws, vs = layer_case(11, 10, 256, 128, 8, 2, 128, "mxfp4")
    want = mok.forward_w4(x, rw, ids, ws)
    out = torch.empty_like(x)
    before = out._version
    assert mok.forward_w4(x, rw, ids, ws, out=out) is not None and out._version > before
    assert torch.equal(out, want)
    for _ in range(3):
        assert torch.equal(mok.forward_w4(x, rw, ids, ws), want)


def test_captured_and_replayed_with_new_inputs():
    how = "sym64"
    x, rw, ids, ws, vs = layer_case(12, 7, 256, 128, 16, 3, 128, how)
    w, sc = ws["shared_gate"], ws["shared_gate_scale"]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        mok.forward_w4(x, rw, ids, ws)
    torch.cuda.current_stream().wait_stream(s)
    g, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y, p = mok.forward_w4(x, rw, ids, ws), mok.w4_matmul(x, w, sc)
    with torch.cuda.graph(g2):
        y2 = mok.forward_w4(x, rw, ids, ws)
    for seed in (13, 14, 15):
        nx, nrw, nids, _, _ = layer_case(seed, 7, 256, 128, 16, 3, 128, how)
        x.copy_(nx), rw.copy_(nrw), ids.copy_(nids)
        g.replay()
        g2.replay()
        torch.cuda.synchronize()
        want = mok.forward_w4(nx, nrw, nids, ws)
        assert torch.equal(y, want) and torch.equal(y2, want) and torch.equal(p, mok.w4_matmul(nx, w, sc))


def test_two_streams_at_once():
    a = layer_case(16, 9, 256, 128, 16, 3, 128, "zero32")
    b = layer_case(17, 40, 128, 256, 8, 2, 0, "mxfp4")
    want = [mok.forward_w4(*c[:4]) for c in (a, b)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [None, None]
    for _ in range(4):
        for i, c in enumerate((a, b)):
            with torch.cuda.stream(streams[i]):
                got[i] = mok.forward_w4(*c[:4])
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("how", ["sym128", "zero32", "mxfp4"])
@pytest.mark.parametrize("T,k", [(4, 4), (17, 1), (16, 1), (16, 4), (13, 5), (1, 16), (1, 17), (1, 64)])
def test_layer_at_the_limits_of_its_ways(how, T, k):
    """16 and 64 choices are where the layer changes its way: with choices made twice, by none, and of no expert."""
    E = max(k, 6)
    x, rw, ids, ws, vs = layer_case(50 + T + k, T, 256, 128, E, k, 128 if T % 2 else 0, how)
    if k > 1:
        ids[0, -1] = ids[0, 0]
        ids[T // 2, k // 2] = -1
    else:
        ids[: T // 2] = 3
        ids[T - 1] = E
    check_layer(x, rw, ids, ws, vs, how)


@pytest.mark.parametrize("how", FORMATS)
def test_scales_and_zero_points_at_their_own_alignment(how):
    """Whole chunks whose scales and zero points cannot be loaded at once."""
    (c, s, z), v = w4(normal(70, 48, 512, std=0.1), how)

    def shifted(t):
        if t is None:
            return None
        buf = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
        buf[1:] = t.reshape(-1)
        return buf[1:].view(t.shape)
    x = normal(71, 5, 512).cuda()
    got = mok.w4_matmul(x, c, shifted(s), shifted(z))
    want = f64(x) @ v.T
    close(got, want, 2.0 ** -8 * np.abs(want) + 8 * 512 ** 0.5 * 2.0 ** -24 * mags_of(f64(x), v, s, how))
    X, rw, ids, ws, vs = layer_case(72, 9, 256, 128, 8, 2, 128, how)
    moved = {n: shifted(t) if n.endswith(("scale", "zero")) else t for n, t in ws.items()}
    check_layer(X, rw, ids, ws, vs, how, got=mok.forward_w4(X, rw, ids, moved))


@pytest.mark.parametrize("how", ["sym128", "zero64", "mxfp4"])
def test_more_than_2_31_bytes_of_codes(how):
    """The last expert of a large set gives what it gives alone; quantizing past 2^31 elements gives its rows' codes."""
    E, H, I = 300, 8192, 2048
    form, group, zero = FORMATS[how]
    gen = torch.Generator(device="cuda").manual_seed(1)
    ws = {}
    for name, n, k in (("gate", I, H), ("up", I, H), ("down", H, I)):
        ws["routed_" + name] = torch.randint(0, 256, (E, n, k // 2), dtype=torch.uint8, device="cuda", generator=gen)
        if form == "mxfp4":
            s = torch.randint(115, 122, (E, n, k // group), dtype=torch.uint8, device="cuda", generator=gen)
        else:
            s = torch.rand(E, n, k // group, device="cuda", generator=gen).mul_(0.02).to(torch.bfloat16)
        ws[f"routed_{name}_scale"] = s
        if zero:
            ws[f"routed_{name}_zero"] = torch.randint(0, 16, s.shape, dtype=torch.uint8, device="cuda", generator=gen)
    last = {n: t[-1:].clone() for n, t in ws.items()}
    for T in (2, 20):
        x, rw = normal(80, T, H).cuda(), torch.rand(T, 1, device="cuda", generator=gen)
        ids = torch.full((T, 1), E - 1, dtype=torch.int64, device="cuda")
        assert torch.equal(mok.forward_w4(x, rw, ids, ws), mok.forward_w4(x, rw, torch.zeros_like(ids), last))
    del ws
    w = torch.zeros((1 << 19) + 2, 4224, dtype=torch.bfloat16, device="cuda")
    w[-2:] = normal(81, 2, 4224).cuda()
    q, alone = mok.w4_quantize(w, form, group, zero), mok.w4_quantize(w[-2:], form, group, zero)
    for a, b in zip(q, alone):
        assert a is None and b is None or torch.equal(a[-2:], b)
    assert torch.equal(mok.w4_dequantize(*q)[-2:], mok.w4_dequantize(*alone))


@pytest.mark.parametrize("how", FORMATS)
@pytest.mark.parametrize("T,n", [(3, 4096), (3, 4099), (17, 4096), (17, 4112), (33, 4099), (20, 8208), (900, 300)])
def test_product_at_the_limits_of_its_tiles(how, T, n):
    """One, two and four times 16 weight rows per workgroup, K in whole chunks and not, more chunks than waves."""
    for k in (256,) if "128" in how else (192, 2304):
        w = normal(90, n, k, std=0.05)
        form, group, zero = FORMATS[how]
        q = mok.w4_quantize(w.cuda(), form, group, zero)  # (bit for bit the oracle's: tested above)
        x = normal(91, T, k).cuda()
        got = mok.w4_matmul(x, *q)
        for rows in (slice(0, 40), slice(n // 2 - 20, n // 2 + 20), slice(n - 40, n)):
            (c, s, z), v = w4(w[rows], how)
            assert torch.equal(q[0][rows], c)
            want = f64(x) @ v.T
            close(got[:, rows], want, 2.0 ** -8 * np.abs(want) + 8 * k ** 0.5 * 2.0 ** -24 * mags_of(f64(x), v, s, how))
