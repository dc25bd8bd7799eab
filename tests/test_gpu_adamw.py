"""The multi-tensor AdamW step on the GPU against the float64 oracle: types,
sizes that end inside a block, misaligned tensors, more tensors than a launch
holds, both widths of the moments, the 8-bit states' rounding, the optimizer.

Tolerances. m and v are sums of two products of fp32 values: 4 roundings
each (5 with grad_scale), so 2^-21 of the sum of their magnitudes. p: the
update's quotient has the roundings of m, a root, a reciprocal (1 ulp each),
two products and a sum: 2^-20 of rate / den * (b1 |m| + c1 |g|); the decayed p
and the subtraction 2^-22 of |p|. A stored bf16 adds 2^-8 of its value."""
import numpy as np
import pytest

from mokutil import ROOT  # noqa: F401
from oracle import ops as oops

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import mixture_experts_layer_build_amd as mok  # noqa: E402
from mixture_experts_layer_build_amd.optim import MoKAdamW  # noqa: E402

BF, F32 = torch.bfloat16, torch.float32
LR, B1, B2, EPS, WD = 1e-2, 0.9, 0.95, 1e-8, 0.1


def f64(t):
    return t.detach().double().cpu().numpy()


def draw(rng, n, dtype, std, off=0):
    """n values in a buffer of their own, `off` elements into it."""
    t = torch.from_numpy((rng.standard_normal(n + off) * std).astype(np.float32)).to(dtype).cuda()
    return t[off:]


def near(got, ref, rel, absolute, what):
    got = f64(got) if isinstance(got, torch.Tensor) else got
    bad = ~(np.abs(got - ref) <= rel * np.abs(ref) + absolute + 1e-37)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size}, worst {np.abs(got - ref)[bad].max():.3g}"


def moments8(m, r, off=0):
    """States of fp32 m and r = sqrt(v), by the scale rule, nearest codes."""
    out = []
    for t in (m, r):
        x = oops.state_exponent(t)
        f = np.repeat(np.exp2(x), 32)[:t.size]
        codes = torch.from_numpy(t / f).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
        buf = torch.zeros(t.size + off, dtype=torch.uint8, device="cuda")
        buf[off:] = torch.from_numpy(codes).cuda()
        out.append((buf[off:], torch.from_numpy((x + 127).astype(np.uint8)).cuda()))
    return out


def check(sizes, pt, gt, bits, master=False, step=3, gscale=None, off=0, seed=11):
    rng = np.random.default_rng([len(sizes), sizes[0], bits])
    params = [draw(rng, n, pt, 0.5, off) for n in sizes]
    grads = [draw(rng, n, gt, 0.1, off) for n in sizes]
    masters = [draw(rng, n, F32, 0.5, off) for n in sizes] if master else None
    ms, vs = [], []
    for n in sizes:
        m = rng.standard_normal(n) * 0.05 * np.exp(rng.standard_normal(n))
        v = (rng.standard_normal(n) * 0.1) ** 2 * np.exp(rng.standard_normal(n) * 2)
        if n > 40:
            m[:32] = v[:32] = 0  # a block without a history
        if bits == 32:
            for lst, a in ((ms, m), (vs, v)):
                t = torch.zeros(n + off, device="cuda")
                t[off:] = torch.from_numpy(a.astype(np.float32)).cuda()
                lst.append(t[off:])
        else:
            a, b = moments8(m, np.sqrt(v), off)
            ms.append(a)
            vs.append(b)

    def values(pair, root):
        if bits == 32:
            return f64(pair)
        d = oops.decode8(pair[0].cpu().numpy(), pair[1].cpu().numpy())
        return d * d if root else d

    before = [(f64(masters[i] if master else params[i]), f64(grads[i]), values(ms[i], False), values(vs[i], True))
              for i in range(len(sizes))]
    gs = None if gscale is None else torch.tensor([gscale], device="cuda")
    print(f"adamw {len(sizes)} tensors of {sizes[:4]} {pt} {gt} {bits} master={master} off={off}", flush=True)
    mok.adamw_step(params, grads, ms, vs, masters, step=step, lr=LR, betas=(B1, B2), eps=EPS, weight_decay=WD,
                   grad_scale=gs, seed=seed)
    number = 0
    for i, n in enumerate(sizes):
        p, g, m, v = before[i]
        g = g * (1.0 if gscale is None else gscale)
        rp, rm, rv = oops.adamw(p, g, m, v, step, LR, B1, B2, EPS, WD)
        den = np.sqrt(rv / (1 - B2 ** step)) + EPS
        size_m = B1 * np.abs(m) + (1 - B1) * np.abs(g)
        tol = 2.0 ** -22 * np.abs(p) + 2.0 ** -20 * LR / (1 - B1 ** step) * size_m / den
        near(params[i], rp, 2.0 ** -8 if pt == BF else 0, tol, "p")
        if master:
            near(masters[i], rp, 0, tol, "master")
            assert torch.equal(params[i], masters[i].to(BF))
        if bits == 32:
            near(ms[i], rm, 0, 2.0 ** -21 * size_m, "m")
            near(vs[i], rv, 2.0 ** -21, 0, "v")
        else:
            check8(ms[i], vs[i], rm, rv, size_m, number, seed)
        number += (n + 31) // 32 * 32


def check8(mq, vq, m, v, size_m, number, seed):
    """8-bit states of values within 2^-20 of m (of size_m) and v."""
    n = m.size
    if n == 0:
        return
    slack = {0: size_m * 2.0 ** -20, 1: np.sqrt(v) * 2.0 ** -20}
    for which, (pair, val) in enumerate(((mq, m), (vq, np.sqrt(v)))):
        x = pair[1].cpu().numpy().astype(np.int64) - 127
        lo, hi = oops.state_exponent(np.maximum(np.abs(val) - slack[which], 0)), oops.state_exponent(np.abs(val) + slack[which])
        assert ((x >= lo) & (x <= hi)).all(), "scale"
        f = np.repeat(np.exp2(x.astype(np.float64)), 32)[:n]
        q = oops.decode8(pair[0].cpu().numpy(), pair[1].cpu().numpy()) / f
        u = val / f
        s = slack[which] / f
        if which == 0:
            assert (np.abs(q - np.clip(u, -448, 448)) <= np.maximum(np.abs(u) * 2.0 ** -4, 2.0 ** -10) + s).all(), "m"
            continue
        # the two codes around r
        step = np.exp2(np.floor(np.log2(np.maximum(u, 2.0 ** -6))) - 3)
        a = np.floor(u / step) * step
        b = a + step
        rnd = oops.uniforms(n, seed, number)
        want = np.where(rnd * (b * b - a * a) < u * u - a * a, b, a)
        want = np.minimum(want, 448)
        want = np.where((u > 0) & (want == 0), 2.0 ** -9, want)
        # elements whose choice, neighbours or block scale hang on the last fp32 bits may differ
        sure = (np.abs(rnd * (b * b - a * a) - (u * u - a * a)) > 1e-5 * b * b) & (u - a > 4 * s) & (b - u > 4 * s)
        assert sure.mean() > 0.9 or n < 64
        np.testing.assert_array_equal(q[sure], want[sure])
        assert (((q >= a - step) & (q <= b + step)) | (q == 2.0 ** -9)).all()
        assert (q[u > 1e-30] > 0).all()


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("pt,master", [(F32, False), (BF, False), (BF, True)])
@pytest.mark.parametrize("gt", [F32, BF])
def test_types(pt, master, gt, bits):
    check([4096, 1, 31, 32, 33, 2049, 70001], pt, gt, bits, master, gscale=0.25)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("off", [1, 3, 8])
def test_misaligned_tensors(bits, off):
    check([100, 5000, 7], BF, BF, bits, True, off=off)
    check([100, 5000, 7], F32, F32, bits, False, off=off)


@pytest.mark.parametrize("bits", [32, 8])
def test_many_tensors_and_empty_ones(bits):
    check([(i * 37) % 300 for i in range(1, 130)] + [0, 40, 0], BF, F32, bits, True)


@pytest.mark.parametrize("bits", [32, 8])
def test_large_tensors_take_the_long_chunks(bits):
    check([20_000_003, 64, 1_000_001], BF, BF, bits, False, step=100)


@pytest.mark.parametrize("bits", [32, 8])
def test_first_step_from_zero_states(bits):
    g = torch.randn(1000, device="cuda")
    p = torch.zeros(1000, device="cuda")
    z = [torch.zeros(1000, device="cuda") for _ in range(2)] if bits == 32 else \
        [(torch.zeros(1000, dtype=torch.uint8, device="cuda"), torch.zeros(32, dtype=torch.uint8, device="cuda")) for _ in range(2)]
    mok.adamw_step([p], [g], [z[0]], [z[1]], step=1, lr=0.5, betas=(B1, B2))
    # the first update is lr * sign(g) up to eps: 2^-20 by the tolerance above
    assert ((p + 0.5 * g.sign()).abs() <= 0.5 * 2.0 ** -20 + 0.5 * 1e-8 / g.abs()).all()


def test_rows_behind_a_tensor_stay():
    flat = {n: torch.full((200,), 3.0, device="cuda") for n in "pgmv"}
    codes = {n: torch.full((200,), 77, dtype=torch.uint8, device="cuda") for n in "mv"}
    scales = {n: torch.full((9,), 127, dtype=torch.uint8, device="cuda") for n in "mv"}
    mok.adamw_step([flat["p"][:101]], [flat["g"][:101]], [flat["m"][:101]], [flat["v"][:101]], step=1, lr=0.1)
    assert all((flat[n][101:] == 3).all() for n in "pmv")
    mok.adamw_step([flat["p"][:101]], [flat["g"][:101]], [(codes["m"][:101], scales["m"][:4])],
                   [(codes["v"][:101], scales["v"][:4])], step=1, lr=0.1)
    assert (flat["p"][101:] == 3).all()
    assert all((codes[n][101:] == 77).all() and (scales[n][4:] == 127).all() for n in "mv")


def test_eight_bit_second_moment_decays_and_keeps_its_mean():
    """Without a gradient v decays by b2 a step on average, where the nearest
    code would never move. The stored v is a martingale around it: a step's
    relative variance is at most (1/4)^2 / 4 (codes of the root are 1/8
    apart), so after 40 steps the mean of 2^18 elements is within 5 *
    sqrt(40 / 64) / 512 < 0.8 % of b2^40 (and 2^-9 of fp32 rounding)."""
    n = 1 << 18
    r = np.full(n, 0.01)
    (_, _), v = moments8(np.zeros(n), r)
    m = (torch.zeros(n, dtype=torch.uint8, device="cuda"), torch.zeros(n // 32, dtype=torch.uint8, device="cuda"))
    p, g = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
    start = (oops.decode8(v[0].cpu().numpy(), v[1].cpu().numpy()) ** 2).mean()
    for step in range(1, 41):
        mok.adamw_step([p], [g], [m], [v], step=step, lr=1e-3, betas=(B1, B2))
    mean = (oops.decode8(v[0].cpu().numpy(), v[1].cpu().numpy()) ** 2).mean()
    assert abs(mean / (start * B2 ** 40) - 1) < 0.01
    assert not p.any()


def test_a_gradient_that_is_not_finite_is_seen():
    n = 96
    p, g = torch.zeros(n, device="cuda"), torch.ones(n, device="cuda")
    g[40] = float("nan")
    g[70] = float("inf")
    z = [(torch.zeros(n, dtype=torch.uint8, device="cuda"), torch.zeros(3, dtype=torch.uint8, device="cuda")) for _ in range(2)]
    mok.adamw_step([p], [g], [z[0]], [z[1]], step=1, lr=0.1)
    assert torch.isnan(p[40]) and torch.isfinite(p[:32]).all()
    assert z[0][1].tolist()[1:] == [255, 255] and z[1][1].tolist()[1:] == [255, 255]
    mok.adamw_step([p], [torch.ones(n, device="cuda")], [z[0]], [z[1]], step=2, lr=0.1)
    assert torch.isnan(p[32:]).all() and torch.isfinite(p[:32]).all()


def test_the_same_seed_gives_the_same_bits():
    rng = np.random.default_rng(1)
    n = 100_003
    g, m0, r0 = draw(rng, n, F32, 0.1), rng.standard_normal(n) * 0.05, np.abs(rng.standard_normal(n)) * 0.1
    got = []
    for seed in (5, 5, 6):
        m, v = moments8(m0, r0)
        p = torch.ones(n, device="cuda")
        mok.adamw_step([p], [g], [m], [v], step=4, lr=LR, seed=seed)
        got.append((p, *m, *v))
    assert all(torch.equal(a, b) for a, b in zip(got[0], got[1]))
    assert torch.equal(got[0][0], got[2][0]) and not torch.equal(got[0][3], got[2][3])


def test_python_refusals():
    p, g = torch.zeros(64, device="cuda"), torch.zeros(64, device="cuda")
    m, v = torch.zeros(64, device="cuda"), torch.zeros(64, device="cuda")
    ok = dict(step=1, lr=1e-3)
    for args, match in ((([p], [g, g], [m], [v]), "tensors"), (([p], [g[:32]], [m], [v]), "sizes"),
                        (([p], [g.double()], [m], [v]), "float"), (([p], [g], [m.bfloat16()], [v]), "float32"),
                        (([p], [g], [m], [m]), "twice"), (([p, p], [g, g], [m, m.clone()], [v, v.clone()]), "twice"),
                        (([p, p.bfloat16()], [g, g], [m, m.clone()], [v, v.clone()]), "all be"),
                        (([p], [g.cpu()], [m], [v]), "every tensor"), (([p], [g], [m], [v], [p.clone()]), "masters"),
                        (([p], [g.view(8, 8).t()], [m], [v]), "contiguous"),
                        (([p], [g], [(m,)], [(v,)]), "pairs")):
        with pytest.raises(ValueError, match=match):
            mok.adamw_step(*args, **ok)
    q = (torch.zeros(64, dtype=torch.uint8, device="cuda"), torch.zeros(1, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError, match="sizes"):
        mok.adamw_step([p], [g], [q], [(q[0].clone(), q[1])], **ok)
    with pytest.raises(ValueError, match="one element"):
        mok.adamw_step([p], [g], [m], [v], grad_scale=torch.ones(2, device="cuda"), **ok)
    with pytest.raises(mok.MokError):
        mok.adamw_step([p], [g], [m], [v], step=0, lr=1e-3)
    mok.adamw_step([], [], [], [], **ok)


@pytest.mark.parametrize("bits", [32, 8])
def test_optimizer(bits):
    torch.manual_seed(0)
    shapes = [(33, 17), (64,), (5, 7, 9), (128, 128)]
    params = [torch.nn.Parameter(torch.randn(s, device="cuda").to(BF if i % 2 else F32)) for i, s in enumerate(shapes)]
    opt = MoKAdamW([{"params": params[:2]}, {"params": params[2:], "lr": 3e-3, "weight_decay": 0.0}], lr=LR,
                   betas=(B1, B2), weight_decay=WD, state_bits=bits)
    ref = [(f64(p).ravel(), np.zeros(p.numel()), np.zeros(p.numel())) for p in params]
    for step in range(1, 4):
        for p in params:
            p.grad = torch.randn_like(p)
        if bits == 8:  # each step alone: the oracle starts from the stored states
            for i, p in enumerate(params):
                st = opt.state.get(p)
                if st:
                    dec = [oops.decode8(st[n].cpu().numpy(), st[n + "_scale"].cpu().numpy()) for n in ("exp_avg", "exp_avg_sq")]
                    ref[i] = (ref[i][0], dec[0], dec[1] ** 2)
        for i, p in enumerate(params):
            lr, wd = (LR, WD) if i < 2 else (3e-3, 0.0)
            ref[i] = oops.adamw(ref[i][0], f64(p.grad).ravel() * 0.5, ref[i][1], ref[i][2], step, lr, B1, B2, 1e-8, wd)
        opt.step(grad_scale=torch.tensor([0.5], device="cuda"))
    for i, p in enumerate(params):
        got = opt.state[p].get("master", p)
        assert ("master" in opt.state[p]) == (p.dtype == BF)
        # three steps of the tolerance above; an update is at most about 3 lr where |m| <= 3 sqrt(v)
        near(f64(got).ravel(), ref[i][0], 3 * 2.0 ** -22, 3 * 2.0 ** -20 * 4 * LR, f"param {i}")
        if p.dtype == BF:
            assert torch.equal(p.detach(), got.to(BF))
    # a saved and loaded optimizer goes on with the same bits
    copies = [torch.nn.Parameter(p.detach().clone()) for p in params]
    other = MoKAdamW([{"params": copies[:2]}, {"params": copies[2:]}], state_bits=bits)
    other.load_state_dict(opt.state_dict())
    for p, q in zip(params, copies):
        p.grad = torch.randn_like(p)
        q.grad = p.grad.clone()
    opt.step()
    other.step()
    assert all(torch.equal(p, q) for p, q in zip(params, copies))


def test_optimizer_refuses_capture():
    p = torch.nn.Parameter(torch.zeros(64, device="cuda"))
    p.grad = torch.ones(64, device="cuda")
    opt = MoKAdamW([p])
    opt.step()
    graph = torch.cuda.CUDAGraph()
    with pytest.raises(RuntimeError, match="captured"):
        with torch.cuda.graph(graph):
            opt.step()
    torch.cuda.synchronize()
    opt.step()


def test_a_refused_step_is_not_counted():
    p = torch.nn.Parameter(torch.ones(64, device="cuda"))
    p.grad = torch.ones(64, device="cuda")
    opt = MoKAdamW([p])
    with pytest.raises(ValueError):
        opt.step(grad_scale=torch.ones(2, device="cuda"))
    assert opt.state[p]["step"] == 0 and torch.equal(p.detach(), torch.ones(64, device="cuda"))
    opt.step()
    assert opt.state[p]["step"] == 1


def test_overlapping_tensors_are_refused():
    buf = torch.zeros(400, device="cuda")
    p, g, m, v = (torch.zeros(64, device="cuda") for _ in range(4))
    for args in (([buf[:64]], [g], [buf[32:96]], [v]), ([p], [buf[:64]], [m], [buf[63:127]]),
                 ([buf[:64], buf[16:80]], [g, g], [m, buf[100:164]], [v, buf[200:264]]),
                 ([buf[:300], buf[8:72]], [torch.zeros(300, device="cuda"), g], [torch.zeros(300, device="cuda"), m],
                  [torch.zeros(300, device="cuda"), v])):
        with pytest.raises(ValueError, match="overlaps"):
            mok.adamw_step(*args, step=1, lr=1e-3)
    # neighbours in one buffer, and one gradient for two tensors, are no overlap
    mok.adamw_step([buf[:64], buf[64:128]], [g, g], [buf[128:192], m], [buf[192:256], v], step=1, lr=1e-3)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("eps", [0.0, 1e-30])
def test_second_moments_below_the_normal_range(bits, eps):
    """Gradients of 1e-19: v is subnormal, its root is not. The first update
    is -lr * sign(g); g^2 and v are rounded to multiples of 2^-149, by at most
    2^-150 / 1e-38 and 2^-150 / 5e-40 (1.5e-6 together, half of it in the
    root), and four roundings of 2^-23 follow: below 2^-19."""
    g = (torch.rand(4000, device="cuda") * 2e-19 + 1e-19) * torch.randn(4000, device="cuda").sign()
    p = torch.zeros(4000, device="cuda")
    st = [torch.zeros(4000, device="cuda") for _ in range(2)] if bits == 32 else \
        [(torch.zeros(4000, dtype=torch.uint8, device="cuda"), torch.zeros(125, dtype=torch.uint8, device="cuda"))
         for _ in range(2)]
    mok.adamw_step([p], [g], [st[0]], [st[1]], step=1, lr=0.5, betas=(B1, B2), eps=eps)
    assert ((p + 0.5 * g.sign()).abs() <= 0.5 * 2.0 ** -19).all()
