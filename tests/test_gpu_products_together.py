"""The experts' products together with the operators around the layer, as a
program uses them: a routed expert function built on the grouped product and its
training step, the 4-bit layer after the router against its weights read back,
and the same on other streams and in captured graphs.

Tolerances bound the roundings on the way: to bf16 by 2^-8 of the value each, an
fp32 sum of n products by n 2^-24 of the sum of their magnitudes, and what a
value is off by goes on times the magnitudes of what it is multiplied with (silu:
times 1.1 at most)."""
import numpy as np
import pytest

from mokutil import ROOT  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import mixture_experts_layer_build_amd as mok  # noqa: E402
from mixture_experts_layer_build_amd import autograd as ag  # noqa: E402
from mixture_experts_layer_build_amd.optim import MoKAdamW  # noqa: E402

HALF, F32 = 2.0 ** -8, 2.0 ** -24


def normal(seed, *shape, std=1.0):
    gen = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=gen) * std).to(torch.bfloat16).cuda()


def f64(t):
    return t.detach().cpu().double().numpy()


def sorted_rows(ids, E):
    """The choices in the order of their experts: (choice, offsets)."""
    order = ids.reshape(-1).argsort(stable=True)
    count = torch.bincount(ids.reshape(-1), minlength=E)
    return order, torch.cat([count.new_zeros(1), count.cumsum(0)]).to(torch.int32)


def silu_mul(g, u):
    """The fp32 product, rounded once."""
    return (torch.nn.functional.silu(g.float()) * u.float()).to(torch.bfloat16)


def experts_of(x, rw, ids, W):
    """Routed experts by grouped products: out fp32 [T, H]."""
    T, k = ids.shape
    order, off = sorted_rows(ids, W["gate"].shape[0])
    xs = x[order // k]
    h = silu_mul(ag.grouped_matmul(xs, W["gate"], off), ag.grouped_matmul(xs, W["up"], off))
    y = ag.grouped_matmul(h, W["down"], off)
    rows = y.float() * rw.reshape(-1)[order, None]
    return torch.zeros(T, x.shape[1], device=x.device).index_add(0, order // k, rows)


def want_of(x, rw, ids, W, rounded):
    """(float64 output, its bound). `rounded`: steps of bf16 in g, u, h and y (0: none, but one in h)."""
    X, RW, ID = f64(x), f64(rw), ids.cpu().numpy()
    G, U, D = (f64(W[n]) for n in ("gate", "up", "down"))
    out, lim = np.zeros(X.shape), np.zeros(X.shape)
    H, I = X.shape[1], G.shape[1]
    for t in range(X.shape[0]):
        for j in range(ID.shape[1]):
            e, w = ID[t, j], RW[t, j]
            g, u = G[e] @ X[t], U[e] @ X[t]
            eg = HALF * rounded * np.abs(g) + 2 * H * F32 * (np.abs(G[e]) @ np.abs(X[t]))
            eu = HALF * rounded * np.abs(u) + 2 * H * F32 * (np.abs(U[e]) @ np.abs(X[t]))
            s = g / (1 + np.exp(-g))
            h = s * u
            eh = 1.1 * eg * (np.abs(u) + eu) + np.abs(s) * eu
            eh += (HALF + 2.0 ** -18) * (np.abs(h) + eh)
            y = D[e] @ h
            ey = np.abs(D[e]) @ eh + 2 * I * F32 * (np.abs(D[e]) @ (np.abs(h) + eh))
            ey += HALF * rounded * (np.abs(y) + ey)
            out[t] += w * y
            lim[t] += np.abs(w) * (ey + 8 * F32 * np.abs(y))
    return out, lim


def weights(seed, E, H, I):
    return {"gate": normal(seed, E, I, H, std=0.05), "up": normal(seed + 1, E, I, H, std=0.05),
            "down": normal(seed + 2, E, H, I, std=0.05)}


@pytest.mark.parametrize("T,H,I,E,k", [(1, 64, 96, 4, 2), (77, 128, 200, 8, 3), (300, 100, 75, 5, 2)])
def test_routed_experts_on_the_grouped_product(T, H, I, E, k):
    x, W = normal(1, T, H), weights(2, E, H, I)
    rw, ids = mok.router_topk(normal(5, T, E), k)
    out, lim = want_of(x, rw, ids, W, 1)
    got = f64(experts_of(x, rw, ids, W))
    assert (np.abs(got - out) <= lim).all()


def test_routed_experts_against_the_fused_layer():
    T, H, I, E, k = 200, 256, 128, 8, 3
    x, W = normal(11, T, H), weights(12, E, H, I)
    rw, ids = mok.router_topk(normal(15, T, E), k)
    cfg = mok.MoKConfig(H, I, E, k, T, capacity_multiplier=float(E))
    ws = mok.create_workspace(cfg)
    sched = mok.build_schedule(ws, ids)
    fused = mok.forward(ws, sched, x, rw, {f"routed_{n}": w for n, w in W.items()})
    fused = f64(fused[0] if isinstance(fused, tuple) else fused)
    _, lim = want_of(x, rw, ids, W, 1)
    here = f64(experts_of(x, rw, ids, W))
    # (both are within the bound of the exact output, the layer's rounded to bf16 once more)
    assert (np.abs(here - fused) <= 2 * lim + HALF * (np.abs(here) + 2 * lim)).all()


def test_training_step_of_routed_experts():
    """Gradients of a whole expert function against float64, each product's from what reached it; then an optimizer
    step that moves every parameter."""
    T, H, I, E, k = 60, 72, 40, 6, 2
    torch.manual_seed(0)
    lin = {n: ag.MoKGroupedLinear(E, *s, device="cuda") for n, s in
           dict(gate=(H, I), up=(H, I), down=(I, H)).items()}
    for i, m in enumerate(lin.values()):
        m.init_weights(0.1, torch.Generator().manual_seed(i))
    x = normal(21, T, H).requires_grad_()
    _, ids = mok.router_topk(normal(25, T, E), k)
    order, off = sorted_rows(ids, E)
    seen = {}

    def keep(name, t):
        t.retain_grad()
        seen[name] = t
        return t

    xs = keep("xs", x[order // k])
    g, u = keep("gate", lin["gate"](xs, off)), keep("up", lin["up"](xs, off))
    h = keep("h", silu_mul(g, u))
    y = keep("down", lin["down"](h, off))
    y.backward(normal(26, T * k, H))
    o = off.cpu().numpy()
    for name, src in (("gate", xs), ("up", xs), ("down", h)):
        dy, a = f64(seen[name].grad), f64(src)
        got = f64(lin[name].weight.grad)
        for e in range(E):
            r = slice(o[e], o[e + 1])
            want, mags = dy[r].T @ a[r], np.abs(dy[r]).T @ np.abs(a[r])
            assert (np.abs(got[e] - want) <= HALF * np.abs(want) + (o[e + 1] - o[e] + 1) * F32 * mags).all()
    W = {n: f64(m.weight) for n, m in lin.items()}
    of = np.repeat(np.arange(E), np.diff(o))
    dh = np.einsum("rn,rnk->rk", f64(y.grad), W["down"][of])
    mags = np.einsum("rn,rnk->rk", np.abs(f64(y.grad)), np.abs(W["down"][of]))
    assert (np.abs(f64(h.grad) - dh) <= HALF * np.abs(dh) + H * F32 * mags).all()
    # x: two gradients, each rounded, their sum rounded
    parts = [np.einsum("rn,rnk->rk", f64(t.grad), W[n][of]) for n, t in (("gate", g), ("up", u))]
    mags = sum(np.einsum("rn,rnk->rk", np.abs(f64(t.grad)), np.abs(W[n][of])) for n, t in (("gate", g), ("up", u)))
    size = sum(np.abs(p) for p in parts)
    assert (np.abs(f64(xs.grad) - sum(parts)) <= 2.01 * HALF * size + 1.01 * I * F32 * mags).all()
    opt = MoKAdamW([m.weight for m in lin.values()], lr=1e-2)
    before = [m.weight.detach().clone() for m in lin.values()]
    opt.step()
    assert all(not torch.equal(m.weight, b) for m, b in zip(lin.values(), before))


@pytest.mark.parametrize("T", [1, 4, 9, 40])
def test_serving_step_in_four_bits(T):
    """Norm, router and the 4-bit layer; the weights read back (MXFP4 values are exact in bf16) give the grouped
    products' output."""
    H, I, E, k = 256, 128, 8, 2
    res = normal(31, T, H)
    x = mok.rms_norm(res, normal(32, H))
    x = x[0] if isinstance(x, tuple) else x
    rw, ids = mok.router_topk(normal(33, T, E), k)
    W = weights(34, E, H, I)
    q = {n: mok.w4_quantize(w, format="mxfp4") for n, w in W.items()}
    back = {n: mok.w4_dequantize(*v) for n, v in q.items()}
    packed = {}
    for n, v in q.items():
        packed["routed_" + n], packed[f"routed_{n}_scale"] = v[0], v[1]
    got = f64(mok.forward_w4(x, rw, ids, packed))
    want, lim = want_of(x, rw, ids, back, 0)
    assert (np.abs(got - want) <= lim + HALF * (np.abs(want) + lim)).all()
    _, wide = want_of(x, rw, ids, back, 1)
    assert (np.abs(f64(experts_of(x, rw, ids, back)) - want) <= wide).all()
    # one expert's gate by itself, on the same weight
    y = f64(mok.w4_matmul(x, q["gate"][0][3], q["gate"][1][3]))
    exact = f64(x) @ f64(back["gate"][3]).T
    mags = np.abs(f64(x)) @ np.abs(f64(back["gate"][3])).T
    assert (np.abs(y - exact) <= HALF * np.abs(exact) + H * F32 * mags).all()


def test_on_another_stream_than_the_tensors():
    T, H, I, E, k = 33, 128, 64, 6, 2
    x, W = normal(41, T, H), weights(42, E, H, I)
    rw, ids = mok.router_topk(normal(45, T, E), k)
    q = {n: mok.w4_quantize(w, group=32, zero_point=True) for n, w in W.items()}
    packed = {}
    for n, v in q.items():
        packed["routed_" + n], packed[f"routed_{n}_scale"], packed[f"routed_{n}_zero"] = v
    want = experts_of(x, rw, ids, W), mok.forward_w4(x, rw, ids, packed), mok.w4_dequantize(*q["up"])
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        again = mok.w4_quantize(W["gate"], group=32, zero_point=True)
        got = experts_of(x, rw, ids, W), mok.forward_w4(x, rw, ids, packed), mok.w4_dequantize(*q["up"])
    s.synchronize()
    # (index_add sums a token's two rows in either order: a rounding of the fp32 sum at most)
    assert (got[0] - want[0]).abs().max() <= 4 * F32 * want[0].abs().max() * k
    assert torch.equal(got[1], want[1]) and torch.equal(got[2], want[2])
    assert all(torch.equal(a, b) for a, b in zip(again, q["gate"]))


def test_training_captured_and_replayed_with_eager_steps_between():
    """A step whose dW and y are cut into parts (few outputs, long sums), captured; eager steps of other leaves run
    between the replays."""
    R, n, k = 2200, 64, 1200
    off = torch.tensor([0, 1000, 1000, R], dtype=torch.int32, device="cuda")
    x, dy = normal(51, R, k).requires_grad_(), normal(52, R, n)
    lin = ag.MoKGroupedLinear(3, k, n, device="cuda")
    lin.init_weights(0.05)

    def step():
        x.grad = lin.weight.grad = None
        y = lin(x, off)
        y.backward(dy)
        return y

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for _ in range(2):
            step()
    torch.cuda.current_stream().wait_stream(s)
    x.grad = lin.weight.grad = None
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = lin(x, off)
        y.backward(dy)
    for seed in (61, 62, 63):
        with torch.no_grad():
            x.copy_(normal(seed, R, k)), dy.copy_(normal(seed + 9, R, n))
        graph.replay()
        torch.cuda.synchronize()
        want_y = mok.grouped_matmul(x.detach(), lin.weight.detach(), off)
        want = mok.grouped_matmul_backward(dy, x.detach(), lin.weight.detach(), off)
        assert torch.equal(y, want_y) and torch.equal(x.grad, want[0]) and torch.equal(lin.weight.grad, want[1])
