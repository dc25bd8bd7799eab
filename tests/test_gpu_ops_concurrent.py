"""The operators beside each other and far out: calls that overlap on two
streams, two captured graphs replayed in turn and together, and tensors of
more than 2^31 elements, whose last rows must equal a call on those rows
alone, bit for bit."""
import numpy as np
import pytest

from mokutil import ROOT  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import mixture_experts_layer_build_amd as mok  # noqa: E402

BF = torch.bfloat16


def step(x, r, w, l, dl):
    """One pass through the operators that need scratch memory."""
    y, s, rstd = mok.rms_norm(x, w, r)
    ds, dw = mok.rms_norm_backward(y, s, rstd, w, s)
    rw, ids, counts, losses = mok.router_topk(l, 8, losses=True)
    dlog = mok.router_topk_backward(rw, l, ids, counts=counts, d_losses=dl)
    return y, s, ds, dw, rw, ids, counts, losses, dlog


def inputs(seed, rows=4096):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    return n(rows, 2048).to(BF), n(rows, 2048).to(BF), n(2048).to(BF), n(rows * 4, 128), torch.ones(2, device="cuda")


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


def test_overlapping_calls_on_two_streams():
    a, b = inputs(1), inputs(2, 3000)
    want = [[t.clone() for t in step(*a)], [t.clone() for t in step(*b)]]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for k, (s, i) in enumerate(zip(streams, (a, b))):
            with torch.cuda.stream(s):
                got[k].append(step(*i))
    torch.cuda.synchronize()
    for k in range(2):
        assert all(same(g, want[k]) for g in got[k]), k


def test_two_graphs_replayed_in_turn_and_together():
    a, b = inputs(3), inputs(4, 2500)
    want = [[t.clone() for t in step(*a)], [t.clone() for t in step(*b)]]
    graphs, outs = [], []
    for i in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step(*i))
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for turn in range(3):
        for o in outs:
            for t in o:
                t.zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            if turn == 2:  # at the same time
                with torch.cuda.stream(s):
                    g.replay()
            else:
                g.replay()
        torch.cuda.synchronize()
        eager = step(*a)  # work of the program's own between the replays
        assert same(outs[0], want[0]) and same(outs[1], want[1]) and same(eager, want[0]), turn


def fill(t):
    """Random values into a large tensor, a part at a time."""
    flat = t.view(-1)
    for i in range(0, flat.numel(), 1 << 28):
        part = flat[i:i + (1 << 28)]
        part.copy_(torch.randn(part.numel(), device="cuda"))
    return t


def test_norm_past_32_bits():
    rows, cols = 131100, 16384
    assert rows * cols > 1 << 31
    x = fill(torch.empty(rows, cols, dtype=BF, device="cuda"))
    w = torch.randn(cols, device="cuda").to(BF)
    print("norm past 32 bits", flush=True)
    y, s, rstd = mok.rms_norm(x, w, x)
    tail = x[-5:].clone()
    y2, s2, rstd2 = mok.rms_norm(tail, w, tail)
    assert torch.equal(y[-5:], y2) and torch.equal(s[-5:], s2) and torch.equal(rstd[-5:], rstd2)
    del s
    ds, _ = mok.rms_norm_backward(y, x, rstd, w)
    ds2, _ = mok.rms_norm_backward(y2, tail, rstd2, w)
    assert torch.equal(ds[-5:], ds2)
    del ds
    codes, scale, _ = mok.rms_norm_mxfp8(x, w)
    codes2, scale2, _ = mok.rms_norm_mxfp8(tail, w)
    assert torch.equal(codes[-5:], codes2) and torch.equal(scale[-5:], scale2)


def test_router_past_32_bits():
    T, E = (1 << 21) + 77, 1024
    l = fill(torch.empty(T, E, dtype=BF, device="cuda"))
    print("router past 32 bits", flush=True)
    w, ids, counts, losses = mok.router_topk(l, 4, losses=True)
    tail = l[-9:].clone()
    w2, ids2 = mok.router_topk(tail, 4)
    assert torch.equal(w[-9:], w2) and torch.equal(ids[-9:], ids2)
    assert int(counts[E]) == T and int(counts[:E].sum()) == 4 * T and torch.isfinite(losses).all()
    assert torch.equal(counts[:E].long(), torch.bincount(ids.view(-1), minlength=E))
    d = mok.router_topk_backward(w, l, ids)
    assert torch.equal(d[-9:], mok.router_topk_backward(w2, tail, ids2))


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_past_32_bits(bits):
    n = (1 << 31) + 1000
    p, g = fill(torch.empty(n, dtype=BF, device="cuda")), fill(torch.empty(n, dtype=BF, device="cuda"))
    if bits == 32:
        m, v = torch.zeros(n, device="cuda"), torch.ones(n, device="cuda")
    else:
        m, v = [(torch.zeros(n, dtype=torch.uint8, device="cuda"),
                 torch.zeros((n + 31) // 32, dtype=torch.uint8, device="cuda")) for _ in range(2)]
    cut = n - 1000  # a multiple of 32
    tails = [t[cut:].clone() for t in (p, g)]
    tm, tv = (m[cut:].clone(), v[cut:].clone()) if bits == 32 else \
        [(t[0][cut:].clone(), t[1][cut // 32:].clone()) for t in (m, v)]
    print(f"adamw past 32 bits, {bits}", flush=True)
    mok.adamw_step([p], [g], [m], [v], step=2, lr=1e-2, seed=5)
    mok.adamw_step([tails[0]], [tails[1]], [tm], [tv], step=2, lr=1e-2, seed=5)
    assert torch.equal(p[cut:], tails[0])
    if bits == 32:
        assert torch.equal(m[cut:], tm) and torch.equal(v[cut:], tv)
    else:  # (v's roundings go by the element's number, which differs)
        assert torch.equal(m[0][cut:], tm[0]) and torch.equal(m[1][cut // 32:], tm[1])
        assert torch.equal(v[1][cut // 32:], tv[1]) and bool(v[0][cut:].any())
