"""Tensors handed to a call that overlap what it writes: refused where other
workgroups would read what one has written, taken where a call may run in
place."""
import pytest

from mokutil import ROOT  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import mixture_experts_layer_build_amd as mok  # noqa: E402

BF = torch.bfloat16


def test_a_step_refuses_a_grad_scale_among_what_it_writes():
    p, g, m, v = (torch.ones(64, device="cuda") for _ in range(4))
    for written in (p, m, v):
        with pytest.raises(ValueError, match="overlaps"):
            mok.adamw_step([p], [g], [m], [v], step=1, lr=1e-3, grad_scale=written[5:6])
    assert (p == 1).all()
    mok.adamw_step([p], [g], [m], [v], step=1, lr=1e-3, grad_scale=g[5:6])  # only read
    assert (p != 1).all()


def test_a_norm_refuses_outputs_that_overlap_its_inputs():
    buf = torch.zeros(5 * 64, dtype=BF, device="cuda")
    x, w = buf[:256].view(4, 64), torch.ones(64, dtype=BF, device="cuda")
    r = torch.zeros(4, 64, dtype=BF, device="cuda")
    wide = torch.zeros(4, 128, dtype=BF, device="cuda")
    f = torch.zeros(4, 64, device="cuda")
    many = torch.ones(1024, dtype=BF, device="cuda")
    for args, kw in (((x, w), dict(y=buf[64:].view(4, 64))), ((wide[:, :64], w), dict(y=wide.view(-1)[:256].view(4, 64))),
                     ((f, w), dict(y=f.view(BF).view(-1)[:256].view(4, 64))), ((x, many[64:128]), dict(y=many[:256].view(4, 64))),
                     ((x, w, r), dict(y=r.view(-1).as_strided((4, 64), (64, 1), 0), rstd=r.view(torch.float32).view(-1)[:4])),
                     ((f, w), dict(rstd=f.view(-1)[8:12])), ((x, w), dict(rstd=buf.view(torch.float32)[:4]))):
        with pytest.raises(ValueError, match="overlaps"):
            mok.rms_norm_mxfp8(*args, **kw)
    rstd = torch.ones(4, device="cuda")
    for args, dx in (((x, r, rstd, w), buf[64:].view(4, 64)), ((r, x, rstd, w), buf[64:].view(4, 64)),
                     ((r, f, rstd, w), f.view(BF).view(-1)[256:].view(4, 64)),
                     ((r, r.clone(), rstd, many[:64]), many[:256].view(4, 64)),
                     ((r, r.clone(), rstd, w, x), buf[64:].view(4, 64))):
        with pytest.raises(ValueError, match="overlaps"):
            mok.rms_norm_backward(*args, dx=dx)


@pytest.mark.parametrize("rows,cols", [(300, 2048), (37, 512), (5, 8192)])
def test_a_norm_runs_in_place(rows, cols):
    torch.manual_seed(rows)
    x, r, dy = (torch.randn(rows, cols, device="cuda").to(BF) for _ in range(3))
    w = torch.randn(cols, device="cuda").to(BF)
    y = torch.empty_like(x)
    codes, scale, s = mok.rms_norm_mxfp8(x, w, r, y=y)
    for k in range(2):
        a, b = x.clone(), r.clone()
        got = mok.rms_norm_mxfp8(a, w, b, y=(a, b)[k])
        assert torch.equal((a, b)[k], y) and all(torch.equal(p, q) for p, q in zip(got, (codes, scale, s)))
    rstd = mok.rms_norm(x, w, r)[2]
    dx = torch.empty_like(x)
    ds, dw = mok.rms_norm_backward(dy, s, rstd, w, r, dx=dx)
    for k in range(3):
        t = [dy.clone(), s.clone(), r.clone()]
        got = mok.rms_norm_backward(t[0], t[1], rstd, w, t[2], dx=t[k])
        assert torch.equal(t[k], dx) and torch.equal(got[0], ds) and torch.equal(got[1], dw)


@pytest.mark.parametrize("cols", [333, 16400])
def test_a_backward_of_any_width_runs_in_place(cols):
    torch.manual_seed(cols)
    dy, s, d = (torch.randn(37, cols, device="cuda").to(BF) for _ in range(3))
    w, rstd = torch.randn(cols, device="cuda").to(BF), torch.rand(37, device="cuda")
    dx = torch.empty_like(s)
    ds, dw = mok.rms_norm_backward(dy, s, rstd, w, d, dx=dx)
    for k in range(3):
        t = [dy.clone(), s.clone(), d.clone()]
        got = mok.rms_norm_backward(t[0], t[1], rstd, w, t[2], dx=t[k])
        assert torch.equal(t[k], dx) and torch.equal(got[0], ds) and torch.equal(got[1], dw)


@pytest.mark.parametrize("shuffled", [False, True])
@pytest.mark.parametrize("bits", [32, 8])
def test_one_overlap_among_many_tensors_is_found(shuffled, bits):
    """40 tensors in one buffer per list, in their order or in none: no
    overlap, then one shifted into its neighbour, in each list in turn."""
    n, size = 40, 64
    order = torch.randperm(n, generator=torch.Generator().manual_seed(2)).tolist() if shuffled else range(n)
    buf = torch.zeros(4, n * size, device="cuda")
    codes = torch.zeros(2, n * size, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(2, n * 2, dtype=torch.uint8, device="cuda")

    def lists(which, at):
        cut = lambda b, l, w: [b[i * w - (1 if (l, i) == (which, at) else 0):][:w] for i in order]  # noqa: E731
        p, g = cut(buf[0], 0, size), cut(buf[1], 1, size)
        if bits == 32:
            return p, g, cut(buf[2], 2, size), cut(buf[3], 3, size)
        return (p, g, *(list(zip(cut(codes[k], 2 + k, size), cut(scales[k], 4 + k, 2))) for k in range(2)))

    mok.adamw_step(*lists(None, None), step=1, lr=1e-3)
    mok.adamw_step(*lists(1, 7), step=1, lr=1e-3)  # gradients are only read
    for which in (0, 2, 3) if bits == 32 else (0, 2, 3, 4, 5):
        for at in (1, 23, n - 1):
            with pytest.raises(ValueError, match="overlaps"):
                mok.adamw_step(*lists(which, at), step=1, lr=1e-3)
