"""RMS norm on the GPU against the float64 oracle: widths of each kernel
variant and between them, odd and misaligned ones, row counts around the
workgroups' rows, types, strides, in-place sums, MXFP8 output, backward.

Tolerances. A stored bf16 is off by at most 2^-8 of its value (half a step).
fp32 work: rstd comes from a sum whose longest chain is 64 terms of a thread
plus 10 of the tree, so it is within 74 * 2^-24 / 2 of its value; with the
three products and the addition behind it, y is within 48 * 2^-24 < 2^-18."""
import numpy as np
import pytest

from mokutil import ROOT  # noqa: F401
from oracle import ops as oops

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import mixture_experts_layer_build_amd as mok  # noqa: E402
from mixture_experts_layer_build_amd.autograd import MoKRMSNorm, rms_norm  # noqa: E402

BF, F32 = torch.bfloat16, torch.float32
H8 = 2.0 ** -8


def draw(rng, shape, dtype, std=1.0):
    return torch.from_numpy((rng.standard_normal(shape) * std).astype(np.float32)).to(dtype).cuda()


def f64(t):
    return t.detach().double().cpu().numpy()


def near(got, ref, rel, absolute=0.0, what=""):
    got = f64(got) if isinstance(got, torch.Tensor) else got
    assert got.shape == ref.shape, what
    bad = ~(np.abs(got - ref) <= rel * np.abs(ref) + absolute + 1e-37)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size}, worst {np.abs(got - ref)[bad].max():.3g}"


def rel_of(dtype):
    return (H8 if dtype == BF else 0.0) + 2.0 ** -18


def check_mxfp8(codes, scale, y):
    """Codes and scales of fp32 values within 2^-18 of y."""
    y = y.reshape(-1, 32)
    amax = np.abs(y).max(1)
    x = scale.cpu().numpy().reshape(-1).astype(np.int64) - 127
    with np.errstate(divide="ignore"):
        lo = np.floor(np.log2(amax * (1 - 2.0 ** -18))) - 8
        hi = np.floor(np.log2(amax * (1 + 2.0 ** -18))) - 8
    lo, hi = np.where(amax > 0, np.clip(lo, -127, 127), -127), np.where(amax > 0, np.clip(hi, -127, 127), -127)
    assert ((x >= lo) & (x <= hi)).all()
    got = oops.decode8(codes.cpu().numpy().reshape(-1), scale.cpu().numpy().reshape(-1)).reshape(-1, 32)
    f = np.exp2(x)[:, None].astype(np.float64)
    u = np.clip(y / f, -448, 448)
    # half a step: 2^-4 of a normal code's value, 2^-10 below 2^-6
    tol = np.maximum(np.abs(u) * 2.0 ** -4, 2.0 ** -10) + np.abs(y / f) * 2.0 ** -17
    assert (np.abs(got / f - u) <= tol).all()


@pytest.mark.parametrize("cols", [8, 32, 504, 512, 520, 1024, 1544, 2048, 2056, 4096, 4104, 7168, 8192, 8200, 16384, 16392,
                                  1, 7, 129, 1001, 5003])
@pytest.mark.parametrize("rows", [1, 5])
def test_forward_widths(rows, cols):
    rng = np.random.default_rng([rows, cols])
    x, r, w = draw(rng, (rows, cols), BF), draw(rng, (rows, cols), BF, 2.0), draw(rng, cols, BF)
    print(f"forward {rows} x {cols}", flush=True)
    y, s, rstd = mok.rms_norm(x, w, r)
    ry, rs, rr = oops.rms_norm(f64(x), f64(w), f64(r))
    near(s, rs, H8 + 2.0 ** -24, what="sum")
    near(y, ry, rel_of(BF), what="y")
    near(rstd, rr, 2.0 ** -18, what="rstd")


@pytest.mark.parametrize("xt,rt,wt", [(BF, None, BF), (F32, None, F32), (BF, F32, BF), (F32, F32, F32), (BF, BF, F32),
                                      (F32, None, BF)])
@pytest.mark.parametrize("cols", [256, 2048, 7168, 333])
def test_forward_types(xt, rt, wt, cols):
    rng = np.random.default_rng(cols)
    rows = 1031
    x, w = draw(rng, (rows, cols), xt), draw(rng, cols, wt)
    r = None if rt is None else draw(rng, (rows, cols), rt)
    y, s, rstd = mok.rms_norm(x, w, r, eps=1e-5)
    ry, rs, rr = oops.rms_norm(f64(x), f64(w), None if r is None else f64(r), 1e-5)
    assert y.dtype == BF and (s is None) == (rt is None)
    if s is not None:
        assert s.dtype == rt
        near(s, rs, (H8 if rt == BF else 0) + 2.0 ** -23, what="sum")
    near(y, ry, rel_of(BF), what="y")
    near(rstd, rr, 2.0 ** -18, what="rstd")


@pytest.mark.parametrize("rows,cols", [(1, 32), (3, 2048), (777, 4096), (130, 7168), (5, 16384), (9, 96)])
@pytest.mark.parametrize("rt", [None, BF, F32])
def test_mxfp8_output(rows, cols, rt):
    rng = np.random.default_rng([rows, cols])
    x, w = draw(rng, (rows, cols), BF), draw(rng, cols, BF)
    r = None if rt is None else draw(rng, (rows, cols), rt)
    y, rstd = torch.empty_like(x), torch.empty(rows, device="cuda")
    codes, scale, s = mok.rms_norm_mxfp8(x, w, r, y=y, rstd=rstd)
    ry, rs, rr = oops.rms_norm(f64(x), f64(w), None if r is None else f64(r))
    check_mxfp8(codes, scale, ry)
    near(y, ry, rel_of(BF), what="y")
    near(rstd, rr, 2.0 ** -18, what="rstd")
    alone = mok.rms_norm_mxfp8(x, w, r)
    assert torch.equal(alone[0], codes) and torch.equal(alone[1], scale)


def test_mxfp8_zero_rows_and_blocks_that_are_not_finite():
    x = torch.ones(4, 64, dtype=BF, device="cuda")
    w = torch.ones(64, dtype=BF, device="cuda")
    x[1] = 0
    x[2, 40] = float("nan")
    w[3] = float("inf")
    codes, scale, _ = mok.rms_norm_mxfp8(x, w)
    sc = scale.cpu().numpy()
    assert sc[0, 0] == 255 and sc[0, 1] != 255  # the infinite weight's block, and its neighbour
    assert sc[1, 1] == 0 and not codes[1, 32:].any()  # zeros
    assert (sc[2] == 255).all()  # a NaN reaches its whole row


def test_strided_rows_in_place_sum_and_untouched_neighbours():
    rng = np.random.default_rng(5)
    for cols, ld in ((128, 200), (128, 129), (2048, 2304), (33, 40)):
        wide = draw(rng, (6, ld), BF)
        x, w = wide[:, :cols], draw(rng, cols, BF)
        resw = draw(rng, (6, ld), F32)
        r = resw[:, :cols]
        y, s, _ = mok.rms_norm(x, w, r)
        ry, rs, _ = oops.rms_norm(f64(x), f64(w), f64(r))
        near(y, ry, rel_of(BF), what="y")
        near(s, rs, 2.0 ** -23, what="sum")
    # sum into the residual's own buffer, y into x's, through the C ABI
    for cols in (256, 77):
        x, r, w = draw(rng, (9, cols), BF), draw(rng, (9, cols), BF), draw(rng, cols, BF)
        ry, rs, _ = oops.rms_norm(f64(x), f64(w), f64(r))
        guard = r.clone()
        st = mok.lib().mok_rms_norm(x.data_ptr(), 0, cols, r.data_ptr(), 0, cols, w.data_ptr(), 0, 8, cols, 1e-6,
                                    r.data_ptr(), x.data_ptr(), None, None, None,
                                    torch.cuda.current_stream().cuda_stream)
        assert st == 0
        near(r[:8], rs[:8], H8 + 2.0 ** -24, what="sum in place")
        near(x[:8], ry[:8], rel_of(BF), what="y in place")
        assert torch.equal(r[8], guard[8])  # the row behind the last one


def test_empty_batch_and_leading_dimensions():
    w = torch.ones(64, dtype=BF, device="cuda")
    x = torch.zeros(0, 64, dtype=BF, device="cuda")
    y, s, rstd = mok.rms_norm(x, w, x)
    assert y.shape == (0, 64) and s.shape == (0, 64) and rstd.shape == (0,)
    ds, dw = mok.rms_norm_backward(y, s, rstd, w)
    assert ds.shape == (0, 64) and not dw.any()
    rng = np.random.default_rng(6)
    x = draw(rng, (2, 3, 64), BF)
    y, _, rstd = mok.rms_norm(x, w)
    assert y.shape == x.shape and rstd.shape == (2, 3)
    assert torch.equal(y.view(6, 64), mok.rms_norm(x.view(6, 64), w)[0])


def bounds(dy, s, rstd, w, dsum):
    """|ds| and |dw| errors of the fp32 work. along is a sum of at most 74
    chained terms, so off by 74 * 2^-24 < 2^-17 of its terms' magnitudes; dw
    chains at most rows / workgroup (here below 128) + 80 terms: 2^-16."""
    xh = np.abs(s * rstd[..., None])
    g = np.abs(dy * w)
    b = rstd[..., None] * (g + xh * np.mean(g * xh, axis=-1, keepdims=True))
    if dsum is not None:
        b = b + np.abs(dsum)
    return b * 2.0 ** -17, (np.abs(dy) * xh).sum(0) * 2.0 ** -16


@pytest.mark.parametrize("cols", [8, 512, 520, 1024, 2048, 2056, 4096, 7168, 8200, 16384, 16392, 1, 333])
@pytest.mark.parametrize("rows,st,wt,with_dsum", [(1, BF, BF, False), (7, F32, F32, True), (1037, BF, F32, True)])
def test_backward(rows, cols, st, wt, with_dsum):
    rng = np.random.default_rng([rows, cols])
    dy, s, w = draw(rng, (rows, cols), BF), draw(rng, (rows, cols), st, 1.5), draw(rng, cols, wt)
    dsum = draw(rng, (rows, cols), st) if with_dsum else None
    rstd = torch.from_numpy(oops.rms_norm(f64(s), f64(w))[2].astype(np.float32)).cuda()
    dx = torch.empty(rows, cols, dtype=BF, device="cuda") if st == F32 else None
    print(f"backward {rows} x {cols} {st}", flush=True)
    ds, dw = mok.rms_norm_backward(dy, s, rstd, w, dsum, dx=dx)
    args = f64(dy), f64(s), f64(rstd), f64(w), None if dsum is None else f64(dsum)
    rds, rdw = oops.rms_norm_backward(*args)
    bds, bdw = bounds(*args)
    near(ds, rds, H8 if st == BF else 0, bds, "ds")
    near(dw, rdw, H8 if wt == BF else 0, bdw, "dw")
    if dx is not None:
        near(dx, rds, H8, bds, "dx")
    again = mok.rms_norm_backward(dy, s, rstd, w, dsum)
    assert torch.equal(ds, again[0]) and torch.equal(dw, again[1])  # the same bits


def test_backward_strided():
    rng = np.random.default_rng(8)
    dy, s, dsum = (draw(rng, (13, 300), BF)[:, :256] for _ in range(3))
    w = draw(rng, 256, BF)
    rstd = torch.from_numpy(oops.rms_norm(f64(s), f64(w))[2].astype(np.float32)).cuda()
    ds, dw = mok.rms_norm_backward(dy, s, rstd, w, dsum)
    want = mok.rms_norm_backward(dy.contiguous(), s.contiguous(), rstd, w, dsum.contiguous())
    # 300 elements a row is not a multiple of 8: the other kernel, within both bounds
    args = f64(dy), f64(s), f64(rstd), f64(w), f64(dsum)
    bds, bdw = bounds(*args)
    rds, rdw = oops.rms_norm_backward(*args)
    for got in ((ds, dw), want):
        near(got[0], rds, H8, bds, "ds")
        near(got[1], rdw, H8, bdw, "dw")


@pytest.mark.parametrize("xt,rt", [(BF, None), (BF, BF), (BF, F32), (F32, F32)])
def test_autograd(xt, rt):
    rng = np.random.default_rng(9)
    rows, cols = 37, 256
    x, w = draw(rng, (rows, cols), xt).requires_grad_(), draw(rng, cols, BF).requires_grad_()
    r = None if rt is None else draw(rng, (rows, cols), rt).requires_grad_()
    dy = draw(rng, (rows, cols), BF)
    d_sum = None if rt is None else draw(rng, (rows, cols), rt)
    y, s = rms_norm(x, w, r)
    loss = (y.float() * dy.float()).sum()
    if s is not None:
        loss = loss + (s.float() * d_sum.float()).sum()
    loss.backward()
    saved = x if s is None else s
    _, _, rstd = oops.rms_norm(f64(x), f64(w), None if r is None else f64(r))
    # the backward starts from the stored sum: the oracle from the same values
    args = f64(dy), f64(saved), rstd.astype(np.float32).astype(np.float64), f64(w), \
        None if d_sum is None else f64(d_sum)
    rds, rdw = oops.rms_norm_backward(*args)
    bds, bdw = bounds(*args)
    bds = bds * 2  # the saved rstd is the GPU's, within 2^-18 of the oracle's
    near(x.grad, rds, H8 if xt == BF else 0, bds, "x")
    near(w.grad, rdw, H8, bdw * 2, "w")
    if r is not None:
        near(r.grad, rds, H8 if rt == BF else 0, bds, "residual")
        assert x.grad.data_ptr() != r.grad.data_ptr()


def test_autograd_partial_gradients():
    rng = np.random.default_rng(10)
    x, r = draw(rng, (5, 64), BF).requires_grad_(), draw(rng, (5, 64), F32).requires_grad_()
    norm = MoKRMSNorm(64, device="cuda")
    y, s = norm(x, r)
    s.sum().backward()  # only the sum: an expanded gradient of ones
    assert torch.equal(x.grad, torch.ones_like(x)) and torch.equal(r.grad, torch.ones_like(r))
    assert not norm.weight.grad.any()
    x.grad = r.grad = None
    with torch.no_grad():
        assert not norm(x, r)[0].requires_grad
    norm.weight.requires_grad_(False)
    y, s = norm(x, r.detach())
    y.float().sum().backward()
    assert x.grad is not None and r.grad is None


def test_python_refusals():
    x, w = torch.zeros(4, 64, dtype=BF, device="cuda"), torch.ones(64, dtype=BF, device="cuda")
    with pytest.raises(ValueError, match="bfloat16"):
        mok.rms_norm(x.half(), w)
    with pytest.raises(ValueError, match="shape"):
        mok.rms_norm(x, w[:32])
    with pytest.raises(ValueError, match="shape"):
        mok.rms_norm(x, w, x[:2])
    with pytest.raises(ValueError, match="dense rows"):
        mok.rms_norm(x.t(), torch.ones(4, dtype=BF, device="cuda"))
    with pytest.raises(ValueError, match="dense rows"):
        mok.rms_norm(x[:1].expand(4, 64), w)
    with pytest.raises(ValueError, match="multiple of 32"):
        mok.rms_norm_mxfp8(x[:, :48], w[:48])
    with pytest.raises(ValueError, match="is on"):
        mok.rms_norm(x, w.cpu())
    with pytest.raises(mok.MokError):
        mok.rms_norm(x, w, eps=-1.0)
    with pytest.raises(mok.MokError):
        mok.rms_norm(x.float(), w, x)
    with pytest.raises(mok.MokError):  # a row stride that 16-byte loads do not allow
        mok.rms_norm_mxfp8(torch.zeros(4, 68, dtype=BF, device="cuda")[:, :64], w)


def test_another_stream_and_a_replayed_graph():
    rng = np.random.default_rng(11)
    x, r, w = draw(rng, (300, 2048), BF), draw(rng, (300, 2048), BF), draw(rng, 2048, BF)
    dy = draw(rng, (300, 2048), BF)

    def step():
        y, s, rstd = mok.rms_norm(x, w, r)
        return y, s, *mok.rms_norm_backward(dy, s, rstd, w, s)

    want = [t.clone() for t in step()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(3):
        x.copy_(draw(rng, (300, 2048), BF))
        graph.replay()
        torch.cuda.synchronize()
        eager = step()
        assert all(torch.equal(a, b) for a, b in zip(out, eager)), i
