"""What the Python calls of the experts' products refuse of tensors on the GPU,
before anything is enqueued."""
import pytest

from mokutil import ROOT  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import mixture_experts_layer_build_amd as mok  # noqa: E402


def bf(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16, device="cuda")


def test_grouped():
    x, w, off, dy = bf(6, 16), bf(2, 8, 16), torch.tensor([0, 2, 6], dtype=torch.int32).cuda(), bf(6, 8)
    f, b = mok.grouped_matmul, mok.grouped_matmul_backward
    for call in (lambda: f(x.float(), w, off), lambda: f(x, w.float(), off), lambda: f(x, w, off.float()),
                 lambda: f(x, w, off[:2]), lambda: f(x[:, :8], w, off), lambda: f(x.view(2, 3, 16), w, off),
                 lambda: f(x, w[0], off), lambda: f(x, w.transpose(1, 2), off), lambda: f(x.t(), w, off),
                 lambda: f(x.cpu(), w, off), lambda: f(x, w.cpu(), off), lambda: f(x, w, off.cpu()),
                 lambda: f(x, w, off, out=dy[:5]), lambda: f(x, w, off, out=dy.float()),
                 lambda: f(x, w, off, out=x[:, :8]), lambda: f(x, w, off, out=w.view(-1)[:48].view(6, 8)),
                 lambda: f(bf(1, 8).expand(6, 8), bf(2, 8, 8), off),
                 lambda: f(x, w[:0], off[:1]), lambda: f(x, w[:, :0], off),
                 lambda: b(dy, x[:5], w, off), lambda: b(x, x, w, off), lambda: b(dy, dy, w, off),
                 lambda: b(dy.float(), x, w, off), lambda: f(x, bf(1025, 8, 16), torch.zeros(1026).int().cuda())):
        with pytest.raises(ValueError):
            call()


def test_w4():
    w = bf(8, 256)
    c, s, z = mok.w4_quantize(w, "int4", 64, True)
    for call in (lambda: mok.w4_quantize(w, "mxfp4", 64), lambda: mok.w4_quantize(w, "mxfp4", zero_point=True),
                 lambda: mok.w4_quantize(w, "int4", 48), lambda: mok.w4_quantize(w[:, :96], "int4", 64),
                 lambda: mok.w4_quantize(w.half()), lambda: mok.w4_quantize(w.t()),
                 lambda: mok.w4_quantize(w.view(2, 4, 256)[:, :2]),
                 lambda: mok.w4_dequantize(c, s[:, :3], z), lambda: mok.w4_dequantize(c, s.float(), z),
                 lambda: mok.w4_dequantize(c, s, z[:4]), lambda: mok.w4_dequantize(c, s, z.int()),
                 lambda: mok.w4_dequantize(c, z, None), lambda: mok.w4_dequantize(c.t(), s.t()),
                 lambda: mok.w4_matmul(bf(2, 128), c, s, z), lambda: mok.w4_matmul(bf(2, 256).float(), c, s, z),
                 lambda: mok.w4_matmul(bf(2, 256), c.cpu(), s, z), lambda: mok.w4_matmul(bf(2, 256), c, s.cpu(), z),
                 lambda: mok.w4_matmul(bf(2, 256), c.view(2, 4, 128), s.view(2, 4, 4)),
                 lambda: mok.w4_matmul(bf(256, 2).t(), c, s, z)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(mok.MokError):  # rows that are no multiple of 16 bytes apart
        mok.w4_quantize(torch.zeros(4, 132, dtype=torch.bfloat16, device="cuda")[:, :128])


def test_layer():
    H, I, E, T = 256, 128, 4, 3

    def q(*shape, how=("int4", 64, False)):
        return mok.w4_quantize(bf(*shape), *how)[:2]

    ws = {}
    for n, shape in dict(routed_gate=(E, I, H), routed_up=(E, I, H), routed_down=(E, H, I)).items():
        ws[n], ws[n + "_scale"] = q(*shape)
    x, rw, ids = bf(T, H), torch.zeros(T, 2, device="cuda"), torch.zeros(T, 2, dtype=torch.int64, device="cuda")
    f = mok.forward_w4
    f(x, rw, ids, ws)
    sg, sgs = q(I, H)
    wrong, wrongs = q(E, I, H, how=("int4", 32, False))
    mx, mxs = q(E, I, H, how=("mxfp4", 32, False))
    z = torch.zeros(E, I, H // 64, dtype=torch.uint8, device="cuda")
    for call in (lambda: f(x.float(), rw, ids, ws), lambda: f(x, rw.bfloat16(), ids, ws), lambda: f(x, rw, ids.int(), ws),
                 lambda: f(x, rw[:2], ids, ws), lambda: f(x, rw, ids[:2], ws), lambda: f(x[:, :128], rw, ids, ws),
                 lambda: f(x, rw, ids[:, :0], ws), lambda: f(x, rw.cpu(), ids, ws),
                 lambda: f(x, rw, ids, {**ws, "routed_gate": None}), lambda: f(x, rw, ids, {}),
                 lambda: f(x, rw, ids, {**ws, "routed_up": wrong, "routed_up_scale": wrongs}),
                 lambda: f(x, rw, ids, {**ws, "routed_up": mx, "routed_up_scale": mxs}),
                 lambda: f(x, rw, ids, {**ws, "routed_up_zero": z}),
                 lambda: f(x, rw, ids, {**ws, "routed_up": ws["routed_up"][:3], "routed_up_scale": ws["routed_up_scale"][:3]}),
                 lambda: f(x, rw, ids, {**ws, "shared_gate": sg, "shared_gate_scale": sgs}),
                 lambda: f(x, rw, ids, {**ws, "shared_up": sg, "shared_up_scale": sgs}),
                 lambda: f(x, rw, ids, {**ws, "shared_up_scale": sgs}),
                 lambda: f(x, rw, ids, ws, out=x), lambda: f(x, rw, ids, ws, out=x.float()),
                 lambda: f(x.t().contiguous().t(), rw, ids, ws),
                 lambda: f(x, rw, ids, {**ws, "routed_gate": ws["routed_gate"].cpu()})):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: f(x, rw, ids, ws, swiglu_limit=-1.0), lambda: f(x, rw, ids, ws, swiglu_limit=float("nan")),
                 lambda: f(bf(8193, H), torch.zeros(8193, 1).cuda(), torch.zeros(8193, 1).long().cuda(), ws)):
        with pytest.raises(mok.MokError):
            call()
