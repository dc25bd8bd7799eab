"""Refusals of the experts' products outside the layer, on the CPU: every case
fails the host-side checks of the C ABI (pointers are never followed) or of the
Python binding before any device work."""
import ctypes as C

import pytest

from mokutil import ROOT  # noqa: F401

torch = pytest.importorskip("torch")
import mixture_experts_layer_build_amd as mok  # noqa: E402
from mixture_experts_layer_build_amd import _lib  # noqa: E402

INVALID, UNSUPPORTED, SMALL, OK = (_lib.MOK_ERR_INVALID_ARGUMENT, _lib.MOK_ERR_UNSUPPORTED,
                                   _lib.MOK_ERR_BUFFER_TOO_SMALL, _lib.MOK_OK)
P = 1 << 20  # an address that is never followed


def grouped(which="", a=P, lda=64, b=P, ldb=64, off=P, o64=0, rows=4, E=2, n=64, k=64, out=P, ldo=64, rest=1, f32=0,
            scratch=None, nbytes=0):
    lib = _lib.load()
    if which == "dw":
        return lib.mok_grouped_matmul_dw(a, lda, b, ldb, off, o64, rows, E, n, k, out, f32, scratch, nbytes, None)
    return getattr(lib, "mok_grouped_matmul" + which)(a, lda, b, off, o64, rows, E, n, k, out, ldo, rest, scratch,
                                                      nbytes, None)


@pytest.mark.parametrize("which", ["", "_dx"])
@pytest.mark.parametrize("want,kw", [
    (INVALID, dict(rows=-1)), (INVALID, dict(E=0)), (INVALID, dict(n=0)), (INVALID, dict(k=0)), (INVALID, dict(o64=2)),
    (INVALID, dict(rest=-1)), (INVALID, dict(a=None)), (INVALID, dict(b=None)), (INVALID, dict(off=None)),
    (INVALID, dict(out=None)), (INVALID, dict(lda=63)), (INVALID, dict(ldo=63)), (INVALID, dict(a=P + 1)),
    (INVALID, dict(b=P + 1)), (INVALID, dict(out=P + 1)), (INVALID, dict(off=P + 2)), (INVALID, dict(o64=1, off=P + 4)),
    (UNSUPPORTED, dict(E=1025)), (UNSUPPORTED, dict(n=(1 << 20) + 1, lda=1 << 21, ldo=1 << 21)),
    (UNSUPPORTED, dict(k=(1 << 20) + 1)), (UNSUPPORTED, dict(lda=(1 << 21) + 1)),
    (UNSUPPORTED, dict(ldo=(1 << 21) + 1)), (UNSUPPORTED, dict(rows=(1 << 30) + 1)),
    (OK, dict(rows=0, a=None, b=None, out=None, off=None))])
def test_grouped_refusals(which, want, kw):
    assert grouped(which, **kw) == want


@pytest.mark.parametrize("want,kw", [
    (INVALID, dict(rows=-1)), (INVALID, dict(f32=2)), (INVALID, dict(a=None)), (INVALID, dict(b=None)),
    (INVALID, dict(out=None)), (INVALID, dict(out=P + 2, f32=1)), (INVALID, dict(lda=63)), (INVALID, dict(ldb=63)),
    (INVALID, dict(rows=0, out=None)), (INVALID, dict(rows=0, off=None)), (UNSUPPORTED, dict(ldb=(1 << 21) + 1))])
def test_grouped_dw_refusals(want, kw):
    assert grouped("dw", **kw) == want


def test_grouped_scratch():
    """Only a long sum for few outputs is cut into parts, which need scratch."""
    def need(op, rows, E, n, k):
        return _lib.load().mok_grouped_matmul_scratch_bytes(op, rows, E, n, k)
    Y, DX, DW = _lib.MOK_GROUPED_Y, _lib.MOK_GROUPED_DX, _lib.MOK_GROUPED_DW
    assert need(Y, 64, 2, 128, 4096) % (64 * 128 * 4) == 0 and need(Y, 64, 2, 128, 4096) > 64 * 128 * 4
    assert need(Y, 64, 2, 128, 64) == 0 and need(Y, 65536, 128, 768, 2048) == 0 and need(Y, 0, 2, 128, 4096) == 0
    assert need(DX, 64, 2, 4096, 128) == need(Y, 64, 2, 128, 4096) and need(DX, 64, 2, 128, 4096) == 0
    assert need(DW, 40000, 2, 128, 64) > 2 * 128 * 64 * 4 and need(DW, 64, 2, 128, 64) == 0
    for bad in ((3, 64, 2, 128, 4096), (-1, 64, 2, 128, 4096), (Y, -1, 2, 128, 4096), (Y, 64, 0, 128, 4096),
                (Y, 64, 2000, 128, 4096), (Y, 64, 2, 0, 4096), (Y, 64, 2, 128, (1 << 20) + 1)):
        assert need(*bad) == 0, bad
    few = dict(rows=64, E=2, n=128, k=4096, lda=4096, ldo=128)
    assert grouped(**few, scratch=P, nbytes=need(Y, 64, 2, 128, 4096) - 1) == SMALL
    assert grouped(**few, scratch=P + 2, nbytes=1 << 30) == INVALID
    assert grouped(**few, scratch=P + 8, nbytes=1 << 30) == INVALID
    assert grouped("dw", rows=40000, n=128, k=64, lda=128, scratch=P, nbytes=64) == SMALL


def quantize(src=P, f32=0, rows=4, cols=256, ld=256, form=0, group=128, codes=P, scale=P, zero=None):
    return _lib.load().mok_w4_quantize(src, f32, rows, cols, ld, form, group, codes, scale, zero, None)


@pytest.mark.parametrize("want,kw", [
    (INVALID, dict(rows=-1)), (INVALID, dict(cols=-128)), (INVALID, dict(f32=3)), (INVALID, dict(form=2)),
    (INVALID, dict(form=-1)), (INVALID, dict(src=None)), (INVALID, dict(codes=None)), (INVALID, dict(scale=None)),
    (INVALID, dict(ld=255)), (INVALID, dict(scale=P + 1)), (INVALID, dict(form=1, group=32, zero=P)),
    (UNSUPPORTED, dict(group=16)), (UNSUPPORTED, dict(group=256)), (UNSUPPORTED, dict(form=1, group=64)),
    (UNSUPPORTED, dict(cols=192, ld=192)), (UNSUPPORTED, dict(ld=260)), (UNSUPPORTED, dict(src=P + 8)),
    (UNSUPPORTED, dict(codes=P + 2)), (UNSUPPORTED, dict(rows=1 << 40)), (UNSUPPORTED, dict(ld=1 << 40)),
    (OK, dict(rows=0)), (OK, dict(cols=0, ld=0))])
def test_quantize_refusals(want, kw):
    assert quantize(**kw) == want


def weight(codes=P, scale=P, zero=None):
    return _lib.MokW4(codes, scale, zero)


def test_dequantize_refusals():
    def call(w=weight(), rows=4, cols=256, form=0, group=128, dst=P):
        return _lib.load().mok_w4_dequantize(None if w is None else C.byref(w), rows, cols, form, group, dst, None)
    for kw in (dict(w=None), dict(rows=-1), dict(dst=None), dict(w=weight(codes=None)), dict(w=weight(scale=None)),
               dict(w=weight(scale=P + 1)), dict(form=1, group=32, w=weight(zero=P)), dict(form=7)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(cols=64), dict(group=33), dict(dst=P + 8), dict(w=weight(codes=P + 1)), dict(rows=1 << 40)):
        assert call(**kw) == UNSUPPORTED, kw
    assert call(rows=0, dst=None) == OK


def test_product_refusals():
    def call(x=P, ldx=256, T=2, n=8, k=256, form=0, group=128, w=weight(), y=P, ldy=8):
        return _lib.load().mok_w4_matmul(x, ldx, T, n, k, form, group, None if w is None else C.byref(w), y, ldy, None)
    for kw in (dict(T=-1), dict(n=0), dict(k=0), dict(w=None), dict(x=None), dict(y=None), dict(ldx=255), dict(ldy=7),
               dict(y=P + 1), dict(w=weight(codes=None)), dict(form=1, group=32, w=weight(zero=P))):
        assert call(**kw) == INVALID, kw
    for kw in (dict(T=65536), dict(n=1 << 27), dict(k=1 << 21), dict(k=192), dict(x=P + 8), dict(ldx=260),
               dict(w=weight(codes=P + 8)), dict(group=48)):
        assert call(**kw) == UNSUPPORTED, kw
    assert call(T=0, x=None, y=None) == OK


def layer(T=4, x=P, rw=P, ids=P, out=P, scratch=P, nbytes=1 << 30, null=False, weights=None, **kw):
    l = _lib.MokW4Layer(struct_size=C.sizeof(_lib.MokW4Layer), hidden=256, intermediate=128, num_experts=8, topk=2,
                        shared_intermediate=128, format=0, group=128, swiglu_limit=0.0)
    for n in ("routed_gate", "routed_up", "routed_down", "shared_gate", "shared_up", "shared_down"):
        setattr(l, n, weight())
    for n, v in {**kw, **(weights or {})}.items():
        setattr(l, n, v)
    p = None if null else C.byref(l)
    return (_lib.load().mok_forward_w4(p, x, rw, ids, T, out, scratch, nbytes, None),
            _lib.load().mok_forward_w4_scratch_bytes(p, T))


@pytest.mark.parametrize("want,kw", [
    (INVALID, dict(null=True)), (INVALID, dict(struct_size=8)), (INVALID, dict(T=-1)), (INVALID, dict(hidden=0)),
    (INVALID, dict(intermediate=0)), (INVALID, dict(num_experts=0)), (INVALID, dict(topk=0)),
    (INVALID, dict(shared_intermediate=-128)), (INVALID, dict(swiglu_limit=-1.0)),
    (INVALID, dict(swiglu_limit=float("nan"))), (INVALID, dict(swiglu_limit=float("inf"))), (INVALID, dict(format=2)),
    (UNSUPPORTED, dict(hidden=192)), (UNSUPPORTED, dict(intermediate=64)), (UNSUPPORTED, dict(shared_intermediate=32)),
    (UNSUPPORTED, dict(hidden=1 << 17)), (UNSUPPORTED, dict(num_experts=1025)), (UNSUPPORTED, dict(topk=65)),
    (UNSUPPORTED, dict(T=8193, topk=1)), (UNSUPPORTED, dict(T=4097)), (UNSUPPORTED, dict(group=16))])
def test_layer_size_refusals(want, kw):
    assert layer(**kw) == (want, 0)


def test_layer_refusals():
    bytes_ = layer(x=None)[1]
    assert bytes_ > 0
    for kw in (dict(x=None), dict(rw=None), dict(ids=None), dict(out=None), dict(scratch=None), dict(ids=P + 4),
               dict(rw=P + 2), dict(out=P + 1), dict(weights=dict(routed_up=weight(codes=None))),
               dict(weights=dict(shared_down=weight(scale=None))), dict(weights=dict(routed_down=weight(zero=P))),
               dict(weights=dict(shared_up=weight(scale=P + 1)))):
        assert layer(**kw) == (INVALID, bytes_), kw
    for kw in (dict(x=P + 8), dict(scratch=P + 8), dict(weights=dict(routed_gate=weight(codes=P + 8)))):
        assert layer(**kw) == (UNSUPPORTED, bytes_), kw
    assert layer(nbytes=bytes_ - 1) == (SMALL, bytes_)
    assert layer(T=0, x=None, out=None)[0] == OK


def test_python_refuses_the_cpu_and_what_is_no_tensor():
    x, w, off = torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(2, 8, 8, dtype=torch.bfloat16), torch.zeros(3).int()
    q = torch.zeros(8, 64, dtype=torch.uint8)
    for call in (lambda: mok.grouped_matmul(x, w, off), lambda: mok.grouped_matmul_backward(x, x, w, off),
                 lambda: mok.w4_quantize(x), lambda: mok.w4_dequantize(q, x), lambda: mok.w4_matmul(x, q, x),
                 lambda: mok.forward_w4(x, x, off, {})):
        with pytest.raises(ValueError, match="must live on the GPU"):
            call()
    for call in (lambda: mok.grouped_matmul(None, w, off), lambda: mok.w4_quantize([1.0]),
                 lambda: mok.w4_matmul(3, q, x), lambda: mok.forward_w4("x", x, off, {})):
        with pytest.raises(ValueError, match="must be a tensor"):
            call()
    with pytest.raises(ValueError, match="dw_dtype"):
        mok.grouped_matmul_backward(x, x, w, off, dw_dtype=torch.float16)
    with pytest.raises(ValueError, match="format"):
        mok.w4_quantize(x, format="fp4")
