"""Refusals of the operators around the layer, on the CPU: every case fails
the host-side checks of the C ABI (pointers are never followed) or of the
Python binding before any device work."""
import ctypes as C

import pytest

from mokutil import ROOT  # noqa: F401

torch = pytest.importorskip("torch")
import mixture_experts_layer_build_amd as mok  # noqa: E402
from mixture_experts_layer_build_amd import _lib  # noqa: E402
from mixture_experts_layer_build_amd.autograd import MoKRMSNorm, MoKRouter  # noqa: E402
from mixture_experts_layer_build_amd.optim import MoKAdamW  # noqa: E402

INVALID, UNSUPPORTED, SMALL, OK = (_lib.MOK_ERR_INVALID_ARGUMENT, _lib.MOK_ERR_UNSUPPORTED,
                                   _lib.MOK_ERR_BUFFER_TOO_SMALL, _lib.MOK_OK)
P = 1 << 20  # an address that is never followed


def norm(x=P, x32=0, ldx=64, res=None, res32=0, ldr=0, w=P, w32=0, rows=4, cols=64, eps=1e-6, s=None, y=P, codes=None,
         scale=None, rstd=None):
    return _lib.load().mok_rms_norm(x, x32, ldx, res, res32, ldr, w, w32, rows, cols, eps, s, y, codes, scale, rstd, None)


@pytest.mark.parametrize("want,kw", [
    (INVALID, dict(rows=-1)), (INVALID, dict(cols=0)), (INVALID, dict(x32=2)), (INVALID, dict(w32=-1)),
    (INVALID, dict(eps=-1.0)), (INVALID, dict(eps=float("nan"))), (INVALID, dict(eps=float("inf"))),
    (INVALID, dict(x=None)), (INVALID, dict(w=None)), (INVALID, dict(y=None)), (INVALID, dict(ldx=63)),
    (INVALID, dict(res=P, ldr=64)), (INVALID, dict(s=P)), (INVALID, dict(codes=P)), (INVALID, dict(scale=P)),
    (INVALID, dict(res=P, s=P, ldr=32)), (UNSUPPORTED, dict(x32=1, res=P, s=P, ldr=64)),
    (INVALID, dict(x=P + 1)), (INVALID, dict(x32=1, x=P + 2)), (INVALID, dict(rstd=P + 2)),
    (UNSUPPORTED, dict(cols=1 << 25, ldx=1 << 25)),
    # MXFP8
    (UNSUPPORTED, dict(codes=P, scale=P, cols=48)), (UNSUPPORTED, dict(codes=P, scale=P, cols=16416, ldx=16416)),
    (UNSUPPORTED, dict(codes=P, scale=P, ldx=65)), (UNSUPPORTED, dict(codes=P + 4, scale=P)),
    (UNSUPPORTED, dict(codes=P, scale=P, x=P + 2)), (UNSUPPORTED, dict(codes=P, scale=P, w=P + 8)),
    (OK, dict(rows=0, x=None, w=None, y=None))])
def test_rms_norm_refusals(want, kw):
    assert norm(**kw) == want


def norm_bwd(dy=P, lddy=64, s=P, s32=0, lds=64, rstd=P, w=P, w32=0, dsum=None, ldd=0, rows=4, cols=64, ds=P, dx=None,
             dw=P, scratch=P, nbytes=1 << 30):
    return _lib.load().mok_rms_norm_backward(dy, lddy, s, s32, lds, rstd, w, w32, dsum, ldd, rows, cols, ds, dx, dw,
                                             scratch, nbytes, None)


@pytest.mark.parametrize("want,kw", [
    (INVALID, dict(rows=-1)), (INVALID, dict(cols=0)), (INVALID, dict(s32=3)), (INVALID, dict(dy=None)),
    (INVALID, dict(s=None)), (INVALID, dict(rstd=None)), (INVALID, dict(w=None)), (INVALID, dict(ds=None)),
    (INVALID, dict(dw=None)), (INVALID, dict(scratch=None)), (INVALID, dict(scratch=P + 4)), (INVALID, dict(lddy=63)),
    (INVALID, dict(lds=8)), (INVALID, dict(dsum=P, ldd=8)), (INVALID, dict(dx=P + 1)), (SMALL, dict(nbytes=64))])
def test_rms_norm_backward_refusals(want, kw):
    assert norm_bwd(**kw) == want


def test_scratch_sizes():
    lib = _lib.load()
    assert lib.mok_rms_norm_scratch_bytes(-1, 64) == 0 and lib.mok_rms_norm_scratch_bytes(4, 0) == 0
    assert lib.mok_rms_norm_scratch_bytes(0, 64) >= 1 and lib.mok_rms_norm_scratch_bytes(4, 64) >= 4 * 64 * 4
    assert lib.mok_router_scratch_bytes(-1, 8) == 0 and lib.mok_router_scratch_bytes(4, 1025) == 0
    assert lib.mok_router_scratch_bytes(0, 8) >= 2 * 9 * 4


def router(logits=P, l32=1, T=4, ld=8, E=8, k=2, bias=None, mask=None, scoring=0, renorm=1, scale=1.0, w=P, ids=P,
           counts=None, losses=None, scratch=None, nbytes=0):
    return _lib.load().mok_router_topk(logits, l32, T, ld, E, k, bias, mask, scoring, renorm, scale, w, ids, counts,
                                       losses, scratch, nbytes, None)


@pytest.mark.parametrize("want,kw", [
    (INVALID, dict(T=-1)), (INVALID, dict(E=0)), (INVALID, dict(k=0)), (INVALID, dict(k=9)), (INVALID, dict(l32=2)),
    (INVALID, dict(scoring=2)), (INVALID, dict(scoring=-1)), (INVALID, dict(renorm=5)),
    (INVALID, dict(scale=float("inf"))), (INVALID, dict(scale=float("nan"))), (INVALID, dict(logits=None)),
    (INVALID, dict(ld=7)), (INVALID, dict(w=None)), (INVALID, dict(ids=None)), (INVALID, dict(ids=P + 4)),
    (INVALID, dict(counts=P)), (INVALID, dict(losses=P)), (INVALID, dict(counts=P, losses=P)),
    (SMALL, dict(counts=P, losses=P, scratch=P, nbytes=8)), (INVALID, dict(bias=P + 2)), (INVALID, dict(logits=P + 2)),
    (UNSUPPORTED, dict(E=1025, ld=1025)), (UNSUPPORTED, dict(T=1 << 30)), (UNSUPPORTED, dict(ld=(1 << 22) + 1)), (UNSUPPORTED, dict(E=128, ld=128, k=65)),
    (OK, dict(T=0, logits=None, w=None, ids=None))])
def test_router_refusals(want, kw):
    assert router(**kw) == want


def test_router_backward_refusals():
    def call(dw=P, logits=P, T=4, ld=8, E=8, k=2, ids=P, counts=None, dl=None, out=P, scoring=0):
        return _lib.load().mok_router_topk_backward(dw, logits, 1, T, ld, E, k, None, None, scoring, 1, 1.0, ids, counts,
                                                    dl, out, None)
    for kw in (dict(dw=None), dict(ids=None), dict(out=None), dict(counts=P), dict(dl=P), dict(k=9), dict(scoring=7),
               dict(out=P + 2), dict(T=-1)):
        assert call(**kw) == INVALID, kw
    assert call(E=2000, ld=2000) == UNSUPPORTED
    assert call(T=0, dw=None, ids=None, out=None, logits=None) == OK


def adamw(**kw):
    arr = (C.c_void_p * 1)(P)
    n = (C.c_int64 * 1)(kw.pop("numel", 64))
    a = _lib.MokAdamW(struct_size=C.sizeof(_lib.MokAdamW), count=1, lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8,
                      weight_decay=0.1, step=1, state_bits=32)
    for f in ("params", "grads", "exp_avgs", "exp_avg_sqs"):
        setattr(a, f, C.addressof(arr))
    a.numels = C.addressof(n)
    hold = []
    for f, v in kw.items():
        if isinstance(v, list):
            hold.append((C.c_void_p * 1)(*v))
            v = C.addressof(hold[-1])
        setattr(a, f, v)
    return _lib.load().mok_adamw_step(C.byref(a), None)


@pytest.mark.parametrize("want,kw", [
    (INVALID, dict(struct_size=8)), (INVALID, dict(count=-1)), (OK, dict(count=0)), (INVALID, dict(step=0)),
    (INVALID, dict(lr=-1.0)), (INVALID, dict(lr=float("nan"))), (INVALID, dict(beta1=1.0)), (INVALID, dict(beta2=-0.1)),
    (INVALID, dict(eps=-1.0)), (INVALID, dict(weight_decay=float("inf"))), (UNSUPPORTED, dict(state_bits=16)),
    (INVALID, dict(state_bits=8)), (INVALID, dict(exp_avg_scales=[P])), (INVALID, dict(params=None)),
    (INVALID, dict(grads=[None])), (INVALID, dict(numel=-1)), (INVALID, dict(param_fp32=1, masters=[P])),
    (INVALID, dict(masters=[None])), (INVALID, dict(param_fp32=1, params=[P + 2])), (INVALID, dict(exp_avgs=[P + 2])),
    (INVALID, dict(grad_scale=P + 1)), (INVALID, dict(param_fp32=7))])
def test_adamw_refusals(want, kw):
    assert adamw(**kw) == want
    assert _lib.load().mok_adamw_step(None, None) == INVALID


def test_forward_mxfp8_refuses_null_and_misaligned_codes():
    lib = _lib.load()
    w = _lib.MokWeights()
    assert lib.mok_forward_mxfp8(None, P, 1 << 20, None, P, P, C.byref(w), P, None, 0, None) == INVALID
    assert lib.mok_forward_mxfp8(None, P, 1 << 20, P + 8, P, P, C.byref(w), P, None, 0, None) == UNSUPPORTED
    assert lib.mok_forward_mxfp8(None, P, 1 << 20, P, P + 1, P, C.byref(w), P, None, 0, None) == UNSUPPORTED
    assert lib.mok_forward_mxfp8(None, P, 1 << 20, P, P, P, C.byref(w), P, None, 0, None) == INVALID  # no workspace


def test_cpu_tensors_are_rejected():
    x, w = torch.zeros(2, 64, dtype=torch.bfloat16), torch.ones(64, dtype=torch.bfloat16)
    for call in (lambda: mok.rms_norm(x, w), lambda: mok.rms_norm_mxfp8(x, w),
                 lambda: mok.rms_norm_backward(x, x, torch.ones(2), w), lambda: mok.router_topk(torch.zeros(2, 8), 2),
                 lambda: mok.router_topk_backward(torch.zeros(2, 2), torch.zeros(2, 8), torch.zeros(2, 2, dtype=torch.int64)),
                 lambda: mok.adamw_step([w], [w], [w.float()], [w.float()], step=1, lr=1e-3),
                 lambda: MoKRMSNorm(64)(x), lambda: MoKRouter(64, 8, 2)(x)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_optimizer_checks_its_arguments():
    p = torch.nn.Parameter(torch.zeros(4))
    for kw in (dict(state_bits=16), dict(lr=-1.0), dict(betas=(1.0, 0.9)), dict(eps=-1e-8), dict(weight_decay=-1.0)):
        with pytest.raises(ValueError):
            MoKAdamW([p], **kw)
    opt = MoKAdamW([p])
    opt.step()  # no gradient: nothing to do
    with pytest.raises(ValueError, match="bf16 or fp32"):
        q = torch.nn.Parameter(torch.zeros(4, dtype=torch.float64))
        q.grad = torch.zeros(4, dtype=torch.float64)
        MoKAdamW([q]).step()


def test_a_loaded_state_keeps_its_types():
    p = torch.nn.Parameter(torch.zeros(40, dtype=torch.bfloat16))
    opt = MoKAdamW([p], state_bits=8)
    st = opt._init_state(p, opt.param_groups[0])
    st["exp_avg"].fill_(200)
    st["step"] = 3
    opt.state[p].update(st)
    q = torch.nn.Parameter(torch.zeros(40, dtype=torch.bfloat16))
    other = MoKAdamW([q], state_bits=8)
    other.load_state_dict(opt.state_dict())
    got = other.state[q]
    assert got["exp_avg"].dtype == torch.uint8 and bool((got["exp_avg"] == 200).all()) and got["step"] == 3
    assert got["exp_avg_sq_scale"].dtype == torch.uint8 and got["master"].dtype == torch.float32
    got["exp_avg"].zero_()  # a copy, not the saved tensor
    assert bool((st["exp_avg"] == 200).all())


def test_forward_mxfp8_checks_its_tensors_before_it_calls():
    class Ws:  # (what the checks read of a workspace)
        cfg = mok.MoKConfig(hidden=64, intermediate=128, num_experts=4, topk=2, max_tokens=8)
        device, handle = 0, None

    def call(T=4, rw=None, out=None):
        return mok.forward_mxfp8(Ws, torch.zeros(16, dtype=torch.uint8), torch.zeros(T, 64, dtype=torch.uint8),
                                 torch.zeros(T, 2, dtype=torch.uint8), torch.zeros(rw or T, 2), {}, out=out)
    for match, kw in (("topk", dict(rw=3)), ("max_tokens", dict(T=9)), ("out", dict(out=torch.zeros(4, 64))),
                      ("out", dict(out=torch.zeros(3, 64, dtype=torch.bfloat16))), ("GPU 0", dict())):
        with pytest.raises(ValueError, match=match):
            call(**kw)


def test_a_refused_step_is_not_counted():
    p = torch.nn.Parameter(torch.zeros(4))
    p.grad = torch.ones(4)
    opt = MoKAdamW([p])
    with pytest.raises(ValueError, match="CUDA"):
        opt.step()
    assert opt.state[p]["step"] == 0


def test_what_is_no_tensor_is_refused():
    w = torch.ones(64, dtype=torch.bfloat16)
    for call in (lambda: mok.rms_norm(None, w), lambda: mok.rms_norm_mxfp8([1.0], w), lambda: mok.router_topk(None, 2),
                 lambda: mok.rms_norm_backward(None, w, w, w), lambda: mok.router_topk_backward(w, None, w),
                 lambda: mok.adamw_step([None], [w], [w], [w], step=1, lr=1e-3)):
        with pytest.raises(ValueError, match="must be a tensor"):
            call()
