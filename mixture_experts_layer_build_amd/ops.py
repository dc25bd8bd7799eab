"""The operators around the layer: RMS norm, top-k router, AdamW step.

Direct calls over the C ABI (``include/mok.h`` states formulas, types and
refusals); the package re-exports them. They allocate their outputs with
torch, enqueue on the current stream of the tensors' device, and need no
workspace. Tensors on the CPU are rejected: there is no fallback.
"""
from __future__ import annotations

import ctypes as C

import torch

from . import _lib

__all__ = ["rms_norm", "rms_norm_mxfp8", "rms_norm_backward", "router_topk", "router_topk_backward", "adamw_step"]

_BF16, _F32, _U8 = torch.bfloat16, torch.float32, torch.uint8
_FLOATS = (_BF16, _F32)
_CODES = (_U8, torch.float8_e4m3fn)
_SCALES = (_U8, torch.float8_e8m0fnu)
_SCORING = {"softmax": _lib.MOK_ROUTER_SOFTMAX, "sigmoid": _lib.MOK_ROUTER_SIGMOID}


def _call(name: str, device: torch.device, *args) -> None:
    """Runs one library call on `device` and its current stream."""
    index = device.index
    if index is None or index == torch.cuda.current_device():
        st = getattr(_lib.load(), name)(*args, torch.cuda.current_stream().cuda_stream)
    else:
        with torch.cuda.device(index):
            st = getattr(_lib.load(), name)(*args, torch.cuda.current_stream().cuda_stream)
    if st != _lib.MOK_OK:
        raise _lib.MokError(name, st)


def _gpu(name: str, t: torch.Tensor) -> torch.device:
    if not t.is_cuda:
        raise ValueError(f"{name} must live on the GPU (a CUDA tensor)")
    return t.device


def _check(name: str, t, device: torch.device, dtypes, shape=None) -> None:
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, not on {device}")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, got {t.dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _dense(name: str, t: torch.Tensor) -> int:
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _rows(name: str, t: torch.Tensor) -> tuple[int, int]:
    """(address, row stride) of a tensor whose last dimension is dense and
    whose rows lie at one stride."""
    if t.is_contiguous():
        return t.data_ptr(), t.shape[-1]
    if t.dim() != 2 or (t.stride(1) != 1 and t.shape[1] > 1) or t.stride(0) < t.shape[1]:
        raise ValueError(f"{name} must be contiguous, or 2-D with dense rows that do not overlap")
    return t.data_ptr(), t.stride(0)


def _row_count(t: torch.Tensor) -> int:
    return t.numel() // t.shape[-1] if t.shape[-1] else 0


def _norm(x, weight, residual, eps, y, codes, scale, rstd):
    dev = _gpu("x", x)
    if x.dim() < 1 or x.shape[-1] < 1:
        raise ValueError("x must have a last dimension of at least 1")
    _check("x", x, dev, _FLOATS)
    _check("weight", weight, dev, _FLOATS, x.shape[-1:])
    px, ldx = _rows("x", x)
    total, pr, ldr, res32, ps = None, None, 0, 0, None
    if residual is not None:
        _check("residual", residual, dev, _FLOATS, x.shape)
        pr, ldr = _rows("residual", residual)
        res32 = int(residual.dtype == _F32)
        total = torch.empty(x.shape, dtype=residual.dtype, device=dev)
        ps = total.data_ptr()
    _call("mok_rms_norm", dev, px, int(x.dtype == _F32), ldx, pr, res32, ldr, _dense("weight", weight),
          int(weight.dtype == _F32), _row_count(x), x.shape[-1], eps, ps, y, codes, scale, rstd)
    return total


def rms_norm(x: torch.Tensor, weight: torch.Tensor, residual: torch.Tensor | None = None, eps: float = 1e-6):
    """y = rms_norm(x + residual) * weight in bf16. Returns (y, sum, rstd):
    sum = x + residual in the residual's type (None without a residual), rstd
    fp32 with one value per row. x bf16 or fp32 [..., cols]."""
    _gpu("x", x)
    y = torch.empty(x.shape, dtype=_BF16, device=x.device)
    rstd = torch.empty(x.shape[:-1], dtype=_F32, device=x.device)
    total = _norm(x, weight, residual, eps, y.data_ptr(), None, None, rstd.data_ptr())
    return y, total, rstd


def rms_norm_mxfp8(x: torch.Tensor, weight: torch.Tensor, residual: torch.Tensor | None = None, eps: float = 1e-6,
                   y: torch.Tensor | None = None, rstd: torch.Tensor | None = None):
    """The norm with its output in MXFP8, as ``forward_mxfp8`` takes it.
    Returns (codes uint8 [..., cols], scale uint8 [..., cols/32], sum). Give
    ``y`` (bf16, x's shape) and ``rstd`` (fp32, one per row) to have them
    filled too, for a backward."""
    dev = _gpu("x", x)
    if x.dim() < 1 or x.shape[-1] % 32 != 0:
        raise ValueError("MXFP8 needs a last dimension that is a multiple of 32")
    if y is not None:
        _check("y", y, dev, (_BF16,), x.shape)
    if rstd is not None:
        _check("rstd", rstd, dev, (_F32,), x.shape[:-1])
    codes = torch.empty(x.shape, dtype=_U8, device=dev)
    scale = torch.empty(x.shape[:-1] + (x.shape[-1] // 32,), dtype=_U8, device=dev)
    total = _norm(x, weight, residual, eps, None if y is None else _dense("y", y), codes.data_ptr(),
                  scale.data_ptr(), None if rstd is None else _dense("rstd", rstd))
    return codes, scale, total


def rms_norm_backward(dy: torch.Tensor, s: torch.Tensor, rstd: torch.Tensor, weight: torch.Tensor,
                      d_sum: torch.Tensor | None = None, dx: torch.Tensor | None = None):
    """(ds, d_weight) from dy (bf16), the saved s (the forward's sum, or x
    without a residual) and rstd; ``d_sum`` is the gradient that arrives
    through the sum. ds is the gradient of x and of the residual, in s's
    type; ``dx`` (bf16) receives it in bf16 as well."""
    dev = _gpu("dy", dy)
    if dy.dim() < 1 or dy.shape[-1] < 1:
        raise ValueError("dy must have a last dimension of at least 1")
    _check("dy", dy, dev, (_BF16,))
    _check("s", s, dev, _FLOATS, dy.shape)
    _check("rstd", rstd, dev, (_F32,), dy.shape[:-1])
    _check("weight", weight, dev, _FLOATS, dy.shape[-1:])
    rows, cols = _row_count(dy), dy.shape[-1]
    pdy, lddy = _rows("dy", dy)
    ps, lds = _rows("s", s)
    pd, ldd = None, 0
    if d_sum is not None:
        _check("d_sum", d_sum, dev, (s.dtype,), dy.shape)
        pd, ldd = _rows("d_sum", d_sum)
    if dx is not None:
        _check("dx", dx, dev, (_BF16,), dy.shape)
    ds = torch.empty(s.shape, dtype=s.dtype, device=dev)
    d_weight = torch.empty(weight.shape, dtype=weight.dtype, device=dev)
    nbytes = _lib.load().mok_rms_norm_scratch_bytes(rows, cols)
    scratch = torch.empty(nbytes, dtype=_U8, device=dev)
    _call("mok_rms_norm_backward", dev, pdy, lddy, ps, int(s.dtype == _F32), lds, _dense("rstd", rstd),
          _dense("weight", weight), int(weight.dtype == _F32), pd, ldd, rows, cols, ds.data_ptr(),
          None if dx is None else _dense("dx", dx), d_weight.data_ptr(), scratch.data_ptr(), nbytes)
    return ds, d_weight


def _router_args(logits, bias, token_mask, scoring):
    dev = _gpu("logits", logits)
    if logits.dim() != 2:
        raise ValueError("logits must be [tokens, experts]")
    _check("logits", logits, dev, _FLOATS)
    if scoring not in _SCORING:
        raise ValueError(f"scoring must be one of {sorted(_SCORING)}, got {scoring!r}")
    T, E = logits.shape
    pl, ld = _rows("logits", logits)
    pb = pm = None
    if bias is not None:
        _check("bias", bias, dev, (_F32,), (E,))
        pb = _dense("bias", bias)
    if token_mask is not None:
        _check("token_mask", token_mask, dev, (torch.bool, _U8), (T,))
        pm = _dense("token_mask", token_mask)
    return dev, T, E, pl, ld, pb, pm


def router_topk(logits: torch.Tensor, k: int, *, scoring: str = "softmax", renormalize: bool = True,
                scale: float = 1.0, bias: torch.Tensor | None = None, token_mask: torch.Tensor | None = None,
                losses: bool = False):
    """Top-k routing of logits [T, E] (bf16 or fp32): (weights fp32 [T, k],
    ids int64 [T, k]), the layer's router_weights and top_experts. With
    ``losses`` also (counts int32 [E + 1], losses fp32 [2]): choices per
    expert and the number of live tokens; the load-balance and the z loss."""
    dev, T, E, pl, ld, pb, pm = _router_args(logits, bias, token_mask, scoring)
    weights = torch.empty((T, k), dtype=_F32, device=dev)
    ids = torch.empty((T, k), dtype=torch.int64, device=dev)
    counts = loss = scratch = None
    nbytes = 0
    if losses:
        counts = torch.empty(E + 1, dtype=torch.int32, device=dev)
        loss = torch.empty(2, dtype=_F32, device=dev)
        nbytes = _lib.load().mok_router_scratch_bytes(T, E)
        scratch = torch.empty(nbytes, dtype=_U8, device=dev)
    _call("mok_router_topk", dev, pl, int(logits.dtype == _F32), T, ld, E, k, pb, pm, _SCORING[scoring],
          int(renormalize), scale, weights.data_ptr(), ids.data_ptr(), counts.data_ptr() if losses else None,
          loss.data_ptr() if losses else None, scratch.data_ptr() if losses else None, nbytes)
    return (weights, ids, counts, loss) if losses else (weights, ids)


def router_topk_backward(d_weights: torch.Tensor, logits: torch.Tensor, ids: torch.Tensor, *,
                         scoring: str = "softmax", renormalize: bool = True, scale: float = 1.0,
                         bias: torch.Tensor | None = None, token_mask: torch.Tensor | None = None,
                         counts: torch.Tensor | None = None, d_losses: torch.Tensor | None = None) -> torch.Tensor:
    """Gradient to the logits [T, E] in their type, from d_weights (fp32)
    and the forward's ids; ``counts`` and ``d_losses`` (fp32 [2]) where the
    losses have a gradient. The other arguments as in the forward."""
    dev, T, E, pl, ld, pb, pm = _router_args(logits, bias, token_mask, scoring)
    if ids.dim() != 2:
        raise ValueError("ids must be [tokens, k]")
    k = ids.shape[1]
    _check("ids", ids, dev, (torch.int64,), (T, k))
    _check("d_weights", d_weights, dev, (_F32,), (T, k))
    if (counts is None) != (d_losses is None):
        raise ValueError("counts and d_losses come together")
    if counts is not None:
        _check("counts", counts, dev, (torch.int32,), (E + 1,))
        _check("d_losses", d_losses, dev, (_F32,), (2,))
    d_logits = torch.empty((T, E), dtype=logits.dtype, device=dev)
    _call("mok_router_topk_backward", dev, _dense("d_weights", d_weights), pl, int(logits.dtype == _F32), T, ld, E, k,
          pb, pm, _SCORING[scoring], int(renormalize), scale, _dense("ids", ids),
          None if counts is None else _dense("counts", counts),
          None if d_losses is None else _dense("d_losses", d_losses), d_logits.data_ptr())
    return d_logits


def _one_of(name: str, tensors, dtypes) -> torch.dtype:
    """The one dtype of a list of dense tensors."""
    found = {t.dtype for t in tensors}
    if len(found) != 1 or not found <= set(dtypes):
        raise ValueError(f"{name} must all be {' or all '.join(str(d) for d in dtypes)}, got {found}")
    for t in tensors:
        if not t.is_contiguous():
            raise ValueError(f"every tensor of {name} must be contiguous")
    return found.pop()


def _sizes(name: str, tensors, numels) -> None:
    if [t.numel() for t in tensors] != numels:
        raise ValueError(f"the tensors of {name} must have the sizes of the params")


def _pointers(tensors):
    return (C.c_void_p * len(tensors))(*[t.data_ptr() for t in tensors])


def adamw_step(params, grads, exp_avgs, exp_avg_sqs, masters=None, *, step: int, lr: float,
               betas: tuple[float, float] = (0.9, 0.999), eps: float = 1e-8, weight_decay: float = 0.0,
               grad_scale: torch.Tensor | None = None, seed: int | None = None) -> None:
    """One AdamW step of many tensors, in place. Lists of equal length: params
    (all bf16 or all fp32), grads (all bf16 or all fp32), the moments, and for
    bf16 params optionally their fp32 masters. Moments are fp32 tensors, or
    for 8-bit states pairs (codes, scale): E4M3 codes [numel] of m (of
    sqrt(v)) and E8M0 scales [ceil(numel/32)], zeros at the start. grad_scale:
    a device fp32 tensor of one element that multiplies every gradient. seed
    (default: the step) chooses the 8-bit states' roundings. No two tensors
    may overlap."""
    n = len(params)
    lists = dict(grads=grads, exp_avgs=exp_avgs, exp_avg_sqs=exp_avg_sqs)
    if masters is not None:
        lists["masters"] = masters
    for name, ts in lists.items():
        if len(ts) != n:
            raise ValueError(f"{name} has {len(ts)} tensors, params {n}")
    if n == 0:
        return
    dev = _gpu("params", params[0])
    numels = [t.numel() for t in params]
    pdt = _one_of("params", params, _FLOATS)
    gdt = _one_of("grads", grads, _FLOATS)
    _sizes("grads", grads, numels)
    small = isinstance(exp_avgs[0], (tuple, list))
    written, arrays = list(params), {}
    arrays["params"], arrays["grads"] = _pointers(params), _pointers(grads)
    if masters is not None:
        if pdt != _BF16:
            raise ValueError("masters go with bf16 params")
        _one_of("masters", masters, (_F32,))
        _sizes("masters", masters, numels)
        arrays["masters"] = _pointers(masters)
        written += masters
    for name, ts in (("exp_avg", exp_avgs), ("exp_avg_sq", exp_avg_sqs)):
        if small:
            try:
                codes, scales = zip(*ts)
            except (TypeError, ValueError):
                raise ValueError(f"{name}s must be pairs (codes, scale)") from None
            _one_of(name + "s", codes, _CODES)
            _one_of(name + " scales", scales, _SCALES)
            _sizes(name + "s", codes, numels)
            _sizes(name + " scales", scales, [(m + 31) // 32 for m in numels])
            arrays[name + "s"], arrays[name + "_scales"] = _pointers(codes), _pointers(scales)
            written += codes
            written += scales
        else:
            _one_of(name + "s", ts, (_F32,))
            _sizes(name + "s", ts, numels)
            arrays[name + "s"] = _pointers(ts)
            written += ts
    if {t.device for t in written} | {t.device for t in grads} != {dev}:
        raise ValueError(f"every tensor must be on {dev}")
    where = [t.data_ptr() for t in written if t.numel()]
    if len(set(where)) != len(where):
        raise ValueError("a tensor that the step writes is given twice")
    if grad_scale is not None:
        _check("grad_scale", grad_scale, dev, (_F32,))
        if grad_scale.numel() != 1:
            raise ValueError("grad_scale must have one element")
    a = _lib.MokAdamW(struct_size=C.sizeof(_lib.MokAdamW), count=n, lr=lr, beta1=betas[0], beta2=betas[1], eps=eps,
                      weight_decay=weight_decay, step=step, param_fp32=int(pdt == _F32), grad_fp32=int(gdt == _F32),
                      state_bits=8 if small else 32, seed=(step if seed is None else seed) & 0xFFFFFFFF,
                      grad_scale=None if grad_scale is None else grad_scale.data_ptr())
    arrays["numels"] = (C.c_int64 * n)(*numels)
    for name, array in arrays.items():
        setattr(a, name, C.addressof(array))
    _call("mok_adamw_step", dev, C.byref(a))
