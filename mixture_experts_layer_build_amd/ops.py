"""The operators around the layer: RMS norm, top-k router, AdamW step.

Direct calls over the C ABI (``include/mok.h`` states formulas, types and
refusals); the package re-exports them. They allocate their outputs with
torch, enqueue on the current stream of the tensors' device, and need no
workspace. Tensors on the CPU are rejected: there is no fallback.
"""
from __future__ import annotations

import ctypes as C
import operator

import torch

from . import _lib

__all__ = ["rms_norm", "rms_norm_mxfp8", "rms_norm_backward", "router_topk", "router_topk_backward", "adamw_step"]

_BF16, _F32, _U8 = torch.bfloat16, torch.float32, torch.uint8
_FLOATS = {_BF16, _F32}
_CODES = {_U8, torch.float8_e4m3fn}
_SCALES = {_U8, torch.float8_e8m0fnu}
_SCORING = {"softmax": _lib.MOK_ROUTER_SOFTMAX, "sigmoid": _lib.MOK_ROUTER_SIGMOID}


def _call(name: str, index: int, *args) -> None:
    """Runs one library call on device `index` and its current stream."""
    if index == torch._C._cuda_getDevice():
        st = getattr(_lib.load(), name)(*args, torch._C._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(index):
            st = getattr(_lib.load(), name)(*args, torch._C._cuda_getCurrentRawStream(index))
    if st != _lib.MOK_OK:
        raise _lib.MokError(name, st)


def _gpu(name: str, t: torch.Tensor) -> int:
    """Index of the tensor's GPU."""
    if not t.is_cuda:
        raise ValueError(f"{name} must live on the GPU (a CUDA tensor)")
    return t.get_device()


def _check(name: str, t, dev: int, dtypes, shape=None) -> None:
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, not on cuda:{dev}")
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


def _norm(x, weight, residual, eps, y, codes, scale, rstd):
    dev = _gpu("x", x)
    shape = x.shape
    cols = shape[-1] if shape else 0
    if cols < 1:
        raise ValueError("x must have a last dimension of at least 1")
    if x.dtype not in _FLOATS:
        raise ValueError(f"x must be bfloat16 or float32, got {x.dtype}")
    _check("weight", weight, dev, _FLOATS, (cols,))
    px, ldx = _rows("x", x)
    total, pr, ldr, res32, ps = None, None, 0, 0, None
    if residual is not None:
        _check("residual", residual, dev, _FLOATS, shape)
        pr, ldr = _rows("residual", residual)
        res32 = residual.dtype == _F32
        total = torch.empty_like(residual, memory_format=torch.contiguous_format)
        ps = total.data_ptr()
    _call("mok_rms_norm", dev, px, x.dtype == _F32, ldx, pr, res32, ldr, _dense("weight", weight),
          weight.dtype == _F32, x.numel() // cols, cols, eps, ps, y, codes, scale, rstd)
    return total


def rms_norm(x: torch.Tensor, weight: torch.Tensor, residual: torch.Tensor | None = None, eps: float = 1e-6):
    """y = rms_norm(x + residual) * weight in bf16. Returns (y, sum, rstd):
    sum = x + residual in the residual's type (None without a residual), rstd
    fp32 with one value per row. x bf16 or fp32 [..., cols]."""
    y = torch.empty_like(x, dtype=_BF16, memory_format=torch.contiguous_format)
    rstd = x.new_empty(x.shape[:-1], dtype=_F32)
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
    codes = torch.empty_like(x, dtype=_U8, memory_format=torch.contiguous_format)
    scale = x.new_empty(x.shape[:-1] + (x.shape[-1] // 32,), dtype=_U8)
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
    rows, cols = dy.numel() // dy.shape[-1], dy.shape[-1]
    pdy, lddy = _rows("dy", dy)
    ps, lds = _rows("s", s)
    pd, ldd = None, 0
    if d_sum is not None:
        _check("d_sum", d_sum, dev, (s.dtype,), dy.shape)
        pd, ldd = _rows("d_sum", d_sum)
    if dx is not None:
        _check("dx", dx, dev, (_BF16,), dy.shape)
    ds = torch.empty_like(s, memory_format=torch.contiguous_format)
    d_weight = torch.empty_like(weight)
    nbytes = _lib.load().mok_rms_norm_scratch_bytes(rows, cols)
    scratch = dy.new_empty(nbytes, dtype=_U8)
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
    weights = logits.new_empty((T, k), dtype=_F32)
    ids = logits.new_empty((T, k), dtype=torch.int64)
    counts = loss = scratch = None
    nbytes = 0
    if losses:
        counts = logits.new_empty(E + 1, dtype=torch.int32)
        loss = logits.new_empty(2, dtype=_F32)
        nbytes = _lib.load().mok_router_scratch_bytes(T, E)
        scratch = logits.new_empty(nbytes, dtype=_U8)
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
    d_logits = torch.empty_like(logits, memory_format=torch.contiguous_format)
    _call("mok_router_topk_backward", dev, _dense("d_weights", d_weights), pl, int(logits.dtype == _F32), T, ld, E, k,
          pb, pm, _SCORING[scoring], int(renormalize), scale, _dense("ids", ids),
          None if counts is None else _dense("counts", counts),
          None if d_losses is None else _dense("d_losses", d_losses), d_logits.data_ptr())
    return d_logits


_dtype = operator.attrgetter("dtype")
_size, _address, _device = torch.Tensor.numel, torch.Tensor.data_ptr, torch.Tensor.get_device


class _Lists:
    """The tensors of one multi-tensor call: checks a list at a time (the
    host's share of a step is these checks, so they run in map) and gathers
    the address arrays."""

    def __init__(self, numels, dev: int):
        self.numels, self.dev, self.arrays, self.written = numels, dev, {}, []

    def add(self, name: str, tensors, dtypes, numels, written: bool = True) -> torch.dtype:
        if list(map(_size, tensors)) != numels:
            raise ValueError(f"the tensors of {name} must have the sizes of the params")
        found = set(map(_dtype, tensors))
        if len(found) != 1 or not found <= dtypes:
            raise ValueError(f"{name} must all be {' or all '.join(map(str, dtypes))}, got {found}")
        if set(map(_device, tensors)) != {self.dev}:
            raise ValueError(f"every tensor must be on cuda:{self.dev}: {name}")
        if not all(map(torch.Tensor.is_contiguous, tensors)):
            raise ValueError(f"every tensor of {name} must be contiguous")
        addresses = list(map(_address, tensors))
        self.arrays[name] = (C.c_void_p * len(addresses))(*addresses)
        if written:
            self.written += addresses
        return found.pop()


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
    given = [("grads", grads), ("exp_avgs", exp_avgs), ("exp_avg_sqs", exp_avg_sqs)]
    if masters is not None:
        given.append(("masters", masters))
    for name, ts in given:
        if len(ts) != n:
            raise ValueError(f"{name} has {len(ts)} tensors, params {n}")
    if n == 0:
        return
    dev = _gpu("params", params[0])
    numels = list(map(_size, params))
    lists = _Lists(numels, dev)
    pdt = lists.add("params", params, _FLOATS, numels)
    gdt = lists.add("grads", grads, _FLOATS, numels, written=False)
    if masters is not None:
        if pdt != _BF16:
            raise ValueError("masters go with bf16 params")
        lists.add("masters", masters, {_F32}, numels)
    small = isinstance(exp_avgs[0], (tuple, list))
    blocks = [(m + 31) // 32 for m in numels] if small else None
    for name, ts in (("exp_avg", exp_avgs), ("exp_avg_sq", exp_avg_sqs)):
        if small:
            try:
                codes, scales = zip(*ts)
            except (TypeError, ValueError):
                raise ValueError(f"{name}s must be pairs (codes, scale)") from None
            lists.add(name + "s", codes, _CODES, numels)
            lists.add(name + "_scales", scales, _SCALES, blocks)
        else:
            lists.add(name + "s", ts, {_F32}, numels)
    if len(set(lists.written)) != len(lists.written):  # (empty tensors have no address: all 0)
        where = [a for a in lists.written if a]
        if len(set(where)) != len(where):
            raise ValueError("a tensor that the step writes is given twice")
    if grad_scale is not None:
        _check("grad_scale", grad_scale, dev, (_F32,))
        if grad_scale.numel() != 1:
            raise ValueError("grad_scale must have one element")
    a = _lib.MokAdamW(C.sizeof(_lib.MokAdamW), n)
    a.lr, (a.beta1, a.beta2), a.eps, a.weight_decay, a.step = lr, betas, eps, weight_decay, step
    a.param_fp32, a.grad_fp32, a.state_bits = pdt == _F32, gdt == _F32, 8 if small else 32
    a.seed = (step if seed is None else seed) & 0xFFFFFFFF
    a.grad_scale = None if grad_scale is None else grad_scale.data_ptr()
    lists.arrays["numels"] = (C.c_int64 * n)(*numels)
    for name, array in lists.arrays.items():
        setattr(a, name, C.addressof(array))
    _call("mok_adamw_step", dev, C.byref(a))
