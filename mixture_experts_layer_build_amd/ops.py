"""The operators around the layer: RMS norm, top-k router, AdamW step, and the
experts' products outside it: grouped by expert, and with 4-bit weights.

Direct calls over the C ABI (``include/mok.h`` states formulas, types and
refusals); the package re-exports them. They allocate their outputs with
torch, enqueue on the current stream of the tensors' device, and need no
workspace. Tensors on the CPU are rejected: there is no fallback. What a call
writes into tensors that it was given (``adamw_step``; the outputs handed to a
norm, a product or the 4-bit layer) moves their in-place version counters.

The checks and allocations of these calls are compiled (``csrc/py_ops.cpp``,
built with the library): at a few tokens the host's share decides their time.
"""
from __future__ import annotations

import ctypes as C

import torch

from . import _lib

__all__ = ["rms_norm", "rms_norm_mxfp8", "rms_norm_backward", "router_topk", "router_topk_backward", "adamw_step",
           "grouped_matmul", "grouped_matmul_backward", "w4_quantize", "w4_dequantize", "w4_matmul", "forward_w4"]

_SCORING = {"softmax": _lib.MOK_ROUTER_SOFTMAX, "sigmoid": _lib.MOK_ROUTER_SIGMOID}
_BOUND = ("mok_rms_norm", "mok_rms_norm_scratch_bytes", "mok_rms_norm_backward", "mok_router_scratch_bytes",
          "mok_router_topk", "mok_router_topk_backward", "mok_adamw_step",
          "mok_grouped_matmul_scratch_bytes", "mok_grouped_matmul", "mok_grouped_matmul_dx", "mok_grouped_matmul_dw", "mok_w4_quantize", "mok_w4_dequantize", "mok_w4_matmul",
          "mok_forward_w4_scratch_bytes", "mok_forward_w4")

_host = None


def _load():
    """The compiled host side, bound to the library's functions. Raises if
    either has not been built."""
    global _host
    lib = _lib.load()
    try:
        from . import _ops
    except ImportError as e:
        raise RuntimeError("the host module _ops.so is missing or does not load: build it with "
                           f"`python -m mixture_experts_layer_build_amd.build` ({e})") from e
    _ops.bind(*[C.cast(getattr(lib, n), C.c_void_p).value for n in _BOUND])
    _host = _ops
    return _ops


def _call(name: str, first: torch.Tensor, *args):
    """One call on the GPU of `first` and its current stream."""
    f = getattr(_host or _load(), name)
    try:
        index = first.get_device()
    except AttributeError:
        index = -1
    if index < 0:  # no tensor, or not on a GPU: the call refuses it
        out = f(*args, 0)
    elif index == torch._C._cuda_getDevice():
        out = f(*args, torch._C._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(index):
            out = f(*args, torch._C._cuda_getCurrentRawStream(index))
    if type(out) is int and out != _lib.MOK_OK:
        raise _lib.MokError("mok_" + name, out)
    return out


def rms_norm(x: torch.Tensor, weight: torch.Tensor, residual: torch.Tensor | None = None, eps: float = 1e-6):
    """y = rms_norm(x + residual) * weight in bf16. Returns (y, sum, rstd):
    sum = x + residual in the residual's type (None without a residual), rstd
    fp32 with one value per row. x bf16 or fp32 [..., cols]."""
    return _call("rms_norm", x, x, weight, residual, eps)


def rms_norm_mxfp8(x: torch.Tensor, weight: torch.Tensor, residual: torch.Tensor | None = None, eps: float = 1e-6,
                   y: torch.Tensor | None = None, rstd: torch.Tensor | None = None):
    """The norm with its output in MXFP8, as ``forward_mxfp8`` takes it.
    Returns (codes uint8 [..., cols], scale uint8 [..., cols/32], sum). Give
    ``y`` (bf16, x's shape) and ``rstd`` (fp32, one per row) to have them
    filled too, for a backward. y may be x's or the residual's own tensor
    (dense, bf16); else they overlap no other tensor of the call."""
    return _call("rms_norm_mxfp8", x, x, weight, residual, eps, y, rstd)


def rms_norm_backward(dy: torch.Tensor, s: torch.Tensor, rstd: torch.Tensor, weight: torch.Tensor,
                      d_sum: torch.Tensor | None = None, dx: torch.Tensor | None = None):
    """(ds, d_weight) from dy (bf16), the saved s (the forward's sum, or x
    without a residual) and rstd; ``d_sum`` is the gradient that arrives
    through the sum. ds is the gradient of x and of the residual, in s's
    type; ``dx`` (bf16) receives it in bf16 as well, and may be a dense bf16
    dy, s or d_sum itself, but overlaps no other tensor of the call."""
    return _call("rms_norm_backward", dy, dy, s, rstd, weight, d_sum, dx)


def _scoring(name: str) -> int:
    if name not in _SCORING:
        raise ValueError(f"scoring must be one of {sorted(_SCORING)}, got {name!r}")
    return _SCORING[name]


def router_topk(logits: torch.Tensor, k: int, *, scoring: str = "softmax", renormalize: bool = True,
                scale: float = 1.0, bias: torch.Tensor | None = None, token_mask: torch.Tensor | None = None,
                losses: bool = False):
    """Top-k routing of logits [T, E] (bf16 or fp32): (weights fp32 [T, k],
    ids int64 [T, k]), the layer's router_weights and top_experts. With
    ``losses`` also (counts int32 [E + 1], losses fp32 [2]): choices per
    expert and the number of live tokens; the load-balance and the z loss."""
    out = _call("router_topk", logits, logits, k, _scoring(scoring), bool(renormalize), scale, bias, token_mask,
                bool(losses))
    return out if losses else out[:2]


def router_topk_backward(d_weights: torch.Tensor, logits: torch.Tensor, ids: torch.Tensor, *,
                         scoring: str = "softmax", renormalize: bool = True, scale: float = 1.0,
                         bias: torch.Tensor | None = None, token_mask: torch.Tensor | None = None,
                         counts: torch.Tensor | None = None, d_losses: torch.Tensor | None = None) -> torch.Tensor:
    """Gradient to the logits [T, E] in their type, from d_weights (fp32)
    and the forward's ids; ``counts`` and ``d_losses`` (fp32 [2]) where the
    losses have a gradient. The other arguments as in the forward."""
    return _call("router_topk_backward", logits, d_weights, logits, ids, _scoring(scoring), bool(renormalize), scale,
                 bias, token_mask, counts, d_losses)[0]


def adamw_step(params, grads, exp_avgs, exp_avg_sqs, masters=None, *, step: int, lr: float,
               betas: tuple[float, float] = (0.9, 0.999), eps: float = 1e-8, weight_decay: float = 0.0,
               grad_scale: torch.Tensor | None = None, seed: int | None = None) -> None:
    """One AdamW step of many tensors, in place. Lists of equal length: params
    (all bf16 or all fp32), grads (all bf16 or all fp32), the moments, and for
    bf16 params optionally their fp32 masters. Moments are fp32 tensors, or
    for 8-bit states pairs (codes, scale): E4M3 codes [numel] of m (of
    sqrt(v)) and E8M0 scales [ceil(numel/32)], zeros at the start. grad_scale:
    a device fp32 tensor of one element that multiplies every gradient. seed
    (default: the step) chooses the 8-bit states' roundings. What the step
    writes may overlap no other tensor of the call."""
    if len(params) == 0 and not (len(grads) or len(exp_avgs) or len(exp_avg_sqs) or masters):
        return
    if len(params) == 0:
        raise ValueError("there are no params, but other tensors")
    _call("adamw_step", params[0], params, grads, exp_avgs, exp_avg_sqs, masters, step, lr, betas[0], betas[1], eps,
          weight_decay, grad_scale, step if seed is None else seed)


def grouped_matmul(x: torch.Tensor, weight: torch.Tensor, offsets: torch.Tensor,
                   out: torch.Tensor | None = None) -> torch.Tensor:
    """Matrix product grouped by expert: y[r] = weight[e] @ x[r] for the rows
    offsets[e] <= r < offsets[e + 1]. x bf16 [rows, k] (dense rows), weight bf16
    [experts, n, k], offsets int32 or int64 [experts + 1], not decreasing.
    Returns y bf16 [rows, n]; rows of no expert get zeros, or are left as they
    were in a given ``out``, which overlaps no other tensor of the call."""
    return _call("grouped_matmul", x, x, weight, offsets, out)[0]


def grouped_matmul_backward(dy: torch.Tensor, x: torch.Tensor, weight: torch.Tensor, offsets: torch.Tensor, *,
                            need_dx: bool = True, need_dw: bool = True, dw_dtype: torch.dtype = torch.bfloat16):
    """(dx bf16 [rows, k], dweight [experts, n, k]) from dy bf16 [rows, n];
    None for one that is not needed. Rows of no expert get zeros in dx and
    count in no dweight; an expert without rows gets zeros. ``dw_dtype``: bf16
    or fp32."""
    if dw_dtype not in (torch.bfloat16, torch.float32):
        raise ValueError(f"dw_dtype must be bfloat16 or float32, got {dw_dtype}")
    return _call("grouped_matmul_backward", dy, dy, x, weight, offsets, bool(need_dx), bool(need_dw),
                 dw_dtype == torch.float32)


_W4_FORMATS = {"int4": False, "mxfp4": True}


def w4_quantize(weight: torch.Tensor, format: str = "int4", group: int | None = None, zero_point: bool = False):
    """A weight [..., k] (bf16 or fp32) in 4 bits: (codes uint8 [..., k/2],
    scale [..., k/group], zero). "int4": groups of 32, 64 or 128 (the default)
    along k, scale bf16, and with ``zero_point`` zero uint8 (else None, and the
    zero point is 8). "mxfp4": groups of 32, scale uint8 (E8M0), zero None."""
    if format not in _W4_FORMATS:
        raise ValueError(f"format must be one of {sorted(_W4_FORMATS)}, got {format!r}")
    mx = _W4_FORMATS[format]
    return _call("w4_quantize", weight, weight, mx, (32 if mx else 128) if group is None else group, bool(zero_point))


def w4_dequantize(codes: torch.Tensor, scale: torch.Tensor, zero: torch.Tensor | None = None) -> torch.Tensor:
    """The values of a 4-bit weight in bf16 [..., k], as ``forward`` and
    ``grouped_matmul`` take them (for a prompt). The scale's type tells the
    format."""
    return _call("w4_dequantize", codes, codes, scale, zero)[0]


def w4_matmul(x: torch.Tensor, codes: torch.Tensor, scale: torch.Tensor,
              zero: torch.Tensor | None = None) -> torch.Tensor:
    """y bf16 [..., n] = x bf16 [..., k] times a 4-bit weight [n, k],
    transposed. Made for few rows of x (decoding): from about 400 on (200 for a
    weight of 200 M), ``x @ w4_dequantize(...).t()`` is faster."""
    return _call("w4_matmul", x, x, codes, scale, zero)[0]


_W4_PARTS = tuple(kind + name + end for kind in ("routed_", "shared_") for name in ("gate", "up", "down")
                  for end in ("", "_scale", "_zero"))


def forward_w4(x: torch.Tensor, router_weights: torch.Tensor, top_experts: torch.Tensor, weights: dict,
               swiglu_limit: float = 0.0, out: torch.Tensor | None = None) -> torch.Tensor:
    """The layer's forward for few tokens on 4-bit experts: out bf16 [T, H]
    from x bf16 [T, H], the router's weights fp32 [T, k] and ids int64 [T, k]
    (an id outside the experts is no choice). ``weights``: routed_gate/up
    [E, I, H/2], routed_down [E, H, I/2] and optionally shared_* as
    ``w4_quantize`` gives their codes, with *_scale (and *_zero) entries, all of
    one format and group. ``swiglu_limit`` as in ``MoKConfig``: 0 or inf for
    none. Needs no schedule and no workspace; T * k <= 8192. From some hundred
    tokens on (128 experts of 768 x 2048: 400; 32 of 2048 x 7168: 120),
    ``forward`` on the weights' values is faster."""
    return _call("forward_w4", x, x, router_weights, top_experts, tuple(map(weights.get, _W4_PARTS)), swiglu_limit,
                 out)[0]
