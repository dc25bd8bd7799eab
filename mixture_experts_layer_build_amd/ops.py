"""The operators around the layer: RMS norm, top-k router, AdamW step.

Direct calls over the C ABI (``include/mok.h`` states formulas, types and
refusals); the package re-exports them. They allocate their outputs with
torch, enqueue on the current stream of the tensors' device, and need no
workspace. Tensors on the CPU are rejected: there is no fallback. What a call
writes into tensors that it was given (``adamw_step``; the outputs handed to a
norm) moves their in-place version counters.

The checks and allocations of these calls are compiled (``csrc/py_ops.cpp``,
built with the library): at a few tokens the host's share decides their time.
"""
from __future__ import annotations

import ctypes as C

import torch

from . import _lib

__all__ = ["rms_norm", "rms_norm_mxfp8", "rms_norm_backward", "router_topk", "router_topk_backward", "adamw_step"]

_SCORING = {"softmax": _lib.MOK_ROUTER_SOFTMAX, "sigmoid": _lib.MOK_ROUTER_SIGMOID}
_BOUND = ("mok_rms_norm", "mok_rms_norm_scratch_bytes", "mok_rms_norm_backward", "mok_router_scratch_bytes",
          "mok_router_topk", "mok_router_topk_backward", "mok_adamw_step")

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
