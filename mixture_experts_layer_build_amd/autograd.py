"""PyTorch autograd over the C ABI: the layer as a differentiable function
and a module holding the routed experts' parameters.

This follows the integration layer of the pages ([A]
"nemo_automodel.components.moe.mok_experts": ``_MoKAutogradFunction``,
``_MoKRuntime``, ``GroupedExpertsMoK``, ``_flatten_mok_tensor_dataclass``),
read for one GPU:

- ``MoKRuntime`` owns one layer's configuration, its precision mode and the
  cached workspace of that configuration (one workspace serves every layer
  of the same shape, [R] "The two API layers and the schedule object").
- ``MoKAutogradFunction.forward`` builds the schedule, runs the fused
  forward and keeps its activation context; ``backward`` hands the same
  schedule and context to the fused backward and returns a gradient for
  every float input (none for the runtime and the integer expert ids).
- The schedule and the context are each one flat byte tensor, and both go
  through ``ctx.save_for_backward``: saved-tensor hooks (activation
  checkpointing, CPU offload) see them, and nothing else on ``ctx`` holds a
  tensor, so a layer's context lives only as long as autograd keeps it.
- In MXFP8 mode the parameters stay BF16; the forward takes them quantized
  by ``mxfp8_quantize`` along H (gate, up) and I (down), the backward
  transposed and quantized along each backward GEMM's contraction by
  ``mxfp8_quantize_transposed`` ([R] "Tuning the five hyperparameters
  before production": MXFP8 takes pre-quantized weights). Each quantized
  copy is kept per parameter and made again whenever the parameter's
  in-place version counter moves (an optimizer step, a ``copy_``), so a
  step never runs on stale codes; a captured training step makes them at
  every replay.

Around the layer: ``rms_norm`` and ``MoKRMSNorm`` (the norm in front of it,
with the residual's addition) and ``router_topk`` and ``MoKRouter`` (the
top-k router, with its load statistics and losses), differentiable in every
float input; the schedule takes their expert ids as they are. Beside it:
``grouped_matmul`` and ``MoKGroupedLinear``, the ragged product of experts for
other expert functions. (To capture a step in a graph: warm it up on a side
stream, and let no eager backward graph of the same leaves live meanwhile, as
torch asks of every captured backward.)

Every step of the layer runs in the library's HIP kernels; tensors on the
CPU are rejected.
"""
from __future__ import annotations

import dataclasses
import weakref

import torch
from torch.autograd.function import once_differentiable

from . import (MOK_MODE_BF16, MOK_MODE_MXFP8, MoKConfig, backward, build_schedule, context_bytes, forward,
               get_workspace, mxfp8_quantize, mxfp8_quantize_transposed, ops)

__all__ = ["MoKRuntime", "MoKAutogradFunction", "MoKExperts", "moe_layer", "rms_norm", "MoKRMSNorm", "router_topk",
           "MoKRouter", "grouped_matmul", "MoKGroupedLinear"]

_WEIGHT_NAMES = ("shared_gate", "shared_up", "shared_down", "routed_gate", "routed_up", "routed_down")


class MoKRuntime:
    """One layer's configuration, precision mode and SwiGLU input limit
    ([A] ``_MoKRuntime(mok_config, swiglu_limit)``; None keeps the config's
    own ``swiglu_limit``). The workspace comes from the per-(device, config)
    cache, so layers of one shape and limit share it."""

    def __init__(self, cfg: MoKConfig, mode: int = MOK_MODE_BF16, swiglu_limit: float | None = None):
        if mode not in (MOK_MODE_BF16, MOK_MODE_MXFP8):
            raise ValueError("mode must be MOK_MODE_BF16 or MOK_MODE_MXFP8")
        if swiglu_limit is not None:
            cfg = dataclasses.replace(cfg, swiglu_limit=float(swiglu_limit))
        self.cfg = cfg
        self.mode = mode
        # name -> (weak reference to the weight, its version, its address, codes, scales)
        self._q: dict = {}
        # address -> (codes, scales) that a captured graph reads: kept when the weight's are made again
        self._in_graphs: dict = {}

    def workspace(self, device: torch.device):
        if device.type != "cuda":
            raise ValueError("the MoE layer runs on the GPU only: inputs must be CUDA tensors")
        return get_workspace(self.cfg, device.index if device.index is not None else torch.cuda.current_device())

    def quantized(self, name: str, w: torch.Tensor, transposed: bool = False, trained: bool = False
                  ) -> tuple[torch.Tensor, torch.Tensor]:
        """MXFP8 codes and scales of a BF16 weight along its last dimension
        (the forward's form), or transposed and quantized along its
        second-to-last (the backward's form), made again when the weight
        changed since they were made. A graph does not ask at its replays: in
        a capture the codes of a weight in training are made in the graph,
        and what a capture made is not kept (it holds nothing before the
        first replay). A captured inference forward reads the codes that were
        kept at its capture, which then live as long as this object: capture
        again after the weights change."""
        key = (name, transposed)
        capturing = torch.cuda.is_current_stream_capturing()
        hit = self._q.get(key)
        if hit is not None and not (capturing and trained):
            ref, version, ptr, codes, sc = hit
            if ref() is w and version == w._version and ptr == w.data_ptr():
                if capturing:
                    self._in_graphs[codes.data_ptr()] = (codes, sc)
                return codes, sc
        if transposed:
            codes, sc = mxfp8_quantize_transposed(w.detach())
        else:
            codes, sc = mxfp8_quantize(w.detach().reshape(-1, w.shape[-1]), axis=1)
            codes = codes.view(w.shape)
        if not capturing:
            self._q[key] = (weakref.ref(w), w._version, w.data_ptr(), codes, sc)
        return codes, sc

    def forward_weights(self, w: dict, trained: bool = False) -> dict:
        if self.mode == MOK_MODE_BF16:
            return w
        q = {}
        for name, t in w.items():
            if t is None:
                continue
            q[name], q[name + "_scale"] = self.quantized(name, t, trained=trained and t.requires_grad)
        return q

    def backward_weights(self, w: dict) -> dict:
        """MXFP8: the weights transposed and quantized for the backward's
        GEMMs, kept like the forward's codes until the weight changes."""
        if self.mode == MOK_MODE_BF16:
            return w
        q = {}
        for name, t in w.items():
            if t is None:
                continue
            q[name], q[name + "_scale"] = self.quantized(name, t, transposed=True, trained=t.requires_grad)
        return q


def _check(name: str, t: torch.Tensor | None, dtype: torch.dtype, shape: tuple) -> None:
    if t is None:
        raise ValueError(f"{name} is required")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != shape:
        raise ValueError(f"{name} must have shape {shape}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _run_forward(runtime: MoKRuntime, keep: bool, x, router_weights, top_experts, shared_gate, shared_up,
                 shared_down, routed_gate, routed_up, routed_down):
    """Validate, build the schedule and run the fused forward; the context
    is allocated and filled only when ``keep``. Returns (out, schedule,
    context or None, weights by name)."""
    cfg = runtime.cfg
    if x is None or x.dim() != 2:
        raise ValueError("x must be a [tokens, hidden] tensor")
    T = x.shape[0]
    H, I, Is, E, k = cfg.hidden, cfg.intermediate, cfg.shared_intermediate, cfg.num_experts, cfg.topk
    _check("x", x, torch.bfloat16, (T, H))
    _check("router_weights", router_weights, torch.float32, (T, k))
    _check("top_experts", top_experts, torch.int64, (T, k))
    _check("routed_gate", routed_gate, torch.bfloat16, (E, I, H))
    _check("routed_up", routed_up, torch.bfloat16, (E, I, H))
    _check("routed_down", routed_down, torch.bfloat16, (E, H, I))
    if Is:
        _check("shared_gate", shared_gate, torch.bfloat16, (Is, H))
        _check("shared_up", shared_up, torch.bfloat16, (Is, H))
        _check("shared_down", shared_down, torch.bfloat16, (H, Is))
    elif any(t is not None for t in (shared_gate, shared_up, shared_down)):
        raise ValueError("shared expert weights given but the config has shared_intermediate = 0")
    if T > cfg.max_tokens:
        raise ValueError(f"{T} tokens exceed the config's max_tokens {cfg.max_tokens}")
    w = dict(shared_gate=shared_gate, shared_up=shared_up, shared_down=shared_down,
             routed_gate=routed_gate, routed_up=routed_up, routed_down=routed_down)
    for name, t in [("x", x), ("router_weights", router_weights), ("top_experts", top_experts)] + list(w.items()):
        if t is not None and t.device != x.device:
            raise ValueError(f"{name} is on {t.device}, x on {x.device}: every input must be on one GPU")
    ws = runtime.workspace(x.device)
    sched = build_schedule(ws, top_experts)
    context = torch.empty(context_bytes(cfg, runtime.mode), dtype=torch.uint8, device=x.device) if keep else None
    out = forward(ws, sched, x, router_weights, runtime.forward_weights(w, trained=keep), mode=runtime.mode,
                  context=context)
    return out, sched, context, w


class MoKAutogradFunction(torch.autograd.Function):
    """out = MoE layer (schedule, gathered SwiGLU experts, shared expert,
    combine), differentiable in x, router_weights and every weight."""

    @staticmethod
    def forward(ctx, runtime: MoKRuntime, x, router_weights, top_experts, shared_gate, shared_up, shared_down,
                routed_gate, routed_up, routed_down):
        keep = any(ctx.needs_input_grad[1:])
        out, sched, context, w = _run_forward(runtime, keep, x, router_weights, top_experts, shared_gate,
                                              shared_up, shared_down, routed_gate, routed_up, routed_down)
        ctx.runtime = runtime
        if keep:
            ctx.save_for_backward(sched, context, x, router_weights, *[w[n] for n in _WEIGHT_NAMES])
        return out

    @staticmethod
    def backward(ctx, grad_out):
        runtime = ctx.runtime
        sched, context, x, router_weights, *wl = ctx.saved_tensors
        w = dict(zip(_WEIGHT_NAMES, wl))
        if grad_out.dtype != torch.bfloat16:
            grad_out = grad_out.to(torch.bfloat16)
        grad_out = grad_out.contiguous()
        ws = runtime.workspace(x.device)
        g = backward(ws, sched, context, grad_out, x, router_weights, runtime.backward_weights(w), mode=runtime.mode)
        need = ctx.needs_input_grad

        def pick(i, name):
            return g.get(name) if need[i] else None

        return (None, pick(1, "dx"), pick(2, "d_router_weights"), None,
                pick(4, "d_shared_gate"), pick(5, "d_shared_up"), pick(6, "d_shared_down"),
                pick(7, "d_routed_gate"), pick(8, "d_routed_up"), pick(9, "d_routed_down"))


def moe_layer(runtime: MoKRuntime, x, router_weights, top_experts, shared_gate, shared_up, shared_down,
              routed_gate, routed_up, routed_down) -> torch.Tensor:
    """Functional form of the differentiable layer (argument order of [A]
    ``_MoKAutogradFunction.forward``). When no gradient is wanted (grad mode
    off, or no input requires one) the forward runs without keeping a
    context."""
    args = (x, router_weights, top_experts, shared_gate, shared_up, shared_down, routed_gate, routed_up,
            routed_down)
    if torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in args):
        return MoKAutogradFunction.apply(runtime, *args)
    with torch.no_grad():
        return _run_forward(runtime, False, *args)[0]


class MoKExperts(torch.nn.Module):
    """Routed expert parameters in the library's native layouts (gate and
    up [E, I, H], down [E, H, I], bf16), run by the fused layer. As in [A]
    ``GroupedExpertsMoK``, the router stays outside: forward takes the
    router's weights and expert ids, plus the shared expert's weights, and
    there is no expert bias."""

    def __init__(self, hidden: int, intermediate: int, num_experts: int, topk: int, max_tokens: int,
                 shared_intermediate: int = 0, capacity_multiplier: float = 1.0, expert_pad: int = 32,
                 mode: int = MOK_MODE_BF16, device=None):
        super().__init__()
        self.runtime = MoKRuntime(MoKConfig(hidden=hidden, intermediate=intermediate, num_experts=num_experts,
                                            topk=topk, max_tokens=max_tokens,
                                            shared_intermediate=shared_intermediate,
                                            capacity_multiplier=capacity_multiplier, expert_pad=expert_pad), mode)
        bf = dict(dtype=torch.bfloat16, device=device)
        self.routed_gate_weights = torch.nn.Parameter(torch.empty(num_experts, intermediate, hidden, **bf))
        self.routed_up_weights = torch.nn.Parameter(torch.empty(num_experts, intermediate, hidden, **bf))
        self.routed_down_weights = torch.nn.Parameter(torch.empty(num_experts, hidden, intermediate, **bf))

    @torch.no_grad()
    def init_weights(self, init_std: float = 0.02, generator: torch.Generator | None = None) -> None:
        """Normal(0, init_std) draws, rounded to bf16."""
        for p in (self.routed_gate_weights, self.routed_up_weights, self.routed_down_weights):
            p.copy_(torch.randn(p.shape, generator=generator, dtype=torch.float32).mul_(init_std))

    def forward(self, x, weights, indices, shared_gate_weights=None, shared_up_weights=None,
                shared_down_weights=None) -> torch.Tensor:
        """x bf16 [T, H], weights fp32 [T, k], indices int64 [T, k] -> bf16
        [T, H]: the routed experts' weighted SwiGLU outputs plus the shared
        expert's."""
        return moe_layer(self.runtime, x, weights, indices, shared_gate_weights, shared_up_weights,
                         shared_down_weights, self.routed_gate_weights, self.routed_up_weights,
                         self.routed_down_weights)

    def extra_repr(self) -> str:
        c = self.runtime.cfg
        mode = "mxfp8" if self.runtime.mode == MOK_MODE_MXFP8 else "bf16"
        return (f"hidden={c.hidden}, intermediate={c.intermediate}, experts={c.num_experts}, topk={c.topk}, "
                f"shared_intermediate={c.shared_intermediate}, max_tokens={c.max_tokens}, mode={mode}")



class RMSNormFunction(torch.autograd.Function):
    """(y, sum) of the RMS norm with the residual's addition; sum is None
    without a residual. Keeps the sum (or x) and one fp32 per row."""

    @staticmethod
    def forward(ctx, x, weight, residual, eps):
        y, total, rstd = ops.rms_norm(x, weight, residual, eps)
        ctx.save_for_backward(x if total is None else total, rstd, weight)
        ctx.x_dtype = x.dtype
        ctx.set_materialize_grads(False)
        return y, total

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, d_sum):
        s, rstd, weight = ctx.saved_tensors
        need_x, need_w, need_r = ctx.needs_input_grad[:3]
        if d_sum is not None:
            d_sum = d_sum.contiguous()
        if dy is None:  # only the sum was used
            dw = torch.zeros_like(weight) if need_w else None
            dx = d_sum.to(ctx.x_dtype) if need_x and d_sum is not None else None
            return dx, dw, d_sum if need_r else None, None
        narrow = torch.empty(s.shape, dtype=ctx.x_dtype, device=s.device) if ctx.x_dtype != s.dtype else None
        ds, dw = ops.rms_norm_backward(dy.contiguous(), s, rstd, weight, d_sum, dx=narrow)
        dx = ds if narrow is None else narrow
        return dx if need_x else None, dw if need_w else None, ds if need_r else None, None


def rms_norm(x: torch.Tensor, weight: torch.Tensor, residual: torch.Tensor | None = None, eps: float = 1e-6):
    """Differentiable ``ops.rms_norm``: (y, sum) with y bf16 and sum = x +
    residual in the residual's type (None without a residual)."""
    return RMSNormFunction.apply(x, weight, residual, eps)


class MoKRMSNorm(torch.nn.Module):
    """The norm in front of the layer: forward(x, residual) -> (y, sum)."""

    def __init__(self, hidden: int, eps: float = 1e-6, dtype: torch.dtype = torch.bfloat16, device=None):
        super().__init__()
        self.eps = eps
        self.weight = torch.nn.Parameter(torch.ones(hidden, dtype=dtype, device=device))

    def forward(self, x, residual=None):
        return rms_norm(x, self.weight, residual, self.eps)

    def extra_repr(self) -> str:
        return f"hidden={self.weight.shape[0]}, eps={self.eps}"


class RouterFunction(torch.autograd.Function):
    """(weights, ids, counts, losses) of the top-k router, differentiable in
    the logits through weights and losses (counts and losses None unless
    asked for)."""

    @staticmethod
    def forward(ctx, logits, k, how, want_losses):
        out = ops.router_topk(logits, k, losses=want_losses, **how)
        weights, ids = out[:2]
        counts, losses = out[2:] if want_losses else (None, None)
        ctx.how = {n: v for n, v in how.items() if not isinstance(v, torch.Tensor)}
        ctx.tensors = [n for n, v in how.items() if isinstance(v, torch.Tensor)]
        ctx.save_for_backward(logits, ids, counts, *[how[n] for n in ctx.tensors])
        ctx.mark_non_differentiable(*[t for t in (ids, counts) if t is not None])
        ctx.set_materialize_grads(False)
        return weights, ids, counts, losses

    @staticmethod
    @once_differentiable
    def backward(ctx, d_weights, _ids, _counts, d_losses):
        logits, ids, counts, *rest = ctx.saved_tensors
        if d_weights is None and d_losses is None:
            return None, None, None, None
        if d_weights is None:
            d_weights = torch.zeros(ids.shape, dtype=torch.float32, device=ids.device)
        dl = ops.router_topk_backward(d_weights.contiguous(), logits, ids, **ctx.how, **dict(zip(ctx.tensors, rest)),
                                      counts=counts if d_losses is not None else None,
                                      d_losses=None if d_losses is None else d_losses.contiguous())
        return dl, None, None, None


def router_topk(logits: torch.Tensor, k: int, *, scoring: str = "softmax", renormalize: bool = True,
                scale: float = 1.0, bias: torch.Tensor | None = None, token_mask: torch.Tensor | None = None,
                losses: bool = False):
    """Differentiable ``ops.router_topk``: (weights, ids), and with
    ``losses`` also (counts, losses). ``bias`` only selects: it gets no
    gradient."""
    how = dict(scoring=scoring, renormalize=renormalize, scale=scale,
               bias=None if bias is None else bias.detach(), token_mask=token_mask)
    out = RouterFunction.apply(logits, k, how, losses)
    return out if losses else out[:2]


class MoKRouter(torch.nn.Module):
    """Router of the layer: logits = x W^T in fp32 (a library product), then
    ``router_topk``. forward(x [T, H], token_mask) -> (weights fp32 [T, k],
    ids int64 [T, k]), and with ``losses`` also (counts, losses). With
    ``selection_bias`` the module keeps an fp32 buffer that shifts the choice
    alone, for balancing without a loss: move it by the counts, after the
    backward pass (which reads it, so autograd refuses an earlier change)."""

    def __init__(self, hidden: int, num_experts: int, topk: int, scoring: str = "softmax", renormalize: bool = True,
                 scale: float = 1.0, selection_bias: bool = False, losses: bool = False, device=None):
        super().__init__()
        self.topk, self.scoring, self.renormalize, self.scale, self.losses = topk, scoring, renormalize, scale, losses
        self.weight = torch.nn.Parameter(torch.zeros(num_experts, hidden, dtype=torch.float32, device=device))
        bias = torch.zeros(num_experts, dtype=torch.float32, device=device) if selection_bias else None
        self.register_buffer("bias", bias)

    @torch.no_grad()
    def init_weights(self, init_std: float = 0.02, generator: torch.Generator | None = None) -> None:
        self.weight.copy_(torch.randn(self.weight.shape, generator=generator, dtype=torch.float32).mul_(init_std))

    def forward(self, x, token_mask=None):
        with torch.autocast(x.device.type, enabled=False):  # (it would make the product bf16)
            logits = torch.nn.functional.linear(x.float(), self.weight.float())
        bias = None if self.bias is None else self.bias.float()
        return router_topk(logits, self.topk, scoring=self.scoring, renormalize=self.renormalize, scale=self.scale,
                           bias=bias, token_mask=token_mask, losses=self.losses)

    def extra_repr(self) -> str:
        return (f"hidden={self.weight.shape[1]}, experts={self.weight.shape[0]}, topk={self.topk}, "
                f"scoring={self.scoring}, renormalize={self.renormalize}, scale={self.scale}")


class GroupedMatmulFunction(torch.autograd.Function):
    """The grouped product, differentiable in x and the weight. (The weight's
    gradient is bf16: autograd casts a gradient to its leaf's type. fp32 ones
    come from ``ops.grouped_matmul_backward(..., dw_dtype=torch.float32)``.)"""

    @staticmethod
    def forward(ctx, x, weight, offsets):
        ctx.save_for_backward(x, weight, offsets)
        return ops.grouped_matmul(x, weight, offsets)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, weight, offsets = ctx.saved_tensors
        need_x, need_w = ctx.needs_input_grad[:2]
        dx, dw = ops.grouped_matmul_backward(dy.contiguous(), x, weight, offsets, need_dx=need_x, need_dw=need_w)
        return dx, dw, None


def grouped_matmul(x: torch.Tensor, weight: torch.Tensor, offsets: torch.Tensor) -> torch.Tensor:
    """Differentiable ``ops.grouped_matmul``: y[r] = weight[e] @ x[r] for the
    rows of expert e, zeros for rows of none."""
    return GroupedMatmulFunction.apply(x, weight, offsets)


class MoKGroupedLinear(torch.nn.Module):
    """A linear map per expert (bf16 [experts, out, in], no bias), for expert
    functions other than the layer's: forward(x [rows, in], offsets [experts +
    1]) -> [rows, out], the rows sorted by expert."""

    def __init__(self, num_experts: int, in_features: int, out_features: int, device=None):
        super().__init__()
        self.weight = torch.nn.Parameter(
            torch.empty(num_experts, out_features, in_features, dtype=torch.bfloat16, device=device))

    @torch.no_grad()
    def init_weights(self, init_std: float = 0.02, generator: torch.Generator | None = None) -> None:
        """Normal(0, init_std) draws, rounded to bf16."""
        self.weight.copy_(torch.randn(self.weight.shape, generator=generator, dtype=torch.float32).mul_(init_std))

    def forward(self, x, offsets):
        return grouped_matmul(x, self.weight, offsets)

    def extra_repr(self) -> str:
        e, n, k = self.weight.shape
        return f"experts={e}, in_features={k}, out_features={n}"
