"""AdamW over the library's multi-tensor step, as a torch optimizer.

Every parameter of one type is updated by one kernel launch per 48 tensors
(``ops.adamw_step``). The moments are kept in fp32, or in 8 bits (E4M3 codes
with one scale per 32 elements: about a quarter of the memory). bf16
parameters get an fp32 master by default: an update smaller than half a bf16
step would otherwise be lost. The master is taken from the parameter at its
first step; a parameter changed by others afterwards (a checkpoint loaded into
the model alone) is written from the master again at the next one, so load the
optimizer's state with the model's, or delete the parameter's state.
"""
from __future__ import annotations

import torch

from . import ops

__all__ = ["MoKAdamW"]


class MoKAdamW(torch.optim.Optimizer):
    """AdamW with decoupled weight decay. Parameters: dense bf16 or fp32 GPU
    tensors. ``state_bits``: 32 or 8. ``master_weights``: fp32 masters of
    bf16 parameters. ``step(grad_scale=t)`` multiplies every gradient by the
    one-element fp32 GPU tensor t (a clipping factor, an inverse loss scale),
    read on the GPU. The step number and the learning rate are values of the
    launch, so ``step`` refuses to be captured into a graph, which would
    repeat them."""

    def __init__(self, params, lr: float = 1e-3, betas: tuple[float, float] = (0.9, 0.999), eps: float = 1e-8,
                 weight_decay: float = 0.01, state_bits: int = 32, master_weights: bool = True):
        defaults = dict(lr=lr, betas=tuple(betas), eps=eps, weight_decay=weight_decay, state_bits=state_bits,
                        master_weights=master_weights)
        self._check_group(defaults)
        super().__init__(params, defaults)

    @staticmethod
    def _check_group(g: dict) -> None:
        if g["state_bits"] not in (32, 8):
            raise ValueError("state_bits must be 32 or 8")
        if g["lr"] < 0 or g["eps"] < 0 or g["weight_decay"] < 0 or not all(0 <= b < 1 for b in g["betas"]):
            raise ValueError("lr, eps and weight_decay must not be negative, betas must lie in [0, 1)")

    def add_param_group(self, param_group: dict) -> None:
        self._check_group({**self.defaults, **param_group})
        super().add_param_group(param_group)

    def _init_state(self, p: torch.Tensor, group: dict) -> dict:
        if p.dtype not in (torch.bfloat16, torch.float32):
            raise ValueError(f"parameters must be bf16 or fp32, got {p.dtype}")
        if not p.is_contiguous():
            raise ValueError("parameters must be contiguous")
        st = {"step": 0}
        if group["state_bits"] == 8:
            for name in ("exp_avg", "exp_avg_sq"):
                st[name] = torch.zeros(p.shape, dtype=torch.uint8, device=p.device)
                st[name + "_scale"] = torch.zeros((p.numel() + 31) // 32, dtype=torch.uint8, device=p.device)
        else:
            for name in ("exp_avg", "exp_avg_sq"):
                st[name] = torch.zeros(p.shape, dtype=torch.float32, device=p.device)
        if group["master_weights"] and p.dtype == torch.bfloat16:
            st["master"] = p.detach().float()
        return st

    @torch.no_grad()
    def step(self, closure=None, grad_scale: torch.Tensor | None = None):
        loss = None
        if closure is not None:
            with torch.enable_grad():
                loss = closure()
        if torch.cuda.is_available() and torch.cuda.is_current_stream_capturing():
            raise RuntimeError("MoKAdamW.step cannot be captured: a graph would repeat one step number")
        call = 0
        for group in self.param_groups:
            small = group["state_bits"] == 8
            kinds: dict = {}  # tensors of one call: same types, device and step number
            for p in group["params"]:
                if p.grad is None:
                    continue
                if p.grad.is_sparse:
                    raise ValueError("gradients must be dense")
                st = self.state[p]
                if not st:
                    st.update(self._init_state(p, group))
                key = (p.device, p.dtype, p.grad.dtype, "master" in st, st["step"] + 1)
                kinds.setdefault(key, []).append((p, p.grad.contiguous(), st))
            for (_, _, _, master, step), items in kinds.items():
                states = [st for _, _, st in items]
                moments = [[(st[n], st[n + "_scale"]) if small else st[n] for st in states]
                           for n in ("exp_avg", "exp_avg_sq")]
                ops.adamw_step([p for p, _, _ in items], [g for _, g, _ in items], *moments,
                               masters=[st["master"] for st in states] if master else None, step=step,
                               lr=float(group["lr"]), betas=group["betas"], eps=group["eps"],
                               weight_decay=group["weight_decay"], grad_scale=grad_scale,
                               seed=step * 0xD1B54A35 + call * 0x85EBCA77)
                for st in states:  # (only now: a refused call leaves its tensors and their step as they were)
                    st["step"] = step
                call += 1
        return loss

    def load_state_dict(self, state_dict) -> None:
        """The base class turns every state tensor into the parameter's type;
        here the moments, scales and masters keep their own."""
        super().load_state_dict(state_dict)
        saved = [i for g in state_dict["param_groups"] for i in g["params"]]
        mine = [p for g in self.param_groups for p in g["params"]]
        for i, p in zip(saved, mine):
            for name, value in state_dict["state"].get(i, {}).items():
                if isinstance(value, torch.Tensor):
                    value = value.detach().to(device=p.device, copy=True)
                self.state[p][name] = value
