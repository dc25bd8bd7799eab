"""More refusals on the CPU: tensors of another GPU in a forward on codes, and
the options of an optimizer's groups."""
import pytest

from mokutil import ROOT  # noqa: F401

torch = pytest.importorskip("torch")
import mixture_experts_layer_build_amd as mok  # noqa: E402
from mixture_experts_layer_build_amd.optim import MoKAdamW  # noqa: E402


class On:
    """A tensor that says it is on GPU `index` (what the checks ask)."""

    def __init__(self, t, index):
        self.t, self.index, self.device = t, index, f"cuda:{index}"

    def get_device(self):
        return self.index

    def __getattr__(self, name):
        return getattr(self.t, name)


def test_forward_mxfp8_refuses_a_context_or_weights_of_another_gpu():
    class Ws:  # (what the checks read of a workspace)
        cfg = mok.MoKConfig(hidden=64, intermediate=128, num_experts=4, topk=2, max_tokens=8)
        device, handle = 0, None

    def call(context=0, weight=0):
        u8 = lambda *s: On(torch.zeros(*s, dtype=torch.uint8), 0)  # noqa: E731
        return mok.forward_mxfp8(Ws, u8(16), u8(4, 64), u8(4, 2), On(torch.zeros(4, 2), 0),
                                 {"routed_gate": On(torch.zeros(1), weight), "shared_gate": None},
                                 out=On(torch.zeros(4, 64, dtype=torch.bfloat16), 0), context=On(torch.zeros(4), context))
    for kw in (dict(context=1), dict(weight=1)):
        with pytest.raises(ValueError, match="workspace's GPU 0, got cuda:1"):
            call(**kw)
    with pytest.raises(ValueError, match="must live on the GPU"):  # (the next check, on the tensors behind)
        call()


def test_optimizer_checks_each_group():
    p, q = torch.nn.Parameter(torch.zeros(4)), torch.nn.Parameter(torch.zeros(4))
    for bad in (dict(state_bits=16), dict(lr=-1.0), dict(betas=(0.9, 1.0)), dict(eps=-1.0), dict(weight_decay=-0.1)):
        with pytest.raises(ValueError):
            MoKAdamW([{"params": [p], **bad}])
        opt = MoKAdamW([p])
        with pytest.raises(ValueError):
            opt.add_param_group({"params": [q], **bad})
        assert len(opt.param_groups) == 1
    opt.add_param_group({"params": [q], "state_bits": 8, "lr": 0.5})
    assert opt.param_groups[1]["state_bits"] == 8 and opt.param_groups[1]["eps"] == 1e-8
