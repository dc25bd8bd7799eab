"""Tensors handed to a call that overlap what it writes: refused where other
workgroups would read what one has written, taken where a call may run in
place."""
import pytest

from mokutil import ROOT  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import mixture_experts_layer_build_amd as mok  # noqa: E402

BF = torch.bfloat16


def test_a_step_refuses_a_grad_scale_among_what_it_writes():
    p, g, m, v = (torch.ones(64, device="cuda") for _ in range(4))
    for written in (p, m, v):
        with pytest.raises(ValueError, match="overlaps"):
            mok.adamw_step([p], [g], [m], [v], step=1, lr=1e-3, grad_scale=written[5:6])
    assert (p == 1).all()
    mok.adamw_step([p], [g], [m], [v], step=1, lr=1e-3, grad_scale=g[5:6])  # only read
    assert (p != 1).all()
