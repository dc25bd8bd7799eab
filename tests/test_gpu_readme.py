"""The README's programs, as they stand there: each runs after those before it, and no layer runs on weights that
nobody set."""
import os
import re

import pytest

from mokutil import ROOT

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def blocks():
    with open(os.path.join(ROOT, "README.md")) as f:
        return re.findall(r"```python\n(.*?)```", f.read(), re.S)


def test_the_programs_run():
    T, H, I, E, k = 64, 2048, 768, 128, 8
    gen = torch.Generator(device="cuda").manual_seed(1)

    def normal(*shape, std=1.0):
        return (torch.randn(shape, generator=gen, device="cuda") * std).to(torch.bfloat16)

    top, ids = torch.softmax(torch.randn(T, E, generator=gen, device="cuda"), 1).topk(k)
    env = dict(x=normal(T, H).requires_grad_(), residual=normal(T, H), router_w=top, top_ids=ids,
               shared_gate=normal(I, H, std=0.02), shared_up=normal(I, H, std=0.02),
               shared_down=normal(H, I, std=0.02), loss_of=lambda t: t.float().square().mean())
    found = blocks()
    assert len(found) == 4
    for code in found[:2]:
        exec(code, env)
    # (as they are drawn; the optimizer's step moves none of them by more than its rate, 1e-4)
    for p in env["experts"].parameters():
        assert 0.019 < p.detach()[:4].float().std() < 0.021
    env["y"] = env["y"].detach().requires_grad_()
    exec(found[2], env)
    for name in ("up", "down"):
        w = env[name].weight.detach()
        assert 0.0199 < w.float().std() < 0.0201 and w.float().abs().max() < 0.02 * 8
    assert env["rows"].shape == (T * k, H) and torch.isfinite(env["rows"]).all()
    env["rows"].sum().backward()
    env["weights"] = {n: getattr(env["experts"], n + "_weights").detach()
                      for n in ("routed_gate", "routed_up", "routed_down")}
    env["x"] = normal(T, H)
    env["router_w"] = env["router_w"].detach()
    exec(found[3], env)
    assert env["out"].shape == (T, H) and torch.isfinite(env["out"]).all()
