"""The MXFP8 layer in captured graphs: codes of trained weights are made in
the graph, so a replay after an optimizer's step runs on the new weights, and
codes whose making was only captured are not taken by eager calls."""
import pytest

from mokutil import ROOT  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import mixture_experts_layer_build_amd as mok  # noqa: E402
from mixture_experts_layer_build_amd.autograd import MoKRuntime, moe_layer  # noqa: E402
from mixture_experts_layer_build_amd.optim import MoKAdamW  # noqa: E402

BF = torch.bfloat16
T, H, I, E, K, IS = 96, 256, 128, 4, 2, 128
SHAPES = ((IS, H), (IS, H), (H, IS), (E, I, H), (E, I, H), (E, H, I))


def runtime():
    return MoKRuntime(mok.MoKConfig(hidden=H, intermediate=I, num_experts=E, topk=K, max_tokens=T,
                                    shared_intermediate=IS), mok.MOK_MODE_MXFP8)


def inputs():
    torch.manual_seed(7)
    bf = lambda *s: (torch.randn(s) * 0.05).to(BF).cuda()  # noqa: E731
    rw, ids = mok.router_topk(torch.randn(T, E, device="cuda"), K)
    return bf(T, H) * 20, rw, ids, bf(T, H), [torch.nn.Parameter(bf(*s)) for s in SHAPES]


def train(rt, x, rw, ids, gout, w):
    out = moe_layer(rt, x, rw, ids, *w)
    return [out.detach(), *torch.autograd.grad(out, w, gout)]


def test_a_captured_training_step_follows_the_optimizer():
    x, rw, ids, gout, w = inputs()
    rt = runtime()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):  # (leaves codes of the first weights in the runtime)
        for _ in range(2):
            train(rt, x, rw, ids, gout, w)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = train(rt, x, rw, ids, gout, w)
    opt = MoKAdamW(w, lr=0.02)
    for turn in range(3):
        graph.replay()
        torch.cuda.synchronize()
        want = train(runtime(), x, rw, ids, gout, [torch.nn.Parameter(p.detach().clone()) for p in w])
        assert all(torch.equal(a, b) for a, b in zip(got, want)), turn
        eager = train(rt, x, rw, ids, gout, w)
        assert all(torch.equal(a, b) for a, b in zip(eager, want)), turn
        for p, g in zip(w, got[1:]):
            p.grad = g.clone()
        opt.step()


def test_a_capture_leaves_no_codes_behind():
    x, rw, ids, _, w = inputs()
    rt = runtime()
    with torch.no_grad():
        want = moe_layer(runtime(), x, rw, ids, *w)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = moe_layer(rt, x, rw, ids, *w)
        assert torch.equal(moe_layer(rt, x, rw, ids, *w), want)  # before the first replay
        for _ in range(3):
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(got, want)
            assert torch.equal(moe_layer(rt, x, rw, ids, *w), want)


def test_a_captured_inference_forward_keeps_the_codes_it_reads():
    x, rw, ids, _, w = inputs()
    rt = runtime()
    with torch.no_grad():
        want = moe_layer(rt, x, rw, ids, *w)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = moe_layer(rt, x, rw, ids, *w)
        for p in w:
            p.mul_(2)
        assert not torch.equal(moe_layer(rt, x, rw, ids, *w), want)  # codes made again
        others = [torch.full((n,), 0x55, dtype=torch.uint8, device="cuda")  # would lie where the first codes were
                  for p in w for n in (p.numel(), p.numel() // 32) for _ in range(3)]
        for _ in range(2):
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(got, want)
        assert all((t == 0x55).all() for t in others)
