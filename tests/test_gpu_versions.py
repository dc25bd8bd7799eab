"""What a call writes into tensors that it was given is seen by what watches
them: in-place version counters, autograd's check of saved tensors, and the
MXFP8 layer's quantized weights, which are made again when a counter moves."""
import pytest

from mokutil import ROOT  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import mixture_experts_layer_build_amd as mok  # noqa: E402
from mixture_experts_layer_build_amd.autograd import MoKExperts  # noqa: E402
from mixture_experts_layer_build_amd.optim import MoKAdamW  # noqa: E402

BF = torch.bfloat16
T, H, I, E, K, IS = 96, 256, 128, 4, 2, 128


def states(n, bits):
    if bits == 32:
        return torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
    return tuple((torch.zeros(n, dtype=torch.uint8, device="cuda"),
                  torch.zeros((n + 31) // 32, dtype=torch.uint8, device="cuda")) for _ in range(2))


def flat(*ts):
    return [x for t in ts for x in (t if isinstance(t, tuple) else (t,))]


@pytest.mark.parametrize("bits", [32, 8])
def test_a_step_moves_the_counters_of_what_it_writes(bits):
    n = 100
    p, g, w = torch.zeros(n, dtype=BF, device="cuda"), torch.ones(n, device="cuda"), torch.zeros(n, device="cuda")
    m, v = states(n, bits)
    written = flat(p, w, m, v)
    before, gbefore = [t._version for t in written], g._version
    with pytest.raises(mok.MokError):  # a refused call writes nothing
        mok.adamw_step([p], [g], [m], [v], [w], step=0, lr=0.1)
    assert [t._version for t in written] == before
    mok.adamw_step([p], [g], [m], [v], [w], step=1, lr=0.1)
    assert all(t._version > b for t, b in zip(written, before)) and g._version == gbefore
    q = torch.nn.Parameter(torch.ones(64, device="cuda"))
    q.grad = torch.ones(64, device="cuda")
    was = q._version
    MoKAdamW([q], state_bits=bits).step()
    assert q._version > was


def test_a_step_between_forward_and_backward_is_seen():
    w = torch.nn.Parameter(torch.ones(64, device="cuda"))
    loss = (w * w).sum()
    m, v = states(64, 32)
    mok.adamw_step([w], [torch.ones(64, device="cuda")], [m], [v], step=1, lr=0.1)
    with pytest.raises(RuntimeError, match="inplace"):
        loss.backward()


def test_tensors_without_a_counter_are_stepped():
    with torch.inference_mode():
        p = torch.ones(64, device="cuda")
    m, v = states(64, 32)
    mok.adamw_step([p], [torch.ones(64, device="cuda")], [m], [v], step=1, lr=0.5, weight_decay=0.0)
    assert ((p - 0.5).abs() < 1e-5).all()


def test_given_outputs_move_their_counters():
    x, w = torch.randn(5, 64, device="cuda").to(BF), torch.ones(64, dtype=BF, device="cuda")
    y, rstd = torch.empty_like(x), torch.empty(5, device="cuda")
    was = y._version, rstd._version
    mok.rms_norm_mxfp8(x, w, y=y, rstd=rstd)
    assert y._version > was[0] and rstd._version > was[1]
    s, dx = x.float(), torch.empty_like(x)
    was = dx._version
    mok.rms_norm_backward(y, s, rstd, w, dx=dx)
    assert dx._version > was


def test_the_outputs_of_a_forward_on_codes_move_their_counters():
    cfg = mok.MoKConfig(hidden=H, intermediate=I, num_experts=E, topk=K, max_tokens=T)
    ws = mok.Workspace(cfg)
    w = {}
    for n, s in (("routed_gate", (E, I, H)), ("routed_up", (E, I, H)), ("routed_down", (E, H, I))):
        c, sc = mok.mxfp8_quantize(bf(*s).reshape(-1, s[-1]), axis=1)
        w[n], w[n + "_scale"] = c.view(s), sc
    rw, ids = mok.router_topk(torch.randn(T, E, device="cuda"), K)
    out = torch.empty(T, H, dtype=BF, device="cuda")
    context = torch.empty(mok.context_bytes(cfg, mok.MOK_MODE_MXFP8), dtype=torch.uint8, device="cuda")
    was = out._version, context._version
    got = mok.forward_mxfp8(ws, mok.build_schedule(ws, ids), *mok.mxfp8_quantize(bf(T, H), axis=1), rw, w, out=out,
                            context=context)
    assert got is out and out._version > was[0] and context._version > was[1]


def bf(*shape):
    return (torch.randn(shape) * 0.05).to(BF).cuda()


@pytest.mark.parametrize("bits", [32, 8])
def test_an_mxfp8_layer_runs_on_the_weights_that_the_step_wrote(bits):
    torch.manual_seed(3)
    experts = MoKExperts(H, I, E, K, max_tokens=T, shared_intermediate=IS, mode=mok.MOK_MODE_MXFP8, device="cuda")
    experts.init_weights(0.05)
    shared = [torch.nn.Parameter(t) for t in (bf(IS, H), bf(IS, H), bf(H, IS))]
    x, gout = bf(T, H) * 20, bf(T, H)
    rw, ids = mok.router_topk(torch.randn(T, E, device="cuda"), K)

    def run(layer, sh):
        xi, wi = x.clone().requires_grad_(), rw.clone().requires_grad_()
        for p in [*layer.parameters(), *sh]:
            p.grad = None
        out = layer(xi, wi, ids, *sh)
        out.backward(gout)
        return [out.detach(), xi.grad, wi.grad, *[p.grad.clone() for p in [*layer.parameters(), *sh]]]

    first = run(experts, shared)
    opt = MoKAdamW([*experts.parameters(), *shared], lr=0.02, state_bits=bits)
    for turn in range(2):
        opt.step()
        fresh = MoKExperts(H, I, E, K, max_tokens=T, shared_intermediate=IS, mode=mok.MOK_MODE_MXFP8, device="cuda")
        with torch.no_grad():
            for p, q in zip(fresh.parameters(), experts.parameters()):
                p.copy_(q)
        got, want = run(experts, shared), run(fresh, [torch.nn.Parameter(p.detach().clone()) for p in shared])
        assert not torch.equal(got[0], first[0])
        for i, (a, b) in enumerate(zip(got, want)):
            assert torch.equal(a, b), (turn, i)
