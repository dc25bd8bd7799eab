"""The router where its rules decide: keys of both zeros, and choices that
have no expert.

Tolerances as in test_gpu_router.py: a gradient's element is off by 2^-16 of
M, the row's largest |dw| (finite ones) times scale plus the losses' terms."""
import numpy as np
import pytest

from mokutil import ROOT  # noqa: F401
from oracle import ops as oops

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import mixture_experts_layer_build_amd as mok  # noqa: E402

BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("E,k", [(16, 1), (16, 8), (64, 8), (128, 8), (128, 16), (128, 17), (300, 8), (600, 8), (600, 16)])
def test_keys_of_both_zeros_are_equal(E, k, dtype):
    """Each row has one logit of -0 and, at a higher id, one of +0, all others
    are distinct and below, and the bias is -0: the keys are -0 + -0 = -0 and
    +0 + -0 = +0, which are equal, so the lower id comes first. (No other
    keys are equal, so nothing else sends a row down another path.)"""
    rng = np.random.default_rng([E, k])
    for T in (9, 33000) if E == 64 else (9,):
        l = -1.0 - np.argsort(rng.random((T, E)), 1).astype(np.float32)
        for t in range(T):
            low, high = np.sort(rng.choice(E, 2, replace=False))
            l[t, low], l[t, high] = -0.0, 0.0
        bias = np.full(E, -0.0, np.float32)
        print(f"zeros T={T} E={E} k={k} {dtype}", flush=True)
        _, ids = mok.router_topk(torch.from_numpy(l).cuda().to(dtype), k, bias=torch.from_numpy(bias).cuda())
        np.testing.assert_array_equal(ids[:9].cpu().numpy(), oops.router(l[:9], k, bias=bias)[1])


@pytest.mark.parametrize("scoring,renorm", [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)])
@pytest.mark.parametrize("E,k", [(20, 6), (128, 8), (400, 20), (700, 9)])
@pytest.mark.parametrize("losses", [False, True])
def test_choices_without_an_expert_get_no_gradient(E, k, scoring, renorm, losses):
    """Fewer live experts than k: the forward gives id -1 and weight 0, so a
    logarithm or a quotient of the weights has an infinite or undefined
    gradient there. It must reach nothing."""
    rng = np.random.default_rng(E)
    T = 11
    l = rng.standard_normal((T, E)).astype(np.float32)
    for t in range(T - 1):
        l[t, rng.permutation(E)[1 + t % (k - 1):]] = -np.inf
    lt = torch.from_numpy(l).cuda()
    how = dict(scoring=scoring, renormalize=renorm, scale=1.5)
    out = mok.router_topk(lt, k, losses=losses, **how)
    ids = out[1]
    assert (ids[:-1] == -1).any(1).all() and (ids[-1] >= 0).all()
    dw = torch.from_numpy(rng.standard_normal((T, k)).astype(np.float32)).cuda()
    bad = torch.tensor([float("inf"), -float("inf"), float("nan")], device="cuda")[torch.arange(T * k, device="cuda") % 3].view(T, k)
    dl = np.array([0.7, 0.01], np.float32)
    more = dict(counts=out[2], d_losses=torch.from_numpy(dl).cuda()) if losses else {}
    got = mok.router_topk_backward(torch.where(ids < 0, bad, dw), lt, ids, **how, **more)
    assert torch.equal(got, mok.router_topk_backward(torch.where(ids < 0, 0.0, dw), lt, ids, **how, **more))
    counts = out[2].cpu().numpy() if losses else None
    ref = oops.router_backward(dw.double().cpu().numpy(), l, ids.cpu().numpy(), scoring, renorm, 1.5, counts=counts,
                               d_losses=dl)
    M = np.abs(dw.cpu().numpy()).max(1, keepdims=True) * 1.5
    if losses:
        M = M + 0.7 * E / k / T / T * counts[:E].max() + 0.02 / T * (np.where(np.isfinite(l), np.abs(l), 0).max(1, keepdims=True) + 7)
    err = np.abs(got.double().cpu().numpy() - ref)
    assert (err <= 2.0 ** -16 * M).all(), err.max()
    # an id beyond the experts is no choice either
    ids[-1, 1] = E
    dw[-1, 1] = float("nan")
    assert torch.isfinite(mok.router_topk_backward(torch.where(ids < 0, 0.0, dw), lt, ids, **how, **more)).all()
