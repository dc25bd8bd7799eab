"""The 4-bit layer with long lists of an expert's tokens: the order of a list, and what it costs."""
import numpy as np
import pytest

from mokutil import ROOT  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import mixture_experts_layer_build_amd as mok  # noqa: E402


def layer(E, H=128, I=64):
    gen = torch.Generator(device="cuda").manual_seed(E)
    ws = {}
    for name, shape in dict(routed_gate=(E, I, H), routed_up=(E, I, H), routed_down=(E, H, I)).items():
        w = (torch.randn(shape, generator=gen, device="cuda") * 0.05).to(torch.bfloat16)
        ws[name], ws[name + "_scale"], _ = mok.w4_quantize(w, "int4", 32)
    return ws


@pytest.mark.parametrize("T,k,E", [(65, 1, 1), (33, 2, 3), (257, 1, 2), (300, 3, 5), (8192, 1, 1), (8192, 1, 4),
                                   (1024, 8, 8), (1024, 8, 1024), (128, 64, 64), (4096, 2, 100)])
@pytest.mark.parametrize("kind", ["one", "random", "runs", "some none"])
def test_rows_are_those_of_small_batches(T, k, E, kind):
    """A token's row has the same bits whichever tokens share its row tile: those of batches of 20 tokens."""
    rng = np.random.default_rng(T + E)
    if kind == "one":
        ids = np.tile(np.arange(k) % E, (T, 1))
    elif kind == "runs":
        ids = (np.arange(T)[:, None] * E // T + np.arange(k)) % E
    else:
        ids = rng.integers(0, E, (T, k))
    if kind == "some none":
        ids[rng.random((T, k)) < 0.3] = -1
        ids[rng.random((T, k)) < 0.1] = E
    x = torch.from_numpy(rng.normal(size=(T, 128))).to(torch.bfloat16).cuda()
    rw, ids = torch.from_numpy(rng.random((T, k))).float().cuda(), torch.from_numpy(ids).cuda()
    ws = layer(E)
    got = mok.forward_w4(x, rw, ids, ws)
    for t0 in sorted({0, T // 3, T - 33, T // 2}):
        some = slice(t0, t0 + 33)  # (more than 64 choices, or more than a row tile's parts of them)
        assert torch.equal(got[some], mok.forward_w4(x[some], rw[some], ids[some], ws))


def test_the_cost_of_a_list_grows_with_its_length():
    """Eight times the tokens on one expert take eight times as long, about (51 times where each token was ranked among
    all others)."""
    ws = layer(4)

    def best(T):
        x, rw = torch.randn(T, 128, device="cuda").to(torch.bfloat16), torch.ones(T, 1, device="cuda")
        ids = torch.full((T, 1), 2, dtype=torch.int64, device="cuda")
        times = []
        for _ in range(12):
            a, b = torch.cuda.Event(True), torch.cuda.Event(True)
            a.record()
            mok.forward_w4(x, rw, ids, ws)
            b.record()
            torch.cuda.synchronize()
            times.append(a.elapsed_time(b))
        return min(times)

    assert best(8192) <= 16 * best(1024)
