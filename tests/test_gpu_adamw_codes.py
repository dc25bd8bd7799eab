"""8-bit moments, code by code. With both betas 0 the moments are the
gradient and its square, exactly, so a block's scale must be that of the
definition with no tolerance: the smallest power of two that keeps its largest
magnitude within 448 of it. The codes must be those of the elementary tensor
operations on the same GPU, bit for bit, and each the nearest to its value up
to a unit in the value's last place (2^-23 of it)."""
import numpy as np
import pytest

from mokutil import ROOT  # noqa: F401
from oracle import ops as oops

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import mixture_experts_layer_build_amd as mok  # noqa: E402

F32 = torch.float32


def step(g, m, v, pt=F32, master=False, b1=0.0, b2=0.0):
    n = g.numel()
    p = torch.zeros(n, dtype=pt, device="cuda")
    w = [torch.zeros(n, device="cuda")] if master else None
    mok.adamw_step([p], [g], [m], [v], w, step=1, lr=1e-3, betas=(b1, b2), eps=1.0)


def zeros8(n):
    return (torch.zeros(n, dtype=torch.uint8, device="cuda"), torch.zeros((n + 31) // 32, dtype=torch.uint8, device="cuda"))


def check_m(got, m):
    """Codes and scales of fp32 values m (whole blocks)."""
    x = oops.state_exponent(m)
    np.testing.assert_array_equal(got[1].cpu().numpy(), x + 127)
    k = torch.from_numpy(-x.astype(np.int32)).cuda()
    scaled = torch.ldexp(torch.from_numpy(m).cuda().view(-1, 32), k[:, None])
    np.testing.assert_array_equal(got[0].cpu().numpy(), scaled.to(torch.float8_e4m3fn).view(torch.uint8).view(-1).cpu().numpy())
    f = np.repeat(np.exp2(x), 32)
    u = m.astype(np.float64) / f
    q = oops.decode8(got[0].cpu().numpy(), got[1].cpu().numpy()) / f
    unit = np.exp2(np.floor(np.log2(np.maximum(np.abs(u), 2.0 ** -6))) - 3)
    assert (np.abs(q - u) <= unit / 2 + np.abs(u) * 2.0 ** -23).all()


def test_scales_at_the_low_end():
    """Block maxima from 2^-149 to 2^-109, in and below the top eighth of a
    binade: scale 2^-127 wherever it suffices."""
    rng = np.random.default_rng(0)
    blocks = []
    for e in range(-149, -108):
        for top in (1.0, 1.5, 1.75, 1.9, 1.99):
            b = rng.uniform(-1, 1, 32) * top * 2.0 ** e
            b[rng.integers(32)] = top * 2.0 ** e
            blocks.append(b)
    g = np.concatenate(blocks).astype(np.float32)
    m, v = zeros8(g.size), zeros8(g.size)
    step(torch.from_numpy(g).cuda(), m, v)
    check_m(m, g + np.float32(0))  # (m = 0 + g, so a gradient of -0 gives +0)
    # and the moment of an expert that gets no gradient any more halves at each step
    for _ in range(3):
        half = (oops.decode8(m[0].cpu().numpy(), m[1].cpu().numpy()) * 0.5).astype(np.float32)
        step(torch.zeros(g.size, device="cuda"), m, v, b1=0.5)
        check_m(m, half + np.float32(0))


def blocks_of(values, exponents):
    """Blocks of 448 and 31 of `values`, times 2^x for x in `exponents`."""
    out = []
    for x in exponents:
        for i in range(0, values.size, 31):
            b = np.zeros(32)
            b[0] = 448.0
            b[1:1 + values[i:i + 31].size] = values[i:i + 31]
            out.append(b * 2.0 ** x)
    return np.concatenate(out).astype(np.float32)


@pytest.mark.parametrize("pt,master", [(F32, False), (torch.bfloat16, False), (torch.bfloat16, True)])
@pytest.mark.parametrize("copies", [1, 600])
def test_moments_half_way_between_two_codes(pt, master, copies):
    """Every pair of neighbouring codes under every scale from 2^-60 to 2^49.
    (Many copies: sizes that fill each compute unit several times.)"""
    code = oops.E4M3  # 0, 2^-9, ... 448
    mid = (code[:-1] + code[1:]) / 2
    g = blocks_of(np.concatenate([mid, -mid]), range(-60, 50))
    t = torch.from_numpy(g).cuda().repeat(copies)
    m, v = zeros8(t.numel()), zeros8(t.numel())
    print(f"half way {pt} {master} {t.numel()}", flush=True)
    step(t, m, v, pt, master)
    for i in {0, copies - 1}:
        check_m([a.view(copies, -1)[i] for a in m], g)


def test_a_root_that_is_a_code_is_kept():
    """v = r^2 with r on a code (times 2^x): the random choice has nothing to
    choose, whatever the scale. (From x = -53 on: below, the smallest squares
    are no normal numbers and are rounded.)"""
    g = blocks_of(oops.E4M3[1:], range(-53, 50))
    m, v = zeros8(g.size), zeros8(g.size)
    step(torch.from_numpy(g).cuda(), m, v)
    check_m(v, g)
