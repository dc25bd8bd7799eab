"""Calls beyond the last-level cache, whose loads go past it, against calls on
slices of the same data, whose loads do not: the same arithmetic, so the same
bits. (The slices themselves are pinned to the float64 oracle elsewhere.)
"""
import pytest
import torch

if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import mixture_experts_layer_build_amd as mok  # noqa: E402

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
CACHE = 256 << 20


@pytest.mark.parametrize("cols", [512, 2048, 7168, 16384])
@pytest.mark.parametrize("rt", [BF, F32])
def test_norm(cols, rt):
    rows = CACHE // (cols * 4) + 1003  # x and the residual: 4 or 6 bytes an element
    torch.manual_seed(cols)
    x, w = torch.randn(rows, cols, device="cuda").to(BF), torch.randn(cols, device="cuda").to(BF)
    r = torch.randn(rows, cols, device="cuda").to(rt)
    y, s, rstd = mok.rms_norm(x, w, r)
    codes, scale, s8 = mok.rms_norm_mxfp8(x, w, r)
    dy = x
    ds, dw = mok.rms_norm_backward(dy, s, rstd, w, r, dx=None)
    assert torch.equal(s, s8)
    for a, b in ((0, 7), (rows // 2, rows // 2 + 64), (rows - 5, rows)):
        y2, s2, rstd2 = mok.rms_norm(x[a:b], w, r[a:b])
        assert torch.equal(y[a:b], y2) and torch.equal(s[a:b], s2) and torch.equal(rstd[a:b], rstd2)
        codes2, scale2, _ = mok.rms_norm_mxfp8(x[a:b], w, r[a:b])
        assert torch.equal(codes[a:b], codes2) and torch.equal(scale[a:b], scale2)
        assert torch.equal(ds[a:b], mok.rms_norm_backward(dy[a:b], s2, rstd2, w, r[a:b])[0])
    # dw is the sum over the rows; in fp32, added in another order: each product and sum of a column of n rows
    # rounds by at most 2^-24 of what it holds, so by n 2^-24 of the sum of the magnitudes, and the bf16 result by
    # 2^-8. Blocks of rows keep the reference's memory small.
    want, size = torch.zeros(cols, dtype=torch.float64, device="cuda"), torch.zeros(cols, dtype=torch.float64, device="cuda")
    for a in range(0, rows, 8192):
        t = dy[a:a + 8192].double() * s[a:a + 8192].double() * rstd[a:a + 8192, None].double()
        want += t.sum(0)
        size += t.abs().sum(0)
    assert bool(((dw.double() - want).abs() <= want.abs() * 2.0 ** -8 + size * (rows + 2) * 2.0 ** -24).all())


@pytest.mark.parametrize("pt,gt,master,bits", [(BF, BF, True, 32), (F32, F32, False, 32), (BF, BF, True, 8),
                                               (F32, F32, False, 8), (BF, BF, False, 8), (BF, F32, False, 8)])
def test_adamw(pt, gt, master, bits):
    each = (4 if pt == F32 else 6 if master else 2) + (4 if gt == F32 else 2) + (2 if bits == 8 else 8)
    n = CACHE // each // 32 * 32 + 32 * 1000 + 5  # the last block is not full
    torch.manual_seed(bits)
    p = torch.randn(n, device="cuda").to(pt)
    g = torch.randn(n, device="cuda").to(gt)
    ms = p.float() if master else None
    if bits == 32:
        st = [torch.randn(n, device="cuda"), torch.rand(n, device="cuda")]
    else:
        st = [(torch.randint(0, 120, (n,), dtype=torch.uint8, device="cuda"),
               torch.full(((n + 31) // 32,), 118, dtype=torch.uint8, device="cuda")) for _ in range(2)]
    whole = [t for t in (p, ms, *(st if bits == 32 else [t for pair in st for t in pair])) if t is not None]

    def part(t, a, b):
        return t[a // 32:(b + 31) // 32] if t.numel() == (n + 31) // 32 else t[a:b]
    cuts = [(0, 4128), (n // 64 * 32, n // 64 * 32 + 3200), (n - 5 - 3200, n)]
    before = [[part(t, a, b).clone() for t in whole] for a, b in cuts]
    call = dict(step=3, lr=1e-2, weight_decay=0.1, seed=9)
    mok.adamw_step([p], [g], [st[0]], [st[1]], [ms] if master else None, **call)
    for (a, b), c in zip(cuts, before):
        c = [t.clone() for t in c]  # (dense and aligned, on their own)
        q = c[0]
        rest = c[1 + bool(master):]
        moments = rest if bits == 32 else [(rest[0], rest[1]), (rest[2], rest[3])]
        mok.adamw_step([q], [g[a:b].clone()], [moments[0]], [moments[1]], [c[1]] if master else None, **call)
        for i, (big, small) in enumerate(zip(whole, c)):
            # (the root's codes are rounded by the element's number in the call, alike in the first part alone)
            if bits == 8 and a > 0 and i == len(whole) - 2:
                continue
            assert torch.equal(part(big, a, b), small), (i, a)
