"""The grouped product with offsets that decrease, which give unspecified rows: nothing outside the output is
written, no row holds anything but an expert's product or what it held, and the call ends."""
import numpy as np
import pytest

from mokutil import ROOT  # noqa: F401

torch = pytest.importorskip("torch")
import mixture_experts_layer_build_amd as mok  # noqa: E402


def tiles_of(offsets, rows, bm, most=None):
    """The tile sums of a workgroup of four waves, as the kernel makes them; `most` None: without an end."""
    lo = np.clip(offsets[:-1], 0, rows)
    hi = np.clip(np.maximum(offsets[1:], lo), 0, rows)
    cnt = -(-(hi - lo) // bm)
    end = (lambda v: v) if most is None else (lambda v: np.minimum(v, most))
    tiles, base, largest = [], 0, 0
    for e0 in range(0, cnt.size, 256):
        group = np.pad(cnt[e0:e0 + 256], (0, max(0, e0 + 256 - cnt.size))).reshape(4, 64)
        s = group.cumsum(1)
        part = end(s[:, -1])
        before = base + part.cumsum() - part
        tiles += list(end(before[:, None] + s - group).reshape(-1)[:cnt.size - e0])
        largest = max(largest, (before[:, None] + s).max(), base + part.sum())
        base = end(base + part.sum())
    return np.array(tiles + [base]), largest, cnt


def test_sums_of_tiles_end():
    """In 64 bits: sums of offsets that do not decrease are untouched; of others they never pass an int, never
    decrease, and give an expert no tile that it does not have."""
    rng = np.random.default_rng(0)
    for rows, E in ((0, 1), (1000, 7), (70000, 300), (1 << 30, 1024), (1 << 29, 1024), (1 << 30, 600)):
        good = np.concatenate([[0], np.sort(rng.integers(0, rows + 1, E - 1)), [rows]])
        to_and_fro = np.arange(E + 1) % 2 * rows
        any_ = rng.integers(-5, rows + 6, E + 1)
        for off in (good, to_and_fro, any_):
            for bm in (128, 256):
                most = rows // bm + E
                tiles, largest, cnt = tiles_of(off, rows, bm, most)
                assert largest < 2 ** 31 and tiles[-1] <= most
                assert (np.diff(tiles) >= 0).all() and (np.diff(tiles) <= cnt).all()
                if off is good:
                    assert np.array_equal(tiles, np.concatenate([[0], cnt.cumsum()]))
    assert tiles_of(np.arange(1025) % 2 * (1 << 29), 1 << 29, 128)[1] >= 2 ** 31


def run(rows, E, n, k, offsets):
    """y in the middle of a larger tensor; every weight is the same, so a row is that product or untouched."""
    x = torch.ones(rows, k, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(E, n, k, dtype=torch.bfloat16, device="cuda")
    buf = torch.full((rows + 2, n), 7.0, dtype=torch.bfloat16, device="cuda")
    mok.grouped_matmul(x, w, offsets.cuda(), out=buf[1:-1])
    torch.cuda.synchronize()
    assert (buf[0] == 7).all() and (buf[-1] == 7).all()
    return buf[1:-1]


@pytest.mark.gpu
@pytest.mark.parametrize("rows,E,n,k", [(5000, 1000, 40, 24), (3000, 9, 256, 64), (3001, 33, 5, 3), (300, 257, 64, 64)])
def test_to_and_fro(rows, E, n, k):
    y = run(rows, E, n, k, (torch.arange(E + 1) % 2 * rows).int())
    assert ((y == k) | (y == 7)).all()
    y = run(rows, E, n, k, torch.tensor([0] + [rows] * E))
    assert (y == k).all()


@pytest.mark.gpu
def test_to_and_fro_over_more_tiles_than_an_int_holds():
    rows = 1 << 29
    y = run(rows, 1024, 1, 1, (torch.arange(1025) % 2 * rows).int())
    for part in y.view(16, -1):
        assert ((part == 1) | (part == 7)).all()
