"""4-bit products whose rows of codes lie far apart: at 2^22 bytes, the most that offsets inside a tile allow, and
beyond, where another shape of workgroup takes over. Sums are exact, whatever their order."""
import numpy as np
import pytest

from oracle import mx4
from test_gpu_mx4 import zs  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu

FAR = 1 << 22


def _room(gib):
    import torch
    if torch.cuda.mem_get_info()[0] < gib << 30:
        pytest.skip(f"needs {gib} GiB")


def _far(rows, blocks, stride, where, rng):
    """Random codes in the blocks `where` of a matrix of `blocks` blocks whose rows are `stride` bytes apart (zeros in
    the other blocks), under one scale, and the values of `where`."""
    import torch
    base = torch.empty((rows - 1) * stride + 16 * blocks, dtype=torch.uint8, device="cuda")
    c = base.as_strided((rows, 16 * blocks), (stride, 1))
    if blocks > len(where):
        c.zero_()
    codes = rng.integers(0, 256, (rows, 16 * len(where)), dtype=np.uint8)
    d = torch.from_numpy(codes).to("cuda")
    for i, b in enumerate(where):
        c[:, 16 * b:16 * b + 16] = d[:, 16 * i:16 * i + 16]
    s = torch.full((rows, blocks), 127, dtype=torch.uint8, device="cuda")
    return c, s, mx4.dequantize(codes, np.full((rows, len(where)), 127, np.uint8))


# rows of x and of W (equal: one matrix on both sides): waves that share a row's columns, 16 x 16 results, and the three
# sizes of tiles
SIZES = [(20, 40), (7, 40), (100, 300), (1600, 1600), (3200, 3200)]


@pytest.mark.parametrize("rows,out", SIZES)
@pytest.mark.parametrize("stride", [FAR, FAR + 16], ids=["at", "beyond"])
def test_rows_far_apart(zs, rows, out, stride):
    import torch
    _room(16)
    rng = np.random.default_rng(rows)
    where = list(range(17))
    wc, ws, w = _far(out, 17, stride, where, rng)
    xc, xs, x = (wc, ws, w) if rows == out else _far(rows, 17, stride, where, rng)
    y = torch.full((rows, out), 7.0, device="cuda")
    zs.zs_mx4_matmul(xc, xs, wc, ws, y)
    assert np.array_equal(y.double().cpu().numpy(), x @ w.T)


@pytest.mark.parametrize("rows,out", SIZES)
def test_long_rows_far_apart(zs, rows, out):
    """Rows of 2^23 columns that fill their 2^22 bytes: a tile of 256 rows spans 2^30 bytes."""
    import torch
    _room(16)
    rng = np.random.default_rng(out)
    blocks = FAR // 16
    where = [0, 1, 7, 8, blocks // 2, blocks - 17, blocks - 9, blocks - 2, blocks - 1]
    wc, ws, w = _far(out, blocks, FAR, where, rng)
    xc, xs, x = (wc, ws, w) if rows == out else _far(rows, blocks, FAR, where, rng)
    y = torch.full((rows, out), 7.0, device="cuda")
    zs.zs_mx4_matmul(xc, xs, wc, ws, y)
    assert np.array_equal(y.double().cpu().numpy(), x @ w.T)


def test_more_rows_than_one_launch(zs):
    """W's rows far apart and more rows of x than a launch has tiles for: the rows on both sides of the cut."""
    import torch
    rows, period = 16 * 65535 + 1013, 997
    rng = np.random.default_rng(3)
    wc, ws, w = _far(3, 1, FAR + 16, [0], rng)
    few, _, x = _far(period, 1, 16, [0], rng)
    xc = few.repeat(-(-rows // period), 1)[:rows].contiguous()
    xs = torch.full((rows, 1), 127, dtype=torch.uint8, device="cuda")
    y = torch.full((rows, 3), 7.0, device="cuda")
    zs.zs_mx4_matmul(xc, xs, wc, ws, y)
    assert np.array_equal(y.double().cpu().numpy(), (x @ w.T)[np.arange(rows) % period])
