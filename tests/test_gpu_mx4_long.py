"""4-bit products of up to 32 rows whose columns the waves of a workgroup share, at the sizes where launch shapes, turns
and the scales of a row's end change, against the same oracle and bounds as the other products."""
import numpy as np
import pytest

from oracle import mx4
from test_gpu_mx4 import _check, _operand, zs  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cols", [225, 256, 257, 288, 416, 448, 480, 512, 513, 1000, 1024, 1025, 1280, 2047, 2048, 2049,
                                  2304, 4096, 4127, 5000])
def test_exact_products_by_columns(zs, cols):
    """Every number of blocks in a row's last 256 columns, and turns that are not there."""
    _check(zs, 19, 70, cols, "f32", cols, None)
    _check(zs, 3, 8161, min(cols, 1100), "f32", cols, None)


@pytest.mark.parametrize("rows", [1, 2, 7, 8, 15, 16, 17, 18, 24, 31, 32])
@pytest.mark.parametrize("out", [1, 31, 32, 33, 63, 97, 8160, 8192, 8225])
def test_exact_products_by_rows(zs, rows, out):
    _check(zs, rows, out, 777, "f32", rows + out, None)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,out,cols", [(17, 100, 4096), (32, 1003, 8192), (20, 257, 28672), (1, 8193, 1531),
                                           (16, 9001, 4100), (8, 26000, 4096), (8, 25601, 4095), (8, 25601, 4064)])
def test_products(zs, rows, out, cols, dtype):
    """Scales over a wide range, y of both types, rows apart and scales at odd addresses."""
    _check(zs, rows, out, cols, dtype, 3, (120, 134))
    _check(zs, rows, out, cols, dtype, 4, (60, 70), pad=3, shift=1, y_pad=5)


@pytest.mark.parametrize("cols", [8192, 8161, 7700, 4096, 1000, 300])
@pytest.mark.parametrize("rows,out", [(1, 8200), (20, 300), (9, 102500), (24, 25700), (33, 25700)])
def test_rows_a_multiple_of_4096_bytes_apart(zs, rows, out, cols):
    """Workgroups that begin anywhere in their rows, whole and short ones."""
    _check(zs, rows, out, cols, "f32", cols, None, pad=256 - -(-cols // 32))
    if out < 1000:
        _check(zs, rows, out, cols, "f32", cols, (120, 134), pad=512 - -(-cols // 32))


@pytest.mark.parametrize("rows,out,cols", [(20, 66, 260), (20, 66, 1100), (5, 8200, 1100), (32, 32, 2048)])
def test_nan_blocks(zs, rows, out, cols):
    """A NaN block reaches its row or column alone, the last block of a row too; scales behind a row are not read as
    part of it."""
    import torch
    rng = np.random.default_rng(6)
    xc, xs, x = _operand(rows, cols, rng, (125, 129), pad=2)
    wc, ws, w = _operand(out, cols, rng, (125, 129), pad=2)
    clean = torch.empty(rows, out, device="cuda")
    zs.zs_mx4_matmul(xc, xs, wc, ws, clean)
    nb = -(-cols // 32)
    for bx, bw in ((0, nb - 1), (nb - 1, 0), (nb // 2, nb - 2)):
        xs2, ws2 = xs.clone(), ws.clone()
        xs2[rows - 1, bx] = 255
        ws2[out - 2, bw] = 255
        y = torch.empty(rows, out, device="cuda")
        zs.zs_mx4_matmul(xc, xs2, wc, ws2, y)
        torch.cuda.synchronize()
        bad = torch.isnan(y)
        assert bool(bad[rows - 1].all()) and bool(bad[:, out - 2].all())
        assert int(bad.sum()) == rows + out - 1
        assert torch.equal(y[~bad], clean[~bad])


def test_equal_bits_on_streams_and_in_graphs(zs):
    import torch
    rng = np.random.default_rng(7)
    xc, xs, x = _operand(12, 5000, rng, (125, 129))
    wc, ws, w = _operand(9000, 5000, rng, (125, 129))
    y, z = torch.empty(12, 9000, device="cuda"), torch.empty(12, 9000, device="cuda")
    zs.zs_mx4_matmul(xc, xs, wc, ws, y)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    zs.zs_mx4_matmul(xc, xs, wc, ws, z, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(y, z)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        zs.zs_mx4_matmul(xc, xs, wc, ws, z)
    for _ in range(3):
        z.fill_(0)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, z)
        zs.zs_mx4_matmul(xc, xs, wc, ws, z)
        torch.cuda.synchronize()
        assert torch.equal(y, z)
    want, mag = mx4.matmul(x, w)
    assert (np.abs(y.double().cpu().numpy() - want) <= (-(-157 // 2) + 16) * 2.0 ** -21 * mag).all()
