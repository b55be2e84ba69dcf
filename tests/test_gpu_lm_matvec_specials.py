"""zs_quant_matvec on special values in every layout: scales that are NaN, infinities and NaN in x, and the largest x
whose sums cannot overflow. What no special value reaches has to be exact (integer products, test_gpu_lm_matvec.py)."""
import numpy as np
import pytest

from oracle import lm
from test_gpu_lm_matvec import Payload, _int_x, zs  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu

ROWS = (1, 3, 6, 20, 37)

# (out, in, world, pre, post, align), block
CASES = [
    ((40, 512, 2, 512, 512, 256), 32), ((40, 512, 2, 512, 512, 256), 128), ((40, 512, 2, 512, 512, 256), 256),
    ((40, 512, 2, 512, 512, 256), 16), ((40, 512, 2, 512, 512, 256), 8),
    ((200, 1024, 3, 256, 0, 256), 256),               # shards that end inside a block
    ((33, 1531, 3, 11, 5, 1), 64), ((33, 1531, 3, 11, 5, 1), 128), ((33, 1531, 3, 11, 5, 1), 8),
    ((60, 777, 7, 40, 3, 8), 32), ((60, 777, 7, 40, 3, 8), 256), ((60, 777, 7, 40, 3, 8), 16),
    ((37, 129, 64, 3, 0, 1), 32), ((37, 129, 64, 3, 0, 1), 256),  # rows over several shards
]
_ids = dict(ids=lambda v: "x".join(map(str, v)) if isinstance(v, tuple) else str(v))


def _payload(zs, layout, block, bits, **kw):  # noqa: F811
    out, n_in, world, pre, post, align = layout
    return Payload(zs, out, n_in, bits, block, world, pre, post, align, seed=out + block + bits, **kw)


def _first_and_last(p):
    """Numbers of the scales of the matrix's first and last element."""
    off = p.plan.tensor(1).flat_off

    def at(j):
        return j // p.S * p.n_scales + j % p.S // p.block

    return at(off), at(off + p.out * p.n_in - 1)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("layout,block", CASES, **_ids)
def test_a_nan_scale_gives_nan_where_its_block_is(zs, layout, block, bits):  # noqa: F811
    import torch
    p = _payload(zs, layout, block, bits)
    first, last = _first_and_last(p)
    good = p.scales.copy()
    n = p.n_scales
    # beside the matrix on both sides, at its ends, around the ends of shards, inside rows
    places = {first - 1, first, first + 1, (first + last) // 2, last - 1, last, last + 1}
    places |= {q * n + d for q in range(1, layout[2]) for d in (-2, -1, 0, 1)} if layout[2] < 8 else {n, 9 * n - 1, 9 * n}
    xs = {rows: _int_x(rows, p.n_in, rows) for rows in ROWS}
    for at in sorted(places):
        if not 0 <= at < len(good):
            continue
        p.scales = good.copy()
        p.scales[at] = np.nan
        p.d_scales = torch.from_numpy(p.scales).cuda()
        w = p.weights()
        hit = np.isnan(w).any(axis=1)
        assert hit.any() == bool(first <= at <= last)
        for rows, x in xs.items():
            y = torch.full((rows, p.out), 7.0, device="cuda")
            p.run(zs, x.cuda(), y)
            got = y.cpu().double().numpy()
            ref = lm.quant_matvec(w[~hit], x.double().numpy())[0]
            assert np.isnan(got[:, hit]).all(), (at, rows)
            assert np.array_equal(got[:, ~hit], ref), (at, rows)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("layout,block", CASES, **_ids)
def test_infinities_and_nan_of_x_stay_in_their_row(zs, layout, block, bits):  # noqa: F811
    import torch
    p = _payload(zs, layout, block, bits)
    w = p.weights()
    for rows in ROWS:
        for value, column in ((np.inf, 0), (-np.inf, p.n_in - 1), (np.nan, p.n_in // 2)):
            x = _int_x(rows, p.n_in, rows)
            ref = lm.quant_matvec(w, x.double().numpy())[0]
            r = rows // 2
            x[r, column] = float(value)
            y = torch.full((rows, p.out), 7.0, device="cuda")
            p.run(zs, x.cuda(), y)
            got = y.cpu().double().numpy()
            assert not np.isfinite(got[r]).any(), (rows, column)
            assert np.array_equal(np.delete(got, r, 0), np.delete(ref, r, 0)), (rows, column)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("layout,block", CASES, **_ids)
def test_largest_x(zs, layout, block, bits):  # noqa: F811
    """|x| = 2^114 (8 bits) or 2^122 (4 bits) in every column, against the largest codes: sums of 128 codes times x stay
    below 2^128, the scales bring the products back to ordinary values. Every sum is a whole number below 2^24 times
    2^114 or 2^122, so the products are exact; the same with signs that alternate, and with one column left."""
    import torch
    p = _payload(zs, layout, block, bits)
    huge, qmax = (2.0 ** 122, 7) if bits == 4 else (2.0 ** 114, 127)
    p.scales[:] = 2.0 ** -110
    p.d_scales = torch.from_numpy(p.scales).cuda()
    p.codes[:] = qmax | qmax << 4 if bits == 4 else qmax
    p.d_codes = torch.from_numpy(p.codes).cuda()
    w = p.weights()
    assert (w == qmax * 2.0 ** -110).all() and p.n_in * qmax < 2 ** 24
    for rows in ROWS:
        for kind in range(3):
            x = torch.full((rows, p.n_in), huge)
            if kind == 1:
                x[:, ::2] *= -1
            if kind == 2:
                x[:] = 0
                x[:, p.n_in // 2] = -huge
            x = x.bfloat16()
            y = torch.full((rows, p.out), 7.0, device="cuda")
            p.run(zs, x.cuda(), y)
            assert np.array_equal(y.cpu().double().numpy(), x.double().numpy() @ w.T), (rows, kind)
