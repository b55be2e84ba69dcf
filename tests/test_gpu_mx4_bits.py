"""4-bit products bit for bit: bf16 results of exact sums beside the ties of bf16, the same in every shape of workgroup
and in a row's last columns; zeros under scales whose product passes fp32's range; fp32 values beside the ties of the
4-bit codes. Nothing here is rounded but where the test says how, so that no tolerance is needed."""
import numpy as np
import pytest

from oracle import mx4
from test_gpu_mx4 import _operand, _quantize, zs  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu

# (rows of x, rows of W) of each shape of workgroup at 24 blocks: waves that take turns of 16 x 16 and 64 x 32 results
# and of a row's columns, and the three sizes of tiles
SHAPES = [(1, 1003), (20, 1003), (40, 1001), (40, 10243), (100, 17001), (300, 21003)]


def _rne(v):
    """bf16 bits of float64 values that fp32 holds: nearest, ties to even."""
    u = np.asarray(v, np.float32).view(np.uint32).astype(np.uint64)
    return ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)


def _gpu(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).to("cuda")


def _whole_numbers(values):
    """Codes and scales of a matrix of 24 blocks whose row o times ones in every block's first column is values[o], a
    whole number below 2^24 in magnitude: block i has the number's bit i."""
    bits = (np.abs(values)[:, None] >> np.arange(24)) & 1
    codes = np.zeros((len(values), 24, 16), np.uint8)
    codes[:, :, 0] = bits * np.where(values < 0, 10, 2)[:, None]  # the code of 1, with the sign
    scales = np.broadcast_to(127 + np.arange(24, dtype=np.uint8), (len(values), 24))
    return codes.reshape(len(values), -1), scales


@pytest.mark.parametrize("rows,out", SHAPES)
def test_sums_beside_ties_of_bf16(zs, rows, out):
    """Whole numbers in [2^23, 2^24), whose bf16 neighbours are 2^16 apart: at, one below and one above the tie of an
    even and an odd neighbour, and beside the neighbours themselves, in both signs, under every row's own power of
    two."""
    import torch
    rng = np.random.default_rng(rows)
    low = np.array([0x8000, 0x7FFF, 0x8001, 0, 1, 0xFFFF, 0x4000, 0xC000])
    v = ((0x80 + rng.integers(0, 0x80, out)) << 16) + low[np.arange(out) % 8]
    v = np.where(rng.random(out) < 0.5, -v, v)
    wc, ws = _whole_numbers(v)
    power = rng.integers(-8, 9, rows)
    xc = np.zeros((rows, 24, 16), np.uint8)
    xc[:, :, 0] = 2
    xs = np.broadcast_to((127 + power)[:, None].astype(np.uint8), (rows, 24))
    args = [_gpu(a) for a in (xc.reshape(rows, -1), xs, wc, ws)]
    exact = v[None, :] * np.exp2(power)[:, None]
    y32 = torch.empty(rows, out, device="cuda")
    zs.zs_mx4_matmul(*args, y32)
    assert np.array_equal(y32.double().cpu().numpy(), exact)
    want = _rne(exact)
    for pad in (0, 1, 3):
        y16 = torch.zeros(rows, out + pad, dtype=torch.bfloat16, device="cuda")[:, :out]
        zs.zs_mx4_matmul(*args, y16)
        assert np.array_equal(y16.cpu().contiguous().view(torch.int16).numpy().view(np.uint16), want)


def test_bf16_rows_do_not_depend_on_the_rows_beside_them(zs):
    """Exact sums rounded to bf16 alone, among others, and in a row's last columns."""
    import torch
    rng = np.random.default_rng(4)
    out = 1003
    wc, ws = _whole_numbers(rng.integers(-(1 << 24) + 1, 1 << 24, out))
    x = np.zeros((300, 24, 16), np.uint8)
    x[:, :, 0] = 2
    xc, xs, wc, ws = _gpu(x.reshape(300, -1)), _gpu(np.full((300, 24), 127, np.uint8)), _gpu(wc), _gpu(ws)
    whole = torch.empty(300, out, dtype=torch.bfloat16, device="cuda")
    zs.zs_mx4_matmul(xc, xs, wc, ws, whole)
    for n in (1, 20, 40, 70, 257):
        for o0, o1 in ((0, out), (1, out), (2, 998), (500, 501)):
            part = torch.empty(n, o1 - o0, dtype=torch.bfloat16, device="cuda")
            zs.zs_mx4_matmul(xc[7:7 + n], xs[7:7 + n], wc[o0:o1], ws[o0:o1], part)
            assert torch.equal(part, whole[7:7 + n, o0:o1])


@pytest.mark.parametrize("rows,out", SHAPES)
def test_zeros_under_scales_that_pass_the_range(zs, rows, out):
    """0 times anything finite is 0, whatever 2^(ex + ew) is: blocks of zeros on either side or both under the largest
    scales, alone and beside blocks that are not 0."""
    import torch
    blocks = 24
    rng = np.random.default_rng(out)
    xc, xs, x = _operand(rows, 32 * blocks, rng)
    wc, ws, w = _operand(out, 32 * blocks, rng)
    for some in (slice(0, blocks), slice(0, blocks, 3), slice(blocks - 1, blocks), slice(0, 1)):
        for zero_x, zero_w in ((True, False), (False, True), (True, True)):
            xc2, xs2, wc2, ws2 = (t.clone() for t in (xc, xs, wc, ws))
            if zero_x:
                xc2.view(rows, blocks, 16)[:, some] = 0
            if zero_w:
                wc2.view(out, blocks, 16)[:, some] = 0x80  # -0 and 0
            xs2[:, some] = 254
            ws2[:, some] = 254
            keep = np.ones(blocks, bool)
            keep[some] = False
            keep = np.repeat(keep, 32)
            want = (x * keep) @ (w * keep).T
            y = torch.full((rows, out), 7.0, device="cuda")
            zs.zs_mx4_matmul(xc2, xs2, wc2, ws2, y)
            assert np.array_equal(y.double().cpu().numpy(), want)


def test_fp32_values_beside_the_ties_of_codes(zs):
    """Every tie between neighbouring codes, the fp32 values next to it and the codes themselves, in both signs, under
    every block scale that finite fp32 values have and, in the smallest, magnitudes further down to the last bit."""
    points = np.array([0.25, 0.5, 0.75, 1.0, 1.25, 1.5, 1.75, 2.0, 2.5, 3.0, 3.5, 4.0, 5.0, 6.0, 7.0])
    rows = []
    for e in range(-127, 126):
        with np.errstate(over="ignore"):
            p = np.ldexp(points, e).astype(np.float32)
            p = np.concatenate([p, np.nextafter(p, np.float32(np.inf)), np.nextafter(p, np.float32(0))])
        p = p[np.abs(p) < np.ldexp(8.0, e)]
        p = np.concatenate([p, -p])
        p = np.resize(p, (-(-p.size // 30), 30))
        row = np.zeros((p.shape[0], 32), np.float32)
        row[:, 1:31] = p
        row[:, 0] = np.ldexp(4.0, e)  # the block's exponent, whatever else is in it
        row[:, 31] = np.ldexp(np.float32(1.0), max(e - 10, -149))
        rows.append(row)
    tiny = np.arange(1, 1 << 12, dtype=np.uint32).view(np.float32)  # the smallest magnitudes: codes of 0 under 2^-127
    rows.append(np.resize(tiny, (128, 32)))
    near = (0x00100000 + np.arange(-64, 64)).astype(np.uint32).view(np.float32)  # around the tie 0.25 * 2^-127
    rows.append(near.reshape(4, 32))
    x = np.concatenate(rows)
    import torch
    d = _gpu(x)
    c = torch.empty(x.shape[0], 16, dtype=torch.uint8, device="cuda")
    s = torch.empty(x.shape[0], 1, dtype=torch.uint8, device="cuda")
    zs.zs_mx4_quantize(d, c, s)
    want_c, want_s = _quantize(x.astype(np.float64))
    some = np.r_[0:8, x.shape[0] - 140:x.shape[0]]
    slow = mx4.quantize(x[some])
    assert np.array_equal(slow[0], want_c[some]) and np.array_equal(slow[1], want_s[some])
    assert np.array_equal(s.cpu().numpy(), want_s)
    assert np.array_equal(c.cpu().numpy(), want_c)
