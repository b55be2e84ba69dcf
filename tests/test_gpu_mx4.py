"""The 4-bit format on the GPU against the 64-bit oracle: codes, scales and decoded values have to be equal, products
lie within the bound of their fp32 sums.

Bound of a product: codes multiply exactly (two bits of mantissa each) and scales are powers of two, so what is rounded
are the sums. A matrix instruction adds up to 128 products to an fp32 value; no stage of it is off by more than 2^-23 of
the magnitudes it adds, and it has at most two for the products and one for the sum, hence 2^-21 of the magnitudes an
instruction, which an fp32 value takes part in ceil(blocks / 2) times at most, and 16 more for the sums of a workgroup's
parts. Where all products are multiples of one unit and no sum reaches 2^24 of it, nothing is rounded at all. A bf16
result is then off by half a step, 2^-8 relative, more.
"""
import numpy as np
import pytest

from oracle import mx4

pytestmark = pytest.mark.gpu

SENT = 0xA5


@pytest.fixture(scope="module")
def zs():
    import torch

    import fsdp_sharded_mixed_flatten_amd as m
    torch.cuda.init()
    return m


def _torch_dtype(name):
    import torch
    return {"bf16": torch.bfloat16, "f32": torch.float32}[name]


def _quantize(x):
    """The oracle's quantize in vectors (checked against it below)."""
    rows, cols = x.shape
    blocks = -(-cols // 32)
    p = np.zeros((rows, 32 * blocks))
    p[:, :cols] = x
    p = p.reshape(rows, blocks, 32)
    with np.errstate(all="ignore"):
        bad = ~np.isfinite(p).all(axis=2)
        amax = np.where(bad, 1.0, np.abs(p).max(axis=2))
        e = np.where(amax > 0, np.maximum(np.frexp(amax)[1] - 3, -127), -127)
        y = np.minimum(np.ldexp(np.abs(p), -e[:, :, None]), 6.0)
        step = np.where(y < 2, 0.5, np.where(y < 4, 1.0, 2.0))
        v = np.minimum(np.rint(y / step) * step, 6.0)
    code = np.searchsorted(mx4.VALUES, v).astype(np.int64) | np.where(np.signbit(p), 8, 0)
    code = np.where(bad[:, :, None], 0, code).reshape(rows, 32 * blocks).astype(np.uint8)
    return code[:, 0::2] | (code[:, 1::2] << 4), np.where(bad, 255, e + 127).astype(np.uint8)


def _buffers(rows, cols, dtype, pad=(0, 0, 0), shift=0):
    """(x, codes, scales) as matrices with `pad` elements, 16-byte units and bytes between their rows, and whole arrays.
    All start `shift` elements or bytes into their arrays."""
    import torch
    blocks = -(-cols // 32)

    def matrix(n, width, stride, t, fill):
        base = torch.full((max(n - 1, 0) * stride + width + 64 + shift,), fill, dtype=t, device="cuda")
        return base[shift:].as_strided((n, width), (stride, 1)), base

    x, xb = matrix(rows, cols, cols + pad[0], _torch_dtype(dtype), 7.0)
    codes = torch.full((rows, blocks + pad[1], 16), SENT, dtype=torch.uint8, device="cuda")
    c = codes.view(rows, -1)[:, :16 * blocks]
    s, sb = matrix(rows, blocks, blocks + pad[2], torch.uint8, SENT)
    return x, c, s, (xb, codes, sb)


def _fill(x, values):
    import torch
    x.copy_(torch.from_numpy(np.ascontiguousarray(values, np.float32)).to("cuda"))
    return x.float().cpu().numpy().astype(np.float64)


SHAPES = [(1, 1), (1, 31), (1, 32), (1, 33), (3, 64), (2, 1531), (5, 70), (77, 96), (300, 5), (4, 8192), (33, 1000),
          (1, 40000), (257, 32)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("pad,shift", [((0, 0, 0), 0), ((3, 1, 5), 1)], ids=["tight", "strided"])
def test_round_trip(zs, rows, cols, dtype, pad, shift):
    import torch
    rng = np.random.default_rng(rows * 1000 + cols)
    x, c, s, bases = _buffers(rows, cols, dtype, pad, shift)
    values = _fill(x, rng.standard_normal((rows, cols)) * np.exp2(rng.integers(-20, 20, (rows, 1))))
    zs.zs_mx4_quantize(x, c, s)
    want_c, want_s = _quantize(values)
    if rows * cols < 3000:
        slow = mx4.quantize(values)
        assert np.array_equal(slow[0], want_c) and np.array_equal(slow[1], want_s)
    assert np.array_equal(s.cpu().numpy(), want_s)
    assert np.array_equal(c.cpu().numpy(), want_c)
    # nothing between the rows is written
    held = bases[1].cpu().numpy()
    assert (held[:, -(-cols // 32):] == SENT).all()
    gaps = bases[2].clone()
    gaps[shift:].as_strided(s.shape, s.stride()).fill_(SENT)
    assert bool((gaps == SENT).all())
    y, _, _, (yb, _, _) = _buffers(rows, cols, dtype, pad, shift)
    zs.zs_mx4_dequantize(c, s, y)
    want = mx4.dequantize(want_c, want_s)[:, :cols]
    assert np.array_equal(y.double().cpu().numpy(), want)
    y.fill_(7.0)
    assert bool((yb == 7.0).all())
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_special_values(zs, dtype):
    """Zeros, the smallest and largest magnitudes, ties of every pair of neighbours in both signs, infinities, NaN."""
    top = float(np.float32(2.0 ** 128 * (1 - 2.0 ** -8)))  # bf16's largest
    ties = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0, 6.0]
    rows = [[0.0] * 32, [-0.0] * 32, [2.0 ** -133] * 32, [2.0 ** -126, -2.0 ** -127, 2.0 ** -128, 2.0 ** -129],
            [top, -top, top / 4], [top, 2.0 ** -126], ties + [-t for t in ties], [t * 2.0 ** -120 for t in ties],
            [-t * 2.0 ** 120 for t in ties], [1.0] * 31 + [np.inf], [-np.inf] + [3.0] * 31, [1.0, np.nan, 2.0],
            [np.nan] * 32, [0.0] * 31 + [1.0]]
    values = np.zeros((len(rows), 96))
    for i, r in enumerate(rows):
        values[i, 32:32 + len(r)] = r  # a block of its own between two of zeros
    x, c, s, _ = _buffers(*values.shape, dtype)
    held = _fill(x, values)
    zs.zs_mx4_quantize(x, c, s)
    want_c, want_s = mx4.quantize(held)
    assert np.array_equal(s.cpu().numpy(), want_s) and np.array_equal(c.cpu().numpy(), want_c)
    y = x.clone()
    zs.zs_mx4_dequantize(c, s, y)
    assert np.array_equal(y.double().cpu().numpy(), mx4.dequantize(want_c, want_s), equal_nan=True)


def test_every_bf16_value(zs):
    """All 65536 bit patterns, each the largest of its block and each under a larger one."""
    import torch
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    x = torch.zeros(65536, 64, dtype=torch.bfloat16)
    x[:, 5] = bits
    x[:, 40] = bits
    x[:, 63] = torch.where(torch.isfinite(bits), (bits.float() * 3).clamp(-3e38, 3e38), 0).to(torch.bfloat16)
    values = x.double().numpy()
    d, c, s, _ = _buffers(65536, 64, "bf16")
    d.copy_(x)
    zs.zs_mx4_quantize(d, c, s)
    want_c, want_s = _quantize(values)
    assert np.array_equal(s.cpu().numpy(), want_s) and np.array_equal(c.cpu().numpy(), want_c)
    f, c2, s2, _ = _buffers(65536, 64, "f32")
    f.copy_(d)
    zs.zs_mx4_quantize(f, c2, s2)
    assert torch.equal(c, c2) and torch.equal(s, s2)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_every_code_under_every_scale(zs, dtype):
    codes = np.tile(np.arange(256, dtype=np.uint8), (256, 1))
    scales = np.repeat(np.arange(256, dtype=np.uint8)[:, None], 16, axis=1)
    y, c, s, _ = _buffers(256, 512, dtype)
    import torch
    c.copy_(torch.from_numpy(codes))
    s.copy_(torch.from_numpy(scales))
    zs.zs_mx4_dequantize(c, s, y)
    with np.errstate(over="ignore"):
        want = mx4.dequantize(codes, scales).astype(np.float32)  # 6 * 2^127 is infinite
    assert np.array_equal(y.float().cpu().numpy(), want, equal_nan=True)


def test_a_row_past_32_bits(zs):
    """2^32 + 4131 bf16 elements in one row: blocks on both sides of 2^31 and 2^32 elements."""
    import torch
    n = (1 << 32) + 4131
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GiB")
    x = torch.empty(1, n, dtype=torch.bfloat16, device="cuda")
    for lo in range(0, n, 1 << 28):
        x[:, lo:lo + (1 << 28)].normal_(0.0, 1.0)
    blocks = -(-n // 32)
    c = torch.empty(1, 16 * blocks, dtype=torch.uint8, device="cuda")
    s = torch.empty(1, blocks, dtype=torch.uint8, device="cuda")
    zs.zs_mx4_quantize(x, c, s)
    y = torch.empty_like(x)
    zs.zs_mx4_dequantize(c, s, y)
    for first in (0, (1 << 26) - 64, (1 << 27) - 64, blocks - 128):
        lo, hi = 32 * first, min(32 * (first + 128), n)
        want_c, want_s = _quantize(x[:, lo:hi].double().cpu().numpy())
        assert np.array_equal(c[:, 16 * first:16 * (first + 128)].cpu().numpy(), want_c)
        assert np.array_equal(s[:, first:first + 128].cpu().numpy(), want_s)
        assert np.array_equal(y[:, lo:hi].double().cpu().numpy(), mx4.dequantize(want_c, want_s)[:, :hi - lo])


# ---------------------------------------------------------------- products


def _operand(rows, cols, rng, scales=None, pad=0, shift=0):
    """A quantized matrix on the GPU (codes rows `pad` 16-byte units longer, scales rows `pad` bytes; scales start
    `shift` bytes into their array), and its values."""
    import torch
    blocks = -(-cols // 32)
    codes = rng.integers(0, 256, (rows, 16 * blocks), dtype=np.uint8)
    if cols % 32:  # as zs_mx4_quantize leaves them
        wide = np.stack([codes & 15, codes >> 4], axis=2).reshape(rows, -1)
        wide[:, cols:] = 0
        codes = (wide[:, 0::2] | (wide[:, 1::2] << 4)).astype(np.uint8)
    s = np.full((rows, blocks), 127, np.uint8) if scales is None else \
        rng.integers(scales[0], scales[1] + 1, (rows, blocks)).astype(np.uint8)
    c = torch.full((rows, blocks + pad, 16), SENT, dtype=torch.uint8, device="cuda").view(rows, -1)[:, :16 * blocks]
    c.copy_(torch.from_numpy(codes))
    base = torch.full((rows * (blocks + pad) + shift,), 255, dtype=torch.uint8, device="cuda")
    sd = base[shift:].view(rows, -1)[:, :blocks] if rows else base[shift:].view(0, blocks)
    sd.copy_(torch.from_numpy(s))
    return c, sd, mx4.dequantize(codes, s)


def _bound(blocks, mag, want, dtype):
    tol = (-(-blocks // 2) + 16) * 2.0 ** -21 * mag
    return tol + (2.0 ** -8 * np.abs(want) if dtype == "bf16" else 0)


def _check(zs, rows, out, cols, dtype, seed, scales, pad=0, shift=0, y_pad=0, stream=None):
    import torch
    rng = np.random.default_rng(seed)
    xc, xs, x = _operand(rows, cols, rng, scales, pad, shift)
    wc, ws, w = _operand(out, cols, rng, scales, pad, shift)
    base = torch.full((rows, out + y_pad), 7.0, dtype=_torch_dtype(dtype), device="cuda")
    y = base[:, :out]
    torch.cuda.synchronize()
    zs.zs_mx4_matmul(xc, xs, wc, ws, y, stream=stream)
    torch.cuda.synchronize()
    want, mag = mx4.matmul(x, w)
    got = y.double().cpu().numpy()
    if scales is None and dtype == "f32":
        assert np.array_equal(got, want)  # multiples of 1/4 below 2^22
    else:
        assert (np.abs(got - want) <= _bound(-(-cols // 32), mag, want, dtype)).all()
    assert bool((base[:, out:] == 7.0).all())
    return got


ROWS = [1, 2, 15, 16, 17, 32, 33, 64, 65, 127, 128, 129, 255, 256, 257, 511, 513]
OUTS = [1, 15, 16, 17, 100, 127, 128, 129, 255, 256, 257, 1000]
INS = [1, 32, 33, 96, 128, 160, 256, 257, 480, 511, 512, 513, 1024, 1531, 2048, 4097]


@pytest.mark.parametrize("rows", ROWS)
def test_exact_products_by_rows(zs, rows):
    """Codes under one scale: fp32 sums of quarters are exact, whatever their order."""
    for out, cols in ((1, 32), (17, 33), (129, 512), (256, 544), (300, 1531)):
        _check(zs, rows, out, cols, "f32", rows, None)


@pytest.mark.parametrize("out", OUTS)
def test_exact_products_by_out_features(zs, out):
    for rows, cols in ((1, 64), (5, 544), (70, 256), (260, 352)):
        _check(zs, rows, out, cols, "f32", out, None)


@pytest.mark.parametrize("cols", INS)
def test_exact_products_by_columns(zs, cols):
    for rows, out in ((1, 16), (18, 40), (140, 130), (258, 260)):
        _check(zs, rows, out, cols, "f32", cols, None)


@pytest.mark.parametrize("rows,out", [(1, 25473), (16, 25500), (17, 10113), (20, 30001), (33, 10200), (64, 25600),
                                      (65, 8200), (65, 16390), (128, 16500), (130, 16384), (129, 40800), (257, 20481),
                                      (300, 20600), (512, 20992)])
def test_exact_products_of_many_tiles(zs, rows, out):
    """Sizes at which there are tiles enough for every larger shape of workgroup, and one fewer or more."""
    for cols in (32, 288, 1055, 1600):
        _check(zs, rows, out, cols, "f32", rows, None)


@pytest.mark.parametrize("rows,out", [(20, 26000), (100, 17000), (300, 21000)])
def test_products_of_many_tiles(zs, rows, out):
    for dtype in ("bf16", "f32"):
        _check(zs, rows, out, 1216, dtype, 7, (120, 134), pad=1, shift=1, y_pad=3)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,out,cols", [(1, 4096, 4096), (3, 65, 8192), (20, 1003, 1536), (48, 256, 2048),
                                           (77, 503, 1531), (130, 384, 1024), (300, 520, 4096), (1024, 1024, 512)])
@pytest.mark.parametrize("scales", [(120, 134), (60, 70), (183, 185)], ids=["around1", "small", "large"])
def test_products(zs, rows, out, cols, dtype, scales):
    _check(zs, rows, out, cols, dtype, rows + out, scales)


@pytest.mark.parametrize("rows,out,cols", [(1, 40, 2048), (19, 33, 1024), (80, 200, 1600), (270, 300, 2080)])
def test_strides(zs, rows, out, cols):
    for pad, shift, y_pad in ((1, 1, 0), (3, 2, 5), (0, 3, 1), (2, 0, 64)):
        _check(zs, rows, out, cols, "f32", 5, None, pad, shift, y_pad)
        _check(zs, rows, out, cols, "bf16", 5, (125, 129), pad, shift, y_pad)


@pytest.mark.parametrize("rows,out", [(2, 20), (40, 60), (150, 140), (300, 270), (3, 25600), (70, 16400), (260, 20500)])
def test_nan_blocks_infinities_and_zeros(zs, rows, out):
    """A NaN scale reaches every result of its row and no other; products past fp32's range are infinite; what is below
    its normal range may be 0."""
    import torch
    cols = 1024
    rng = np.random.default_rng(rows)
    xc, xs, x = _operand(rows, cols, rng)
    wc, ws, w = _operand(out, cols, rng)
    xs[rows // 2, 31] = 255
    ws[out - 1, 0] = 255
    wc[out - 1, :16] = 0  # zeros under a NaN scale are NaN too
    y = torch.empty(rows, out, device="cuda")
    zs.zs_mx4_matmul(xc, xs, wc, ws, y)
    want = x @ w.T
    want[rows // 2, :] = np.nan
    want[:, out - 1] = np.nan
    assert np.array_equal(y.double().cpu().numpy(), want, equal_nan=True)
    one = torch.full((rows, cols // 2), 0x22, dtype=torch.uint8, device="cuda")  # ones
    big = torch.full((rows, cols // 32), 254, dtype=torch.uint8, device="cuda")
    wone = torch.full((out, cols // 2), 0x22, dtype=torch.uint8, device="cuda")
    for scale, want1 in ((254, np.inf), (0, cols), (117, cols * 2.0 ** 117)):
        zs.zs_mx4_matmul(one, big, wone, torch.full((out, cols // 32), scale, dtype=torch.uint8, device="cuda"), y)
        assert (y.double().cpu().numpy() == (want1 if scale == 254 else cols * 2.0 ** (scale - 127 + 127))).all()
    small = torch.zeros(rows, cols // 32, dtype=torch.uint8, device="cuda")
    zs.zs_mx4_matmul(one, small, wone, torch.full((out, cols // 32), 100, dtype=torch.uint8, device="cuda"), y)
    assert bool((y.abs() <= cols * 2.0 ** -126).all())


def test_empty_sizes(zs):
    import torch
    rng = np.random.default_rng(0)
    xc, xs, _ = _operand(3, 64, rng)
    wc, ws, _ = _operand(5, 64, rng)
    y = torch.full((3, 5), 7.0, device="cuda")
    zs.zs_mx4_matmul(xc[:, :0], xs[:, :0], wc[:, :0], ws[:, :0], y)
    assert bool((y == 0).all())
    zs.zs_mx4_matmul(xc[:0], xs[:0], wc, ws, y[:0])
    zs.zs_mx4_matmul(xc, xs, wc[:0], ws[:0], y[:, :0])
    zs.zs_mx4_quantize(y[:0], xc[:0, :16], xs[:0, :1])
    zs.zs_mx4_quantize(y[:, :0], xc[:, :0], xs[:, :0])
    zs.zs_mx4_dequantize(xc[:, :0], xs[:, :0], y[:, :0])
    torch.cuda.synchronize()


def test_a_matrix_times_itself_and_equal_bits(zs):
    import torch
    rng = np.random.default_rng(3)
    xc, xs, x = _operand(260, 2048, rng, (120, 130))
    y = [torch.empty(260, 260, device="cuda") for _ in range(2)]
    for t in y:
        zs.zs_mx4_matmul(xc, xs, xc, xs, t)
    want, mag = mx4.matmul(x, x)
    assert torch.equal(y[0], y[1])
    assert (np.abs(y[0].double().cpu().numpy() - want) <= _bound(64, mag, want, "f32")).all()


def test_rows_do_not_depend_on_the_rows_beside_them(zs):
    """A row's exact sums are the same alone and among others."""
    import torch
    rng = np.random.default_rng(4)
    xc, xs, _ = _operand(300, 1056, rng)
    wc, ws, _ = _operand(130, 1056, rng)
    whole = torch.empty(300, 130, device="cuda")
    zs.zs_mx4_matmul(xc, xs, wc, ws, whole)
    for lo, n in ((0, 1), (7, 20), (100, 70), (40, 257)):
        part = torch.empty(n, 130, device="cuda")
        zs.zs_mx4_matmul(xc[lo:lo + n], xs[lo:lo + n], wc, ws, part)
        assert torch.equal(part, whole[lo:lo + n])


def test_binding_refusals(zs):
    import torch
    rng = np.random.default_rng(0)
    xc, xs, _ = _operand(3, 64, rng)
    wc, ws, _ = _operand(5, 64, rng)
    y = torch.empty(3, 5, device="cuda")
    x = torch.empty(3, 64, device="cuda")
    for bad in (lambda: zs.zs_mx4_matmul(xc, xs, wc, ws, y.t().contiguous()),
                lambda: zs.zs_mx4_matmul(xc, xs, wc[:, :16], ws[:, :1], y),
                lambda: zs.zs_mx4_matmul(xc, xs, wc, ws[:4], y),
                lambda: zs.zs_mx4_matmul(xc.int(), xs, wc, ws, y),
                lambda: zs.zs_mx4_matmul(xc, xs, wc, ws, y.double()),
                lambda: zs.zs_mx4_matmul(xc.cpu(), xs, wc, ws, y),
                lambda: zs.zs_mx4_matmul(xc, xs, wc.cpu(), ws, y),
                lambda: zs.zs_mx4_quantize(x.half(), xc, xs),
                lambda: zs.zs_mx4_quantize(x, xc[:, :16], xs),
                lambda: zs.zs_mx4_quantize(x.t(), xc, xs),
                lambda: zs.zs_mx4_dequantize(xc, xs[:2], x)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(zs.ZsError):
        zs.zs_mx4_matmul(xc, xs, wc, ws, xc.view(torch.float32)[:, :5])  # y over x's codes
    with pytest.raises(zs.ZsError):
        zs.zs_mx4_quantize(x[0:1].view(-1)[:32].view(1, 32), x.view(torch.uint8)[:1, 16:32], xs[:1, :1])


def test_streams_and_graphs(zs):
    """On a stream of its own, and captured: replays follow their inputs."""
    import torch
    side = torch.cuda.Stream()
    for rows in (1, 40, 300):
        _check(zs, rows, 260, 1056, "f32", 8, None, stream=side)
        rng = np.random.default_rng(rows)
        wc, ws, w = _operand(260, 1056, rng)
        x = torch.empty(rows, 1056, device="cuda")
        xc = torch.empty(rows, 528, dtype=torch.uint8, device="cuda")
        xs = torch.empty(rows, 33, dtype=torch.uint8, device="cuda")
        y, back = torch.empty(rows, 260, device="cuda"), torch.empty(rows, 1056, dtype=torch.bfloat16, device="cuda")

        def calls():
            zs.zs_mx4_quantize(x, xc, xs)
            zs.zs_mx4_dequantize(xc, xs, back)
            zs.zs_mx4_matmul(xc, xs, wc, ws, y)

        x.normal_()
        calls()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            calls()
        for _ in range(3):
            x.normal_()
            g.replay()
            torch.cuda.synchronize()
            got, held = y.clone(), back.clone()
            y.fill_(0)
            calls()
            torch.cuda.synchronize()
            assert torch.equal(got, y) and torch.equal(held, back)
            want = mx4.dequantize(*_quantize(x.double().cpu().numpy()))
            assert np.array_equal(held.double().cpu().numpy(), want)


def test_gathered_shards_are_one_payload(zs):
    """Shards quantized by their ranks, end to end, are the whole flat buffer's payload, in which a tensor is a matrix."""
    import torch
    n, h, v = 4, 256, 1000
    plan = zs.zs_shard_plan([h, v * h, 32 * 8], n, 0, 128)  # four shards of 64128
    S, T = plan.shard_numel, plan.padded_numel
    assert S % 32 == 0
    flat = torch.randn(T, device="cuda").bfloat16()
    codes, scales = torch.empty(T // 2, dtype=torch.uint8, device="cuda"), \
        torch.empty(T // 32, dtype=torch.uint8, device="cuda")
    for r in range(n):
        zs.zs_mx4_quantize(flat[r * S:(r + 1) * S].view(1, S), codes[r * S // 2:(r + 1) * S // 2].view(1, -1),
                           scales[r * S // 32:(r + 1) * S // 32].view(1, -1))
    want_c, want_s = _quantize(flat.double().cpu().numpy()[None])
    assert np.array_equal(codes.cpu().numpy(), want_c[0]) and np.array_equal(scales.cpu().numpy(), want_s[0])
    off = plan.tensor(1).flat_off
    assert off % 32 == 0
    wc = codes[off // 2:off // 2 + v * h // 2].view(v, h // 2)
    ws = scales[off // 32:off // 32 + v * h // 32].view(v, h // 32)
    rng = np.random.default_rng(1)
    xc, xs, x = _operand(5, h, rng, (125, 129))
    y = torch.empty(5, v, device="cuda")
    zs.zs_mx4_matmul(xc, xs, wc, ws, y)
    w = mx4.dequantize(want_c, want_s)[0, off:off + v * h].reshape(v, h)
    want, mag = mx4.matmul(x, w)
    assert (np.abs(y.double().cpu().numpy() - want) <= _bound(h // 32, mag, want, "f32")).all()
