"""zs_quant_matvec against the 64-bit product with the decoded payload.

Integer cases (codes, small whole x, scales that are powers of two) have every
partial sum exact in fp32, so the result must equal the 64-bit one bit for
bit, whatever the order of the sum. Real-valued cases: a sum of n products in
any order is off by at most n + 1 roundings of 2^-24 of the sum of magnitudes
(each product of a code and a bf16 value is exact in fp32, the scale's product
rounds once), and the stored result by half a step of its type.
"""
import numpy as np
import pytest

from oracle import lm

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def zs():
    import torch

    import fsdp_sharded_mixed_flatten_amd as m
    torch.cuda.init()
    return m


class Payload:
    """A unit of tensors [pre, out x in, post] and a made-up payload of its N shards, on host and device."""

    def __init__(self, zs, out, n_in, bits, block, world, pre=0, post=0, align=1, seed=0, integer=True):
        import torch
        rng = np.random.default_rng(seed)
        self.plan = zs.zs_shard_plan([pre, out * n_in, post], world, 0, align)
        self.out, self.n_in, self.bits, self.block = out, n_in, bits, block
        S = self.plan.shard_numel
        self.S, self.n_scales = S, zs.zs_quant_num_scales(self.plan, block)
        qmax = 7 if bits == 4 else 127
        c = rng.integers(-qmax, qmax + 1, world * S)
        self.codes = (c & 255 if bits == 8 else (c[0::2] & 15) | ((c[1::2] & 15) << 4)).astype(np.uint8)
        n = world * self.n_scales
        self.scales = (2.0 ** rng.integers(-3, 3, n) if integer else rng.uniform(1e-4, 3e-3, n)).astype(np.float32)
        self.d_codes = torch.from_numpy(self.codes).cuda()
        self.d_scales = torch.from_numpy(self.scales).cuda()

    def weights(self):
        info = self.plan.tensor(1)
        return lm.quant_weights(self.codes, self.scales, self.bits, self.block, self.S, self.n_scales, info.flat_off,
                                self.out, self.n_in)

    def run(self, zs, x, y, **kw):
        zs.zs_quant_matvec(self.plan, 1, self.out, self.n_in, self.bits, self.block, self.d_codes, self.d_scales, x, y,
                           **kw)


def _int_x(rows, n_in, seed):
    import torch
    return torch.from_numpy(np.random.default_rng(seed).integers(-4, 5, (rows, n_in)).astype(np.float32)).bfloat16()


# (out, in, world, pre, post, align): rows of W in line with blocks and shards, and not
LAYOUTS = [
    (64, 512, 4, 512, 0, 256),      # everything in line
    (48, 256, 1, 0, 0, 1),
    (16, 128, 2, 0, 128, 128),
    (33, 768, 8, 1000, 77, 256),    # out no multiple of 16
    (1, 4096, 4, 0, 0, 1),
    (200, 1024, 3, 256, 0, 256),    # shards that end inside a block
    (17, 384, 2, 0, 0, 128),
    (130, 96, 2, 32, 0, 32),
    (5, 1531, 3, 11, 5, 1),         # nothing in line
    (37, 129, 64, 3, 0, 1),         # rows over several shards
    (100, 8, 2, 1, 0, 8),
    (9, 1, 2, 0, 0, 1),
    (3, 31, 5, 7, 0, 1),
    (257, 2048, 8, 2048, 8, 128),
    (600, 777, 7, 40, 3, 8),        # shards that end inside rows, with last blocks of any length
    (90, 1001, 16, 13, 0, 1),
    (64, 640, 5, 8, 16, 8),
    (33, 33, 3, 1, 2, 1),
]


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("block", [8, 16, 32, 64, 128, 256])
@pytest.mark.parametrize("layout", LAYOUTS, ids=lambda v: "x".join(map(str, v)))
def test_integer_products_are_exact(zs, layout, block, bits):
    import torch
    out, n_in, world, pre, post, align = layout
    p = Payload(zs, out, n_in, bits, block, world, pre, post, align, seed=out * 7 + block + bits)
    w = p.weights()
    for rows in (1, 3, 16, 37):
        x = _int_x(rows, n_in, rows)
        y = torch.full((rows, out), 7.0, device="cuda")
        p.run(zs, x.cuda(), y)
        ref, mag = lm.quant_matvec(w, x.double().numpy())
        assert mag.max() * 8 < 2 ** 24  # in steps of the smallest scale, 2^-3
        assert np.array_equal(y.cpu().double().numpy(), ref), (rows, layout, block, bits)


@pytest.mark.parametrize("rows", [1, 2, 4, 5, 8, 9, 15, 16, 17, 31, 32, 33, 48, 63, 64])
@pytest.mark.parametrize("bits,block,n_in", [(4, 32, 640), (4, 128, 1024), (8, 64, 448), (4, 16, 333)])
def test_every_row_count(zs, rows, bits, block, n_in):
    import torch
    p = Payload(zs, 70, n_in, bits, block, 2, seed=rows, align=256)
    x = _int_x(rows, n_in, rows)
    y = torch.full((rows, 70), 7.0, device="cuda")
    p.run(zs, x.cuda(), y)
    assert np.array_equal(y.cpu().double().numpy(), lm.quant_matvec(p.weights(), x.double().numpy())[0])


@pytest.mark.parametrize("out,n_in,bits,block,world,align", [
    (515, 4096, 4, 128, 8, 128), (300, 2048, 8, 256, 2, 256), (129, 5000, 4, 32, 4, 1), (64, 11008, 4, 64, 8, 64),
    (77, 1531, 8, 64, 3, 1)])
@pytest.mark.parametrize("rows", [1, 6, 20])
@pytest.mark.parametrize("y_type", ["bfloat16", "float32"])
def test_real_products(zs, out, n_in, bits, block, world, align, rows, y_type):
    import torch
    p = Payload(zs, out, n_in, bits, block, world, pre=99, align=align, seed=5, integer=False)
    x = torch.randn(rows, n_in, generator=torch.Generator().manual_seed(rows)).bfloat16()
    dtype = getattr(torch, y_type)
    y = torch.empty(rows, out, dtype=dtype, device="cuda")
    p.run(zs, x.cuda(), y)
    ref, mag = lm.quant_matvec(p.weights(), x.double().numpy())
    tol = (n_in + 1) * 2.0 ** -24 * mag + torch.finfo(dtype).eps / 2 * np.abs(ref) * (1 + 1e-3)
    assert (np.abs(y.cpu().double().numpy() - ref) <= tol).all()


def test_equals_dequantized_product(zs):
    """The payload of zs_quantize_shard on every rank: the product equals one with zs_dequant_gather's bf16 copy but for
    that copy's rounding, half a step a weight."""
    import torch
    out, n_in, N, bits, block = 192, 1024, 4, 4, 128
    gen = torch.Generator().manual_seed(1)
    plan = zs.zs_shard_plan([n_in, out * n_in], N, 0, 128)
    S, T = plan.shard_numel, plan.padded_numel
    flat = (torch.randn(T, generator=gen) * 0.02).bfloat16().cuda()
    cb, ns = zs.zs_quant_code_bytes(plan, bits), zs.zs_quant_num_scales(plan, block)
    codes = [torch.empty(cb, dtype=torch.uint8, device="cuda") for _ in range(N)]
    scales = [torch.empty(ns, device="cuda") for _ in range(N)]
    for q in range(N):
        zs.zs_quantize_shard(plan, bits, block, flat[q * S:(q + 1) * S].clone(), codes[q], scales[q])
    codes, scales = torch.cat(codes), torch.cat(scales)
    full = torch.empty(T, dtype=torch.bfloat16, device="cuda")
    zs.zs_dequant_gather(plan, bits, block, codes, scales, full)
    x = torch.randn(5, n_in, generator=gen).bfloat16()
    y = torch.empty(5, out, device="cuda")
    zs.zs_quant_matvec(plan, 1, out, n_in, bits, block, codes, scales, x.cuda(), y)
    off = plan.tensor(1).flat_off
    w = full[off:off + out * n_in].view(out, n_in).cpu().double().numpy()
    ref, mag = lm.quant_matvec(w, x.double().numpy())
    assert (np.abs(y.cpu().double().numpy() - ref) <= (2.0 ** -8 + (n_in + 1) * 2.0 ** -24) * mag).all()


def test_strided_and_unaligned_operands(zs):
    """x and y as views into larger matrices at odd places; what lies beside y stays as it was."""
    import torch
    for n_in, align in ((512, 256), (509, 1)):
        p = Payload(zs, 40, n_in, 4, 64, 2, align=align, seed=9)
        big = torch.full((6, n_in + 23), 1000.0).bfloat16()
        big[1:5, 3:3 + n_in] = _int_x(4, n_in, 1)
        x = big.cuda()[1:5, 3:3 + n_in]
        ref = lm.quant_matvec(p.weights(), x.double().cpu().numpy())[0]
        for dtype in (torch.float32, torch.bfloat16):
            buf = torch.full((6, 51), 7.0, dtype=dtype, device="cuda")
            p.run(zs, x, buf[1:5, 5:45])
            want = torch.full((6, 51), 7.0, dtype=torch.float64)
            want[1:5, 5:45] = torch.from_numpy(ref).to(dtype).double()
            assert torch.equal(buf.cpu().double(), want)


def test_special_values(zs):
    """A NaN scale gives NaN in its row only; an infinite x times a nonzero code is infinite; huge x does not overflow
    on the way."""
    import torch
    out, n_in, block = 32, 512, 128
    p = Payload(zs, out, n_in, 4, block, 1, seed=2)
    p.d_scales[5 * 4 + 2] = float("nan")  # row 5, third block
    x = _int_x(2, n_in, 0)
    y = torch.empty(2, out, device="cuda")
    p.run(zs, x.cuda(), y)
    got = y.cpu().double().numpy()
    ref = lm.quant_matvec(p.weights(), x.double().numpy())[0]
    assert np.isnan(got[:, 5]).all()
    assert np.array_equal(np.delete(got, 5, 1), np.delete(ref, 5, 1))
    # x = 2^100 at one place, 0 elsewhere: the weight itself, scaled
    p = Payload(zs, out, n_in, 4, block, 1, seed=3)
    x = torch.zeros(1, n_in)
    x[0, 77] = 2.0 ** 120
    y = torch.empty(1, out, device="cuda")
    p.run(zs, x.bfloat16().cuda(), y)
    assert np.array_equal(y.cpu().double().numpy()[0], p.weights()[:, 77] * 2.0 ** 120)
    x[0, 77] = float("inf")
    p.run(zs, x.bfloat16().cuda(), y)
    w = p.weights()[:, 77]
    want = np.where(w == 0, np.nan, np.sign(w) * np.inf)
    assert np.array_equal(y.cpu().double().numpy()[0], want, equal_nan=True)


def test_empty_products(zs):
    import torch
    plan = zs.zs_shard_plan([0, 16], 2, 0)
    codes = torch.zeros(8, dtype=torch.uint8, device="cuda")
    scales = torch.ones(2, device="cuda")
    y = torch.full((3, 5), 7.0, device="cuda")
    x = torch.zeros(3, 0, dtype=torch.bfloat16, device="cuda")
    zs.zs_quant_matvec(plan, 0, 5, 0, 4, 8, codes, scales, x, y)  # in_features = 0: zeros
    assert (y == 0).all()
    zs.zs_quant_matvec(plan, 1, 2, 8, 4, 8, codes, scales, torch.zeros(0, 8, dtype=torch.bfloat16, device="cuda"),
                       torch.empty(0, 2, device="cuda"))


def test_offsets_past_32_bits(zs):
    """A matrix behind 2^32 elements of the flat buffer."""
    import torch
    out, n_in, bits, block = 24, 256, 4, 256
    plan = zs.zs_shard_plan([(1 << 32) + 512, out * n_in], 2, 0, 256)
    S, ns = plan.shard_numel, zs.zs_quant_num_scales(plan, block)
    off = plan.tensor(1).flat_off
    assert off > 1 << 32
    codes = torch.zeros(S, dtype=torch.uint8, device="cuda")  # 2 ranks of S / 2 bytes
    scales = torch.zeros(2 * ns, device="cuda")
    rng = np.random.default_rng(0)
    c = rng.integers(-7, 8, out * n_in)
    codes[off // 2:] = 0
    codes[off // 2:off // 2 + out * n_in // 2] = torch.from_numpy(
        ((c[0::2] & 15) | ((c[1::2] & 15) << 4)).astype(np.uint8)).cuda()
    # scales of the whole second shard: the matrix's blocks get the value 2
    scales[ns:] = 2.0
    x = _int_x(2, n_in, 5)
    y = torch.empty(2, out, device="cuda")
    zs.zs_quant_matvec(plan, 1, out, n_in, bits, block, codes, scales, x.cuda(), y)
    w = 2.0 * c.reshape(out, n_in)
    assert np.array_equal(y.cpu().double().numpy(), x.double().numpy() @ w.T)


def test_streams_graph_and_two_calls_at_once(zs):
    """On a side stream, on two streams at once, and captured: replays follow the inputs."""
    import torch
    p = Payload(zs, 96, 1024, 4, 128, 2, align=128, seed=4)
    w = p.weights()
    xs = [_int_x(4, 1024, s) for s in range(5)]
    refs = [lm.quant_matvec(w, x.double().numpy())[0] for x in xs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    dx = [x.cuda() for x in xs]
    ys = [torch.empty(4, 96, device="cuda") for _ in xs]
    torch.cuda.synchronize()
    for i in range(5):
        p.run(zs, dx[i], ys[i], stream=streams[i % 2])
    torch.cuda.synchronize()
    for y, ref in zip(ys, refs):
        assert np.array_equal(y.cpu().double().numpy(), ref)
    sx, sy = dx[0].clone(), torch.empty(4, 96, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        p.run(zs, sx, sy)
    for i in (3, 1, 4):
        sx.copy_(dx[i])
        sy.fill_(-1)
        g.replay()
        torch.cuda.synchronize()
        assert np.array_equal(sy.cpu().double().numpy(), refs[i])
        p.run(zs, dx[0], ys[0])  # eager work between the replays
        torch.cuda.synchronize()
        assert np.array_equal(ys[0].cpu().double().numpy(), refs[0])


def test_binding_refusals(zs):
    import torch
    p = Payload(zs, 32, 64, 4, 32, 2)
    x = torch.zeros(2, 64, dtype=torch.bfloat16, device="cuda")
    y = torch.zeros(2, 32, device="cuda")
    for bad_x, bad_y in ((x.float(), y), (x[:, :63], y), (x, y[:1]), (x, y.half()), (x, y.t().contiguous().t()),
                         (x[0], y)):
        with pytest.raises(ValueError):
            p.run(zs, bad_x, bad_y)
    with pytest.raises(zs.ZsError):
        p.run(zs, x[:1].expand(2, 64), y)  # rows that lie on top of each other
    p.d_codes = p.d_codes[:-1]
    with pytest.raises(ValueError):
        p.run(zs, x, y)
