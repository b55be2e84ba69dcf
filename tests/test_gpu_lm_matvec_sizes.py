"""zs_quant_matvec where its launch shapes change: 4096, 8192 and 32768 rows of W on either side, 2048 columns, 1, 4,
16, 32 and 64 rows of x, whole and split blocks of every size, both widths of codes. Integer products, which have to
match the 64-bit ones exactly (test_gpu_lm_matvec.py says why)."""
import numpy as np
import pytest

from oracle import lm
from test_gpu_lm_matvec import Payload, _int_x, zs  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu

ROWS = (1, 2, 4, 5, 16, 17, 32, 33, 64)

# (out, in, world, pre, align, blocks)
WHOLE = [
    (4096, 256, 2, 256, 256, (32, 128)),
    (4097, 256, 1, 0, 256, (64, 256)),
    (8192, 256, 2, 0, 256, (32, 256)),
    (8193, 256, 1, 256, 256, (64, 128)),
    (32767, 256, 1, 0, 256, (32, 256)),
    (32768, 256, 8, 256, 256, (128,)),       # shards that end inside a block: split
    (32784, 256, 2, 0, 256, (128,)),
    (32771, 256, 1, 0, 256, (64, 256)),
    (33000, 96, 1, 96, 32, (32,)),          # a row ends inside a chunk
    (4112, 2304, 2, 0, 256, (32, 64, 256)),  # more than 2048 columns: turns for every wave
    (8192, 2304, 2, 0, 256, (128,)),
    (8208, 2304, 2, 0, 256, (32, 256)),
    (4097, 2048, 1, 0, 256, (64, 128)),
]
SPLIT = [
    (4096, 333, 3, 5, 1, (32, 128)),
    (4097, 333, 3, 0, 1, (64, 256)),
    (8191, 300, 3, 7, 1, (32, 256)),
    (8193, 300, 3, 0, 1, (64, 128)),
    (32771, 97, 3, 0, 1, (32, 256)),
    (33001, 161, 7, 3, 8, (64, 128)),
    (4099, 2100, 3, 0, 1, (32, 256)),
    (8200, 272, 1, 0, 16, (16,)),           # whole blocks of 16
    (33000, 272, 1, 16, 16, (16,)),
    (5000, 72, 2, 8, 8, (8, 16)),
]
CASES = [(c, block) for c in WHOLE + SPLIT for block in c[5]]


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("case,block", CASES, ids=lambda v: "x".join(map(str, v[:5])) if isinstance(v, tuple) else str(v))
def test_integer_products_are_exact(zs, case, block, bits):  # noqa: F811
    import torch
    out, n_in, world, pre, align, _ = case
    p = Payload(zs, out, n_in, bits, block, world, pre, 0, align, seed=out + block + bits)
    x = _int_x(max(ROWS), n_in, n_in)
    ref, mag = lm.quant_matvec(p.weights(), x.double().numpy())
    assert mag.max() * 8 < 2 ** 24  # in steps of the smallest scale, 2^-3
    ref, dx = torch.from_numpy(ref), x.cuda()
    for rows in ROWS:
        y = torch.full((rows, out), 7.0, device="cuda")
        p.run(zs, dx[:rows], y)
        got = y.cpu().double()
        assert torch.equal(got, ref[:rows]), (rows, int((got != ref[:rows]).sum()), np.argwhere(
            (got != ref[:rows]).numpy())[:4].tolist())
