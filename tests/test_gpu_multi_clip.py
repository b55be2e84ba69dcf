"""The clipped multi-tensor step on the GPU against the oracle: the squared norm within the bound of double sums in
another order (n terms: n 2^-53 relative), factor, flag and every element of the step bit-identical."""
import numpy as np
import pytest

import oracle
from gpu_util import dev16, dev32, host16, host32

pytestmark = pytest.mark.gpu

SENT = 0x5A5A


@pytest.fixture(scope="module")
def zs():
    import torch

    import fsdp_sharded_mixed_flatten_amd as m
    torch.cuda.init()
    return m


def _sizes(H=256, V=1000):
    sizes = [V * H]
    for _ in range(2):
        sizes += [H * H, H * 688, H, H]
    return sizes + [H, 1000, 3, 1, 0, 8, 257]


class Run:
    """One rank's pieces on the GPU (in one arena each, or apart) and as the oracle's arrays."""

    def __init__(self, zs, numels, world, rank, seed, persist_below=0, groups=None, fields=("param", "full"),
                 apart=False):
        import torch
        self.zs, self.numels, self.world, self.rank = zs, numels, world, rank
        self.plan = zs.zs_shard_plan_ex(numels, world, rank, persist_below_elems=persist_below, groups=groups)
        self.groups = groups or [0] * len(numels)
        rng = np.random.default_rng(seed)
        self.o, self.pieces = [], []
        for i in range(len(numels)):
            info = self.plan.tensor(i)
            n = info.own_hi - info.own_lo
            real = np.arange(info.own_lo, info.own_hi) < numels[i]
            g = oracle.f32_to_bf16(np.float32(rng.standard_normal(n) * 1e-2 * real))
            master = np.float32(rng.standard_normal(n) * 0.02 * real)
            o = dict(g=g, master=master, m=np.float32(rng.standard_normal(n) * 1e-3 * real),
                     v=np.float32(rng.random(n) * 1e-6 * real), p=np.full(n, SENT, np.uint16),
                     full=np.full(info.padded_numel, SENT, np.uint16), lo=info.own_lo, hi=info.own_hi,
                     replicated=zs.lib().zs_plan_tensor_replicated(self.plan.handle, i))
            self.o.append(o)
            pad = [torch.empty(1 << 16, device="cuda")] if apart else None
            d = dict(grad=dev16(g), master=dev32(master), m=dev32(o["m"]), v=dev32(o["v"]))
            for name in fields:
                d[name] = dev16(o["p" if name == "param" else name])
            self.pieces.append(d)
            del pad
        self.fields = fields
        self.ws = torch.zeros(zs.zs_multi_workspace_bytes(self.plan, 0), dtype=torch.uint8, device="cuda")
        zs.zs_multi_bind(self.plan, self.pieces, None, self.ws)
        self.stats = torch.full((zs.zs_grad_stats_multi_workspace_bytes(self.plan),), 0xFF, dtype=torch.uint8,
                                device="cuda")
        self.sumsq = torch.full((1,), 7.0, dtype=torch.float64, device="cuda")
        self.flag = torch.full((1,), 7, dtype=torch.int32, device="cuda")

    def norm(self, stream=None):
        self.zs.zs_grad_stats_multi(self.plan, self.sumsq, self.flag, self.ws, self.stats, stream=stream)

    def expected(self):
        total, bad, n = 0.0, 0, 1
        for o in self.o:
            if o["g"].size:
                s, f = oracle.grad_sumsq(oracle.bf16_to_f32(o["g"]))
                bad |= f
                if not (o["replicated"] and self.rank):
                    total += s
                n += o["g"].size
        return total, bad, n * 2.0 ** -53

    def check_norm(self):
        want, bad, rel = self.expected()
        got = float(self.sumsq)
        assert int(self.flag) == bad
        if not bad:
            assert abs(got - want) <= rel * want
        return got

    def step_oracle(self, hps, scale, skip, step):
        for i, o in enumerate(self.o):
            if not o["g"].size or skip:
                continue
            h = hps[self.groups[i] if len(hps) > 1 else 0]
            hp = oracle.HParams(h.lr, h.beta1, h.beta2, h.eps, h.weight_decay, step)
            oracle.adamw_f32grad(hp, oracle.bf16_to_f32(o["g"]), 1.0, float(scale), 0, o["master"], o["m"], o["v"],
                                 o["p"])
            o["full"][o["lo"]:o["hi"]] = o["p"]

    def check(self):
        for i, (o, d) in enumerate(zip(self.o, self.pieces)):
            for name in ("master", "m", "v"):
                assert np.array_equal(host32(d[name]).view(np.uint32), o[name].view(np.uint32)), (i, name)
            assert np.array_equal(host16(d["grad"]), o["g"]), i
            if "param" in self.fields:
                assert np.array_equal(host16(d["param"]), o["p"]), i
            if "full" in self.fields:
                assert np.array_equal(host16(d["full"]), o["full"]), i


def _hp(zs, **kw):
    return zs.AdamWHParams(**dict(dict(lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1, step=3), **kw))


@pytest.mark.parametrize("world,rank", [(1, 0), (4, 0), (4, 3), (8, 5), (13, 12), (64, 41)])
@pytest.mark.parametrize("persist_below", [0, 300, 10 ** 7])
def test_norm(zs, world, rank, persist_below):
    r = Run(zs, _sizes(), world, rank, world + rank, persist_below)
    r.norm()
    first = r.check_norm()
    r.stats.fill_(0xFF)
    r.norm()
    assert float(r.sumsq) == first  # the same bits again


@pytest.mark.parametrize("numels", [[8], [1], [255], [256], [16384], [16385], [16384 * 3 + 8], [2048] * 40,
                                    [8] * 1000, [300, 5] * 77, [1 << 22]])
def test_norm_sizes(zs, numels):
    """Chunks of 256 and workgroups of 64 chunks, filled and begun."""
    r = Run(zs, numels, 1, 0, len(numels))
    r.norm()
    r.check_norm()


def test_the_ranks_sums_add_up_to_the_whole_norm(zs):
    """All ranks' parts of one gradient, replicated tensors counted once."""
    numels, world = _sizes(), 4
    total = 0.0
    gen = np.random.default_rng(3)
    whole = [oracle.f32_to_bf16(np.float32(gen.standard_normal(n))) for n in numels]
    for rank in range(world):
        r = Run(zs, numels, world, rank, 1, 300)
        for i, d in enumerate(r.pieces):
            o = r.o[i]
            padded = np.zeros(max(o["full"].size, 1), np.uint16)
            padded[:numels[i]] = whole[i]
            if d["grad"].numel():
                d["grad"].copy_(dev16(padded[o["lo"]:o["hi"]]))
        r.norm()
        total += float(r.sumsq)
    want = sum(float((oracle.bf16_to_f32(w).astype(np.float64) ** 2).sum()) for w in whole)
    assert abs(total - want) <= 1e-12 * want


@pytest.mark.parametrize("bad", [np.inf, -np.inf, np.nan])
def test_flag(zs, bad):
    """One element in any piece, in a replicated one on another rank too; the largest finite values set no flag."""
    import torch
    bits = int(oracle.f32_to_bf16(np.array([bad], np.float32))[0])
    for piece, at in ((0, 0), (0, -1), (3, 5), (5, -1), (6, 0)):
        r = Run(zs, _sizes(), 4, 2, 5, 1001)
        r.o[piece]["g"][at] = bits
        r.pieces[piece]["grad"].copy_(dev16(r.o[piece]["g"]))
        r.norm()
        assert int(r.flag) == 1
        r.o[piece]["g"][at] = 0x7F7F
        r.pieces[piece]["grad"].copy_(dev16(r.o[piece]["g"]))
        r.norm()
        assert int(r.flag) == 0
        r.check_norm()
    torch.cuda.synchronize()


@pytest.mark.parametrize("world,rank,persist_below", [(1, 0, 0), (4, 3, 300), (64, 9, 0)])
@pytest.mark.parametrize("fields", [(), ("param",), ("full",), ("param", "full")])
def test_clipped_step(zs, world, rank, persist_below, fields):
    """Two steps of two groups, clipped by the norm of this rank's pieces."""
    import torch
    numels = _sizes()
    groups = [1 if n < 300 else 0 for n in numels]
    r = Run(zs, numels, world, rank, 7, persist_below, groups, fields)
    scale, skip = torch.empty(1, device="cuda"), torch.empty(1, dtype=torch.int32, device="cuda")
    for step, max_norm in ((3, 0.05), (4, 1e6)):
        hps = [_hp(zs, step=step), _hp(zs, step=step, weight_decay=0.0, lr=3e-4)]
        r.norm()
        zs.zs_clip_scale(r.sumsq, r.flag, max_norm, scale, skip)
        zs.zs_adamw_shard_step_multi_clip(r.plan, hps, r.ws, scale=scale, skip=skip)
        torch.cuda.synchronize()
        want = np.float32(oracle.clip_scale([float(r.sumsq)], max_norm))
        assert np.float32(scale.item()) == want and int(skip) == 0 and (want == 1.0) == (max_norm > 1)
        r.step_oracle(hps, want, 0, step)
        r.check()


def test_skip_leaves_everything(zs):
    import torch
    r = Run(zs, _sizes(), 4, 1, 11)
    r.pieces[1]["grad"][3] = 0x7F80
    r.o[1]["g"][3] = 0x7F80
    scale, skip = torch.empty(1, device="cuda"), torch.empty(1, dtype=torch.int32, device="cuda")
    r.norm()
    zs.zs_clip_scale(r.sumsq, r.flag, 1.0, scale, skip)
    zs.zs_adamw_shard_step_multi_clip(r.plan, [_hp(zs)], r.ws, scale=scale, skip=skip)
    torch.cuda.synchronize()
    assert int(skip) == 1
    r.check()  # as it was


def test_without_scale_and_skip_it_is_the_unclipped_step(zs):
    import torch
    a, b = Run(zs, _sizes(), 4, 2, 12, apart=True), Run(zs, _sizes(), 4, 2, 12)
    zs.zs_adamw_shard_step_multi_clip(a.plan, [_hp(zs)], a.ws)
    zs.zs_adamw_shard_step_multi(b.plan, _hp(zs), b.ws)
    zs.zs_gather_params_multi(b.plan, b.ws)
    torch.cuda.synchronize()
    for x, y in zip(a.pieces, b.pieces):
        assert all(torch.equal(x[name], y[name]) for name in x)


def test_special_gradients(zs):
    """Zeros, subnormals, the largest values, infinities and NaN through the step without a skip."""
    import torch
    r = Run(zs, [4096], 1, 0, 13)
    special = np.array([0, 0x8000, 1, 0x8001, 0x7F7F, 0xFF7F, 0x7F80, 0xFF80, 0x7FC0], np.uint16)
    r.o[0]["g"][:] = np.resize(special, 4096)
    r.pieces[0]["grad"].copy_(dev16(r.o[0]["g"]))
    scale = torch.tensor([0.5], device="cuda")
    zs.zs_adamw_shard_step_multi_clip(r.plan, [_hp(zs)], r.ws, scale=scale)
    torch.cuda.synchronize()
    r.step_oracle([_hp(zs)], 0.5, 0, 3)
    for name in ("master", "m", "v"):
        got, want = host32(r.pieces[0][name]), r.o[0][name]
        assert np.array_equal(np.isnan(got), np.isnan(want))
        fine = ~np.isnan(want)
        assert np.array_equal(got[fine].view(np.uint32), want[fine].view(np.uint32))


def test_empty_plan(zs):
    import torch
    for numels in ([], [0, 0]):
        plan = zs.zs_shard_plan_ex(numels, 4, 1)
        ws = torch.zeros(max(zs.zs_multi_workspace_bytes(plan, 0), 256), dtype=torch.uint8, device="cuda")
        g = torch.zeros(8, dtype=torch.bfloat16, device="cuda")
        f = torch.zeros(8, device="cuda")
        zs.zs_multi_bind(plan, [dict(grad=g, master=f, m=f, v=f) for _ in numels], None, ws)
        sumsq = torch.full((1,), 7.0, dtype=torch.float64, device="cuda")
        flag = torch.full((1,), 7, dtype=torch.int32, device="cuda")
        stats = torch.empty(max(zs.zs_grad_stats_multi_workspace_bytes(plan), 16), dtype=torch.uint8, device="cuda")
        try:
            zs.zs_grad_stats_multi(plan, sumsq, flag, ws, stats)
        except zs.ZsError as e:  # a plan that owns nothing binds no field
            assert e.status == zs.ZS_EINVAL
        else:
            assert float(sumsq) == 0.0 and int(flag) == 0


def test_streams_and_graphs(zs):
    """The clipped step captured once: replays follow the gradients, and a non-finite one skips."""
    import torch
    a, b = Run(zs, _sizes(), 4, 1, 21, 300), Run(zs, _sizes(), 4, 1, 21, 300)
    out = {r: (torch.empty(1, device="cuda"), torch.empty(1, dtype=torch.int32, device="cuda")) for r in (a, b)}

    def step(r):
        r.norm()
        zs.zs_clip_scale(r.sumsq, r.flag, 0.1, *out[r])
        zs.zs_adamw_shard_step_multi_clip(r.plan, [_hp(zs)], r.ws, scale=out[r][0], skip=out[r][1])

    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        step(a)
    step(b)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(a)
    rng = np.random.default_rng(2)
    for k in range(4):
        for i, o in enumerate(a.o):
            bits = oracle.f32_to_bf16(np.float32(rng.standard_normal(o["g"].size)))
            if k == 2 and i == 0:
                bits[7] = 0x7F80
            for r in (a, b):
                if bits.size:
                    r.pieces[i]["grad"].copy_(dev16(bits))
        g.replay()
        step(b)
        torch.cuda.synchronize()
        assert int(out[a][1]) == (k == 2) and float(a.sumsq) == float(b.sumsq) or k == 2
        for x, y in zip(a.pieces, b.pieces):
            assert all(torch.equal(x[name], y[name]) for name in x)


def test_a_workspace_without_a_table_is_left_alone(zs):
    """A table whose tag was cleared on the device (as zs_multi_unbind does) is not followed."""
    import torch
    r = Run(zs, _sizes(), 4, 1, 23)
    held = [d["master"].clone() for d in r.pieces]
    r.ws[:8].zero_()
    zs.zs_adamw_shard_step_multi_clip(r.plan, [_hp(zs)], r.ws)
    r.norm()
    torch.cuda.synchronize()
    assert float(r.sumsq) == 0.0 and int(r.flag) == 0
    assert all(torch.equal(x, d["master"]) for x, d in zip(held, r.pieces))
