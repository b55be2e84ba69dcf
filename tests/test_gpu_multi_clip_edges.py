"""The clipped multi-tensor step where there is nothing to step, and what a captured one repeats."""
import numpy as np
import pytest

import oracle
from gpu_util import dev16
from test_gpu_multi_clip import Run, _hp, _sizes, zs  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("numels", [[], [0], [0, 0, 0]])
@pytest.mark.parametrize("rank", [0, 1])
def test_a_plan_without_elements(zs, numels, rank):
    """Nothing is bound, and nothing has to be: the sum is 0 and the flag 0, in a workspace of the bytes that the
    library names, and the step does nothing."""
    import torch
    plan = zs.zs_shard_plan_ex(numels, 4, rank)
    ws = torch.zeros(zs.zs_multi_workspace_bytes(plan, 0), dtype=torch.uint8, device="cuda")
    zs.zs_multi_bind(plan, [{} for _ in numels], None, ws)
    sumsq = torch.full((2,), 7.0, dtype=torch.float64, device="cuda")
    flag = torch.full((2,), 7, dtype=torch.int32, device="cuda")
    stats = torch.empty(zs.zs_grad_stats_multi_workspace_bytes(plan), dtype=torch.uint8, device="cuda")
    zs.zs_grad_stats_multi(plan, sumsq, flag, ws, stats)
    zs.zs_adamw_shard_step_multi_clip(plan, [_hp(zs)], ws)
    assert sumsq.tolist() == [0.0, 7.0] and flag.tolist() == [0, 7]
    zs.zs_multi_unbind(ws)


def test_other_plans_still_need_their_fields(zs):
    import torch
    plan = zs.zs_shard_plan_ex([4096, 0], 4, 1)
    ws = torch.zeros(zs.zs_multi_workspace_bytes(plan, 0), dtype=torch.uint8, device="cuda")
    g = torch.zeros(1024, dtype=torch.bfloat16, device="cuda")
    stats = torch.empty(zs.zs_grad_stats_multi_workspace_bytes(plan), dtype=torch.uint8, device="cuda")
    sumsq = torch.zeros(1, dtype=torch.float64, device="cuda")
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    for bound in ({}, dict(grad=g)):
        zs.zs_multi_bind(plan, [bound, {}], None, ws)
        if not bound:
            with pytest.raises(zs.ZsError) as e:
                zs.zs_grad_stats_multi(plan, sumsq, flag, ws, stats)
            assert e.value.status == zs.ZS_EINVAL
        with pytest.raises(zs.ZsError) as e:
            zs.zs_adamw_shard_step_multi_clip(plan, [_hp(zs)], ws)
        assert e.value.status == zs.ZS_EINVAL
        zs.zs_multi_unbind(ws)


def test_replays_follow_the_gradient_and_skip(zs):
    """Every replay of a captured norm, factor and step against the eager calls: norm, flag, factor, skip and every
    element, where a replay's gradient is finite and where it is not."""
    import torch
    a, b = Run(zs, _sizes(), 4, 1, 21, 300), Run(zs, _sizes(), 4, 1, 21, 300)
    out = {r: (torch.empty(1, device="cuda"), torch.empty(1, dtype=torch.int32, device="cuda")) for r in (a, b)}

    def step(r):
        r.norm()
        zs.zs_clip_scale(r.sumsq, r.flag, 0.1, *out[r])
        zs.zs_adamw_shard_step_multi_clip(r.plan, [_hp(zs)], r.ws, scale=out[r][0], skip=out[r][1])

    for r in (a, b):
        step(r)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(a)
    rng = np.random.default_rng(5)
    for k in range(5):
        for i, o in enumerate(a.o):
            bits = oracle.f32_to_bf16(np.float32(rng.standard_normal(o["g"].size)))
            if k in (1, 3) and i == 0:
                bits[7] = 0x7F80 if k == 1 else 0x7FC0
            if bits.size:
                for r in (a, b):
                    r.pieces[i]["grad"].copy_(dev16(bits))
        before = a.pieces[0]["master"].clone()
        g.replay()
        step(b)
        torch.cuda.synchronize()
        bad = k in (1, 3)
        assert int(out[a][1]) == int(out[b][1]) == int(a.flag) == int(b.flag) == bad
        assert torch.equal(before, a.pieces[0]["master"]) == bad
        if not bad:
            assert float(a.sumsq) == float(b.sumsq) and float(out[a][0]) == float(out[b][0])
        for x, y in zip(a.pieces, b.pieces):
            assert all(torch.equal(x[name], y[name]) for name in x)


def test_a_captured_step_keeps_its_hyperparameters(zs):
    """Step count and learning rate are passed by value: every replay repeats those of the capture."""
    import torch
    a, b = Run(zs, [5000, 300], 2, 1, 31), Run(zs, [5000, 300], 2, 1, 31)
    g = torch.cuda.CUDAGraph()
    hp = _hp(zs, step=3, lr=1e-3)
    zs.zs_adamw_shard_step_multi_clip(a.plan, [hp], a.ws)
    zs.zs_adamw_shard_step_multi_clip(b.plan, [hp], b.ws)
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        zs.zs_adamw_shard_step_multi_clip(a.plan, [hp], a.ws)
    hp.step, hp.lr = 100, 5e-2  # the structure was read by the call
    for _ in range(3):
        g.replay()
        zs.zs_adamw_shard_step_multi_clip(b.plan, [_hp(zs, step=3, lr=1e-3)], b.ws)
        torch.cuda.synchronize()
        for x, y in zip(a.pieces, b.pieces):
            assert all(torch.equal(x[name], y[name]) for name in x)


def test_replays_follow_the_table(zs):
    """A captured norm and step after the workspace was bound to other pieces, and after it was unbound."""
    import torch
    plan = zs.zs_shard_plan_ex([4096, 24], 1, 0)

    def pieces(value):
        return [dict(grad=torch.full((n,), value, dtype=torch.bfloat16, device="cuda"),
                     master=torch.zeros(n, device="cuda"), m=torch.zeros(n, device="cuda"),
                     v=torch.zeros(n, device="cuda")) for n in (4096, 24)]

    ws = torch.zeros(zs.zs_multi_workspace_bytes(plan, 0), dtype=torch.uint8, device="cuda")
    stats = torch.empty(zs.zs_grad_stats_multi_workspace_bytes(plan), dtype=torch.uint8, device="cuda")
    sumsq = torch.full((1,), 7.0, dtype=torch.float64, device="cuda")
    flag = torch.full((1,), 7, dtype=torch.int32, device="cuda")

    def calls():
        zs.zs_grad_stats_multi(plan, sumsq, flag, ws, stats)
        zs.zs_adamw_shard_step_multi_clip(plan, [_hp(zs)], ws)

    first, second = pieces(1.0), pieces(2.0)
    zs.zs_multi_bind(plan, first, None, ws)
    calls()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        calls()
    g.replay()
    torch.cuda.synchronize()
    assert float(sumsq) == 4120.0 and int(flag) == 0
    held = [d["master"].clone() for d in first]
    zs.zs_multi_bind(plan, second, None, ws)
    for _ in range(2):
        g.replay()
        torch.cuda.synchronize()
        assert float(sumsq) == 4 * 4120.0
    assert all(torch.equal(h, d["master"]) for h, d in zip(held, first))
    assert all(bool((d["master"] < 0).all()) for d in second)
    held = [d["master"].clone() for d in second]
    zs.zs_multi_unbind(ws)
    for _ in range(2):
        flag.fill_(7)
        g.replay()
        torch.cuda.synchronize()
        assert float(sumsq) == 0.0 and int(flag) == 0
    assert all(torch.equal(h, d["master"]) for h, d in zip(held, second))
