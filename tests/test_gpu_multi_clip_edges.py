"""The clipped multi-tensor step where there is nothing to step."""
import pytest

from test_gpu_multi_clip import _hp, zs  # noqa: F401  (the fixture)

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
