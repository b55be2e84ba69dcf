"""Workspaces of the clipped step and of the verification are tensors: an address, which has no length that could be
checked, is refused before anything is enqueued."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def zs():
    import torch

    import fsdp_sharded_mixed_flatten_amd as m
    torch.cuda.init()
    return m


def test_verification(zs):
    import torch
    logits = torch.zeros(3, 100, device="cuda")
    tokens = torch.zeros(1, 2, dtype=torch.int32, device="cuda")
    u = torch.full((1, 3), 0.5, device="cuda")
    accepted = torch.full((1,), 7, dtype=torch.int32, device="cuda")
    out = torch.full((1, 3), 7, dtype=torch.int32, device="cuda")
    work = torch.empty(zs.zs_verify_drafts_workspace_bytes(1, 2, 100), dtype=torch.uint8, device="cuda")
    for bad in (work.data_ptr(), None, work.cpu(), work.view(torch.int32), work.cpu().numpy()):
        with pytest.raises(ValueError, match="workspace"):
            zs.zs_verify_drafts(logits, tokens, u, accepted, out, bad)
    assert int(accepted) == 7 and out.tolist() == [[7] * 3]
    zs.zs_verify_drafts(logits, tokens, u, accepted, out, work)
    assert int(accepted) == 0  # 0.5 * 1 against 1 / 100


def test_norm_and_step(zs):
    import torch
    plan = zs.zs_shard_plan_ex([64], 1, 0)
    d = dict(grad=torch.ones(64, dtype=torch.bfloat16, device="cuda"), master=torch.zeros(64, device="cuda"),
             m=torch.zeros(64, device="cuda"), v=torch.zeros(64, device="cuda"))
    ws = torch.zeros(zs.zs_multi_workspace_bytes(plan, 0), dtype=torch.uint8, device="cuda")
    zs.zs_multi_bind(plan, [d], None, ws)
    sumsq = torch.zeros(1, dtype=torch.float64, device="cuda")
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    stats = torch.empty(zs.zs_grad_stats_multi_workspace_bytes(plan), dtype=torch.uint8, device="cuda")
    for bad in (stats.data_ptr(), None, stats.cpu().numpy()):
        with pytest.raises(ValueError, match="stats_workspace"):
            zs.zs_grad_stats_multi(plan, sumsq, flag, ws, bad)
    for bad in (ws.data_ptr(), None):
        with pytest.raises(ValueError, match="workspace"):
            zs.zs_grad_stats_multi(plan, sumsq, flag, bad, stats)
        with pytest.raises(ValueError, match="workspace"):
            zs.zs_adamw_shard_step_multi_clip(plan, [zs.AdamWHParams()], bad)
    zs.zs_grad_stats_multi(plan, sumsq, flag, ws, stats)
    assert float(sumsq) == 64.0 and int(flag) == 0
    zs.zs_multi_unbind(ws)
