"""The language-model operators on buffers that share an address range and no element: columns side by side in one
matrix, small arrays behind the rows. Results are the bits of the same call on buffers apart, and what belongs to
neither stays as it was."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def zs():
    import torch

    import fsdp_sharded_mixed_flatten_amd as m
    torch.cuda.init()
    return m


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("vocab", [100, 5003, 33000])
def test_logits_and_gradients_side_by_side(zs, vocab, dtype):
    import torch
    rows = 7
    dtype = getattr(torch, dtype)
    gen = torch.Generator().manual_seed(vocab)
    both = torch.full((rows, 2 * vocab + 3), 7.0, dtype=dtype, device="cuda")
    z, g = both[:, :vocab], both[:, vocab + 1:2 * vocab + 1]
    z.copy_((torch.randn(rows, vocab, generator=gen) * 3).to(dtype))
    apart, want = z.clone(), torch.empty(rows, vocab, dtype=dtype, device="cuda")
    tokens = torch.randint(0, vocab, (rows,), generator=gen).to(torch.int32).cuda()
    lp, stats = torch.empty(rows, device="cuda"), torch.empty(rows, 2, device="cuda")
    zs.zs_token_logprobs(z, tokens, logprob=lp, stats=stats)

    def untouched():
        return torch.equal(z, apart) and bool((both[:, vocab] == 7).all()) and bool((both[:, 2 * vocab + 1:] == 7).all())

    zs.zs_token_logprobs_backward(z, tokens, stats, lp, g)
    zs.zs_token_logprobs_backward(apart, tokens, stats, lp, want)
    assert torch.equal(g, want) and untouched()
    ids = torch.randint(0, vocab, (rows, 9), generator=gen).to(torch.int32).cuda()
    teacher = torch.randn(rows, 9, generator=gen).cuda()
    loss, loss2 = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    zs.zs_distill_topk(z, ids, teacher, loss, grad_logits=g)
    zs.zs_distill_topk(apart, ids, teacher, loss2, grad_logits=want)
    assert torch.equal(g, want) and torch.equal(loss, loss2) and untouched()
    with pytest.raises(zs.ZsError):  # one column too far to the left
        zs.zs_distill_topk(z, ids, teacher, loss, grad_logits=both[:, vocab - 1:2 * vocab - 1])


@pytest.mark.parametrize("rows", [1, 4, 6, 40])
def test_x_and_y_side_by_side(zs, rows):
    import torch
    out, n_in = 200, 512
    plan = zs.zs_shard_plan([out * n_in], 2, 0, 256)
    gen = torch.Generator().manual_seed(rows)
    codes = torch.randint(0, 256, (plan.padded_numel // 2,), generator=gen, dtype=torch.uint8).cuda()
    scales = torch.rand(2 * zs.zs_quant_num_scales(plan, 64), generator=gen).cuda()
    both = torch.full((rows, n_in + out + 2), 7.0, dtype=torch.bfloat16, device="cuda")
    x, y = both[:, :n_in], both[:, n_in + 1:n_in + 1 + out]
    x.copy_(torch.randn(rows, n_in, generator=gen))
    apart, want = x.clone(), torch.empty(rows, out, dtype=torch.bfloat16, device="cuda")
    zs.zs_quant_matvec(plan, 0, out, n_in, 4, 64, codes, scales, x, y)
    zs.zs_quant_matvec(plan, 0, out, n_in, 4, 64, codes, scales, apart, want)
    assert torch.equal(y, want) and torch.equal(x, apart)
    assert (both[:, n_in] == 7).all() and (both[:, -1] == 7).all()
