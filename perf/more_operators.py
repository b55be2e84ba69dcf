"""More operators of the library as cases to be timed and checked: microscaled 4-bit floating point (quantisation with
decoding, and products), verification of drafted tokens, and the global norm and clipped step of many tensors.

`run` computes a case in elementary torch operations, or, with `own` set, with the library's entry points.
`exact` computes the same outputs from the operators' definitions in 64 bits.
"""
import math

import torch

own = False

CHUNK_ELEMS = 1 << 27  # elements of one chunk where inputs are made or computed in 64 bits
FP4 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)  # what the lower three bits of a code stand for
ADAMW = {"lr": 1e-4, "beta1": 0.9, "beta2": 0.95, "eps": 1e-8, "weight_decay": 0.1, "step": 2}
MAX_NORM = 1.0


def listed():
    return [
        # 20 tokens' activations of the Llama-70B shape before a product, and what the product sees of them: latency
        {"name": "mx4_round_x", "kind": "mx4_round", "rows": 20, "cols": 8192, "dtype": "bf16"},
        # a gate matrix of that shape quantised from its fp32 master and decoded again, as quantisation-aware training does
        {"name": "mx4_round_matrix", "kind": "mx4_round", "rows": 28672, "cols": 8192, "dtype": "f32"},
        # one token through an attention projection of the Llama-7B shape: the smallest product
        {"name": "mx4_one_4096", "kind": "mx4_matmul", "rows": 1, "in": 4096, "out": 4096, "y": "bf16"},
        # the LM head of the Llama-70B shape for four requests of four drafted tokens each: logits in fp32
        {"name": "mx4_drafts_head", "kind": "mx4_matmul", "rows": 20, "in": 8192, "out": 128256, "y": "f32"},
        # a prompt of 4096 tokens through that shape's gate projection: the largest product
        {"name": "mx4_prompt_up", "kind": "mx4_matmul", "rows": 4096, "in": 8192, "out": 28672, "y": "bf16"},
        # sizes that no tile or block divides (an adapter or expert of odd width)
        {"name": "mx4_odd", "kind": "mx4_matmul", "rows": 77, "in": 1531, "out": 5003, "y": "f32"},
        # one request with four drafted tokens, the Llama-7B vocabulary: latency
        {"name": "verify_one", "kind": "verify", "requests": 1, "drafts": 4, "vocab": 32000, "dtype": "bf16",
         "draft_logits": True, "temperature": 1.0},
        # a batch of requests, up to four drafted tokens each, fp32 logits of the Qwen2.5-3B vocabulary, sampled at 0.8
        {"name": "verify_batch_f32", "kind": "verify", "requests": 64, "drafts": 4, "vocab": 151936, "dtype": "f32",
         "draft_logits": True, "temperature": 0.8},
        # the gradient norm of one rank of 64 of the Qwen2.5-3B shape: 434 pieces, most of them small
        {"name": "norm_pieces_small", "kind": "norm", "shape": "qwen25_3b", "world": 64, "persist_below": 0},
        # the Llama-7B shape wrapped per tensor over 8 ranks, norms replicated: 842M elements
        {"name": "norm_pieces_7b", "kind": "norm", "shape": "llama_7b", "world": 8, "persist_below": 100000},
        # norm, factor and clipped AdamW of a shard of one tensor of 1000003 over 4 ranks: latency
        {"name": "clip_step_tiny", "kind": "clip_step", "shape": "tiny", "world": 4, "persist_below": 0},
        # the same for the Qwen2.5-3B shape over 16 ranks: 193M elements of state
        {"name": "clip_step_3b", "kind": "clip_step", "shape": "qwen25_3b", "world": 16, "persist_below": 100000},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["mx4_round", "mx4_matmul", "mx4_matmul", "verify", "norm", "clip_step"])
    if kind == "mx4_round":
        cols = _log_int(rng, 33, 28672)
        if rng.random() < 0.6:
            cols = -(-cols // 32) * 32
        return {"kind": kind, "rows": _log_int(rng, 1, (1 << 27) // cols), "cols": cols,
                "dtype": rng.choice(["bf16", "f32"])}
    if kind == "mx4_matmul":
        n_in, n_out = _log_int(rng, 256, 28672), _log_int(rng, 256, 128256)
        if rng.random() < 0.6:
            n_in, n_out = -(-n_in // 128) * 128, -(-n_out // 16) * 16
        most = min(8192, (1 << 39) // (n_in * n_out), (1 << 28) // n_out)
        return {"kind": kind, "rows": _log_int(rng, 1, max(1, most)), "in": n_in, "out": n_out,
                "y": rng.choice(["bf16", "f32"])}
    if kind == "verify":
        vocab = _log_int(rng, 2000, 152000)
        if rng.random() < 0.5:
            vocab = vocab // 128 * 128
        drafts = rng.randint(1, 12)
        most = max(1, min(256, (3 << 25) // (vocab * (2 * drafts + 1))))
        return {"kind": kind, "requests": _log_int(rng, 1, most), "drafts": drafts, "vocab": vocab,
                "dtype": rng.choice(["bf16", "f32"]), "draft_logits": rng.random() < 0.7,
                "temperature": rng.choice([0.6, 0.8, 1.0, 1.0, 1.5])}
    shape = rng.choice(["tiny", "qwen25_3b", "llama_7b"])
    fewest = {"tiny": 1, "qwen25_3b": 16, "llama_7b": 48}[shape]
    world = rng.choice([w for w in (1, 2, 3, 4, 6, 8, 12, 16, 24, 32, 48, 64, 96, 128) if w >= fewest])
    return {"kind": kind, "shape": shape, "world": world, "persist_below": rng.choice([0, 5000, 100000])}


# ---------------------------------------------------------------- inputs


def _dtype(name):
    return {"bf16": torch.bfloat16, "f32": torch.float32}[name]


def _shape_numels(name):
    """Numbers of elements of a model shape's tensors, in the order of their registration."""
    if name == "tiny":
        return [1_000_003]
    if name == "qwen25_3b":
        h, n, inner, vocab, kv = 2048, 36, 11008, 151936, 256
        layer = [h * h, h, kv * h, kv, kv * h, kv, h * h, inner * h, inner * h, h * inner, h, h]
        return [vocab * h] + n * layer + [h]
    h, n, inner, vocab = 4096, 32, 11008, 32000
    return [vocab * h] + n * (4 * [h * h] + 3 * [h * inner] + 2 * [h]) + [h, vocab * h]


def _piece_lens(case):
    """Elements of rank 0's piece of each tensor: whole below the persistence threshold, else a rank's share of the
    tensor padded to 8 elements a rank."""
    unit = 8 * case["world"]
    return [-(-n // 8) * 8 if n < case["persist_below"] else -(-n // unit) * 8 for n in _shape_numels(case["shape"])]


def _mx4_codes(x):
    """Codes [rows, 16 * blocks] and scales [rows, blocks] of a float matrix, whose last block is padded with zeros."""
    rows, cols = x.shape
    blocks = -(-cols // 32)
    x = torch.nn.functional.pad(x.float(), (0, 32 * blocks - cols)).view(rows, blocks, 32)
    amax = x.abs().amax(dim=2)
    # floor of the logarithm from the exponent's bits; what lies under fp32's normal range has the smallest scale
    e = ((amax.view(torch.int32) >> 23) - 129).clamp(min=-127)
    bad = ~torch.isfinite(amax)
    y = x.abs() * ((127 - e) << 23).view(torch.float32)[:, :, None]  # 2^-e
    step = torch.where(y < 2, 0.5, torch.where(y < 4, 1.0, 2.0))
    y = (torch.round(y / step) * step).clamp(max=6.0)
    code = torch.where(y < 2, 2 * y, torch.where(y < 4, y + 2, y / 2 + 4)).nan_to_num(0.0).to(torch.int32)
    code = torch.where(bad[:, :, None], 0, code | ((x.view(torch.int32) >> 28) & 8)).view(rows, 32 * blocks)
    return (code[:, 0::2] | (code[:, 1::2] << 4)).to(torch.uint8), torch.where(bad, 255, e + 127).to(torch.uint8)


def _mx4_values(codes, scales):
    """The fp32 values [rows, 32 * blocks] that codes and scales stand for."""
    rows, blocks = scales.shape
    table = torch.tensor(FP4 + tuple(-v for v in FP4), device=codes.device)
    v = table[torch.stack([codes & 15, codes >> 4], dim=2).view(rows, blocks, 32).int()]
    s = scales.int()
    # 2^(s - 127): the smallest one lies under the normal range, and 255 is NaN
    s = torch.where(s == 0, 1 << 22, torch.where(s == 255, 0x7FC00000, s << 23)).view(torch.float32)
    return (v * s[:, :, None]).view(rows, 32 * blocks)


def _mx4_weights(out, n_in, gen):
    """A quantised matrix of standard deviation 0.02, made some rows at a time."""
    blocks = -(-n_in // 32)
    codes = torch.empty(out, 16 * blocks, dtype=torch.uint8, device="cuda")
    scales = torch.empty(out, blocks, dtype=torch.uint8, device="cuda")
    step = max(1, CHUNK_ELEMS // n_in)
    for lo in range(0, out, step):
        hi = min(lo + step, out)
        w = torch.empty(hi - lo, n_in, device="cuda").normal_(0.0, 0.02, generator=gen)
        codes[lo:hi], scales[lo:hi] = _mx4_codes(w)
    return codes, scales


def _activations(rows, cols, gen):
    """Activations of a language model: a few columns are far larger than the rest."""
    x = torch.empty(rows, cols, device="cuda").normal_(0.0, 1.0, generator=gen)
    return x * torch.where(torch.rand(cols, device="cuda", generator=gen) < 0.01, 20.0, 1.0)


def _round_inputs(case, gen):
    rows, cols = case["rows"], case["cols"]
    if case["dtype"] == "bf16":
        x = _activations(rows, cols, gen).to(torch.bfloat16)
    else:
        x = torch.empty(rows, cols, device="cuda").normal_(0.0, 0.02, generator=gen)
    blocks = -(-cols // 32)
    return {"x": x, "y": torch.empty_like(x), "codes": torch.empty(rows, 16 * blocks, dtype=torch.uint8, device="cuda"),
            "scales": torch.empty(rows, blocks, dtype=torch.uint8, device="cuda")}


def _matmul_inputs(case, gen):
    w_codes, w_scales = _mx4_weights(case["out"], case["in"], gen)
    x_codes, x_scales = _mx4_codes(_activations(case["rows"], case["in"], gen))
    return {"x_codes": x_codes, "x_scales": x_scales, "w_codes": w_codes, "w_scales": w_scales,
            "y": torch.empty(case["rows"], case["out"], dtype=_dtype(case["y"]), device="cuda")}


def _verify_inputs(case, gen):
    b, k, vocab, t = case["requests"], case["drafts"], case["vocab"], case["temperature"]
    dtype = _dtype(case["dtype"])
    # target logits: a wide floor and 16 likely tokens a row; the draft model's are these with noise
    target = torch.empty(b * (k + 1), vocab, device="cuda").normal_(0.0, 2.0, generator=gen)
    ids = torch.randint(0, vocab, (b * (k + 1), 16), device="cuda", generator=gen)
    target.scatter_(1, ids, torch.empty(b * (k + 1), 16, device="cuda").normal_(11.0, 3.0, generator=gen))
    target = target.to(dtype)
    noise = torch.empty(b * k, vocab, device="cuda").normal_(0.0, 0.7, generator=gen)
    draft = (target.view(b, k + 1, vocab)[:, :k].reshape(b * k, vocab).float() + noise).to(dtype)
    del noise
    # tokens drawn from the draft model: the largest of its logits with Gumbel noise
    gumbel = -torch.log(torch.empty(b * k, vocab, device="cuda").exponential_(generator=gen))
    tokens = (draft.float() / t + gumbel).argmax(dim=1).to(torch.int32).view(b, k)
    lens = torch.full((b,), k, dtype=torch.int32, device="cuda")
    if b > 4:  # some requests come with fewer drafted tokens
        short = torch.randint(0, k + 1, (b,), device="cuda", generator=gen, dtype=torch.int32)
        lens = torch.where(torch.rand(b, device="cuda", generator=gen) < 0.25, short, lens)
    state = {"target": target, "tokens": tokens, "lens": lens,
             "uniforms": torch.rand(b, k + 1, device="cuda", generator=gen),
             "accepted": torch.empty(b, dtype=torch.int32, device="cuda"),
             "out": torch.empty(b, k + 1, dtype=torch.int32, device="cuda"),
             "logprobs": torch.empty(b, k + 1, device="cuda")}
    if case["draft_logits"]:
        state["draft"] = draft
    if own:
        import fsdp_sharded_mixed_flatten_amd as zs
        state["workspace"] = torch.empty(zs.zs_verify_drafts_workspace_bytes(b, k, vocab), dtype=torch.uint8,
                                         device="cuda")
    return state


def _pieces_inputs(case, gen):
    lens = _piece_lens(case)
    n = sum(lens)
    state = {"grad": torch.empty(n, dtype=torch.bfloat16, device="cuda").normal_(0.0, 1e-3, generator=gen),
             "sumsq": torch.empty(1, dtype=torch.float64, device="cuda"),
             "nonfinite": torch.empty(1, dtype=torch.int32, device="cuda"),
             "scale": torch.empty(1, device="cuda"), "skip": torch.empty(1, dtype=torch.int32, device="cuda")}
    if case["kind"] == "clip_step":  # the state that a first step of gradients of this size leaves
        state["master"] = torch.empty(n, device="cuda").normal_(0.0, 0.02, generator=gen)
        state["m"] = torch.empty(n, device="cuda").normal_(0.0, 1e-4, generator=gen)
        state["v"] = torch.empty(n, device="cuda").normal_(0.0, 1e-3, generator=gen).square_().mul_(0.05)
        state["param"] = state["master"].to(torch.bfloat16)
    if own:
        import fsdp_sharded_mixed_flatten_amd as zs
        state["plan"] = zs.zs_shard_plan_ex(_shape_numels(case["shape"]), case["world"], 0,
                                            persist_below_elems=case["persist_below"])
        names = [name for name in ("grad", "master", "m", "v", "param") if name in state]
        views = {name: state[name].split(lens) for name in names}
        state["workspace"] = torch.zeros(zs.zs_multi_workspace_bytes(state["plan"], 0), dtype=torch.uint8,
                                         device="cuda")
        zs.zs_multi_bind(state["plan"], [{name: views[name][i] for name in names} for i in range(len(lens))], None,
                         state["workspace"])
        state["stats"] = torch.empty(zs.zs_grad_stats_multi_workspace_bytes(state["plan"]), dtype=torch.uint8,
                                     device="cuda")
        state["hp"] = zs.AdamWHParams(**ADAMW)
    return state


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    make = {"mx4_round": _round_inputs, "mx4_matmul": _matmul_inputs, "verify": _verify_inputs,
            "norm": _pieces_inputs, "clip_step": _pieces_inputs}[case["kind"]]
    state = make(case, gen)
    state["case"] = dict(case)
    return state


# ---------------------------------------------------------------- one pass


def run(state):
    kind = state["case"]["kind"]
    if own:
        return _OWN[kind](state)
    return _PLAIN[kind](state)


def _plain_round(state):
    codes, scales = _mx4_codes(state["x"])
    return _mx4_values(codes, scales)[:, :state["case"]["cols"]].to(state["x"].dtype)


def _plain_matmul(state):
    x = _mx4_values(state["x_codes"], state["x_scales"])
    w = _mx4_values(state["w_codes"], state["w_scales"])
    return torch.matmul(x, w.t()).to(state["y"].dtype)


def _plain_verify(state):
    case = state["case"]
    b, k, vocab, t = case["requests"], case["drafts"], case["vocab"], case["temperature"]
    tokens, lens, u = state["tokens"].long(), state["lens"].long(), state["uniforms"].double()
    rows, places = torch.arange(b, device=u.device), torch.arange(k + 1, device=u.device)

    def softmax(z):  # in 64 bits: tokens are drawn where a sum over the vocabulary passes a border
        d = (z.double() - z.amax(dim=-1, keepdim=True).double()) / t
        e = torch.exp(d)
        return e / e.sum(dim=-1, keepdim=True)

    p = softmax(state["target"].view(b, k + 1, vocab))
    at = p[:, :k].gather(2, tokens[:, :, None])[:, :, 0]
    if case["draft_logits"]:
        q = softmax(state["draft"].view(b, k, vocab))
        taken = u[:, :k] * q.gather(2, tokens[:, :, None])[:, :, 0] < at
    else:
        taken = u[:, :k] < at
    n = (taken & (places[:k] < lens[:, None])).long().cumprod(dim=1).sum(dim=1)
    refused = n < lens
    last = p[rows, n]
    i = n.clamp(max=k - 1)
    less = q[rows, i] if case["draft_logits"] else \
        torch.where(torch.arange(vocab, device=u.device) == tokens[rows, i][:, None], math.inf, 0.0)
    rest = torch.where(refused[:, None], (last - less).clamp(min=0.0), last)
    rest = torch.where((rest.sum(dim=1) > 0)[:, None], rest, last)
    total = rest.cumsum(dim=1)
    token = torch.searchsorted(total, total[:, -1:] * u[:, k:], right=True)[:, 0].clamp(max=vocab - 1)
    drafted = torch.cat([tokens, tokens[:, :1]], dim=1)
    out = torch.where(places < n[:, None], drafted, torch.where(places == n[:, None], token[:, None], -1))
    lp = torch.log(p.gather(2, out.clamp(min=0)[:, :, None])[:, :, 0])
    return {"accepted": n.to(torch.int32), "tokens": out.to(torch.int32),
            "logprobs": torch.where(out >= 0, lp, 0.0).float()}


def _plain_norm(state):
    g = state["grad"].double()  # a sum of up to a thousand million squares
    sumsq = (g * g).sum()
    bad = (~torch.isfinite(state["grad"])).any()
    scale = (MAX_NORM / (torch.sqrt(sumsq) + 1e-6)).clamp(max=1.0).float()
    return {"sumsq": sumsq.view(1), "nonfinite": bad.to(torch.int32).view(1), "scale": scale.view(1),
            "skip": bad.to(torch.int32).view(1)}


def _plain_clip_step(state):
    out = _plain_norm(state)
    h = ADAMW
    master, m, v = state["master"], state["m"], state["v"]
    go = out["skip"] == 0
    g = state["grad"].float() * out["scale"]
    m1 = h["beta1"] * m + (1 - h["beta1"]) * g
    v1 = h["beta2"] * v + (1 - h["beta2"]) * (g * g)
    w = master * (1 - h["lr"] * h["weight_decay"])
    w = w - h["lr"] * ((m1 / (1 - h["beta1"] ** h["step"])) /
                       (torch.sqrt(v1 / (1 - h["beta2"] ** h["step"])) + h["eps"]))
    master.copy_(torch.where(go, w, master))
    m.copy_(torch.where(go, m1, m))
    v.copy_(torch.where(go, v1, v))
    state["param"].copy_(torch.where(go, w.to(torch.bfloat16), state["param"]))
    return {**out, **{name: state[name] for name in ("master", "m", "v", "param")}}


_PLAIN = {"mx4_round": _plain_round, "mx4_matmul": _plain_matmul, "verify": _plain_verify, "norm": _plain_norm,
          "clip_step": _plain_clip_step}


def _own_round(state):
    import fsdp_sharded_mixed_flatten_amd as zs
    zs.zs_mx4_quantize(state["x"], state["codes"], state["scales"])
    zs.zs_mx4_dequantize(state["codes"], state["scales"], state["y"])
    return state["y"]


def _own_matmul(state):
    import fsdp_sharded_mixed_flatten_amd as zs
    zs.zs_mx4_matmul(state["x_codes"], state["x_scales"], state["w_codes"], state["w_scales"], state["y"])
    return state["y"]


def _own_verify(state):
    import fsdp_sharded_mixed_flatten_amd as zs
    zs.zs_verify_drafts(state["target"], state["tokens"], state["uniforms"], state["accepted"], state["out"],
                        state["workspace"], draft_logits=state.get("draft"), draft_lens=state["lens"],
                        logprobs=state["logprobs"], temperature=state["case"]["temperature"])
    return {"accepted": state["accepted"], "tokens": state["out"], "logprobs": state["logprobs"]}


def _own_norm(state):
    import fsdp_sharded_mixed_flatten_amd as zs
    zs.zs_grad_stats_multi(state["plan"], state["sumsq"], state["nonfinite"], state["workspace"], state["stats"])
    zs.zs_clip_scale(state["sumsq"], state["nonfinite"], MAX_NORM, state["scale"], state["skip"])
    return {name: state[name] for name in ("sumsq", "nonfinite", "scale", "skip")}


def _own_clip_step(state):
    import fsdp_sharded_mixed_flatten_amd as zs
    out = _own_norm(state)
    zs.zs_adamw_shard_step_multi_clip(state["plan"], [state["hp"]], state["workspace"], scale=state["scale"],
                                      skip=state["skip"])
    return {**out, **{name: state[name] for name in ("master", "m", "v", "param")}}


_OWN = {"mx4_round": _own_round, "mx4_matmul": _own_matmul, "verify": _own_verify, "norm": _own_norm,
        "clip_step": _own_clip_step}


# ---------------------------------------------------------------- what a pass cannot do without


def work(case):
    kind = case["kind"]
    if kind == "mx4_round":
        # the matrix in, codes and scales out and in again, the matrix out
        n, esz = case["rows"] * case["cols"], 2 if case["dtype"] == "bf16" else 4
        return {"bytes": n * (2 * esz + 2 * 17 / 32), "flops": 4 * n}
    if kind == "mx4_matmul":
        rows, n_in, out = case["rows"], case["in"], case["out"]
        return {"bytes": (rows + out) * n_in * 17 / 32 + rows * out * (2 if case["y"] == "bf16" else 4),
                "flops": 2 * rows * n_in * out}
    if kind == "verify":
        # every row once: how many a request needs shows only when they have been read
        n = case["requests"] * (case["drafts"] + 1 + (case["drafts"] if case["draft_logits"] else 0)) * case["vocab"]
        return {"bytes": n * (2 if case["dtype"] == "bf16" else 4) + case["requests"] * (case["drafts"] + 1) * 16,
                "flops": 20 * n}
    n = sum(_piece_lens(case))
    if kind == "norm":
        return {"bytes": 2 * n + 20, "flops": 2 * n}
    return {"bytes": (2 + 12 + 12 + 2) * n + 20, "flops": 16 * n}


# ---------------------------------------------------------------- the definitions in 64 bits


def exact(case, seed):
    state = prepare(case, seed)
    return {"mx4_round": _exact_round, "mx4_matmul": _exact_matmul, "verify": _exact_verify, "norm": _exact_norm,
            "clip_step": _exact_clip_step}[case["kind"]](case, state)


def _exact_round(case, state):
    """Each element's nearest value of its block's grid, found by comparison with the borders between neighbours."""
    rows, cols = case["rows"], case["cols"]
    out = torch.empty(rows, cols, dtype=torch.float64, device="cuda")
    blocks = -(-cols // 32)
    step = max(1, (CHUNK_ELEMS >> 2) // cols)
    for lo in range(0, rows, step):
        x = torch.zeros(min(step, rows - lo), 32 * blocks, dtype=torch.float64, device="cuda")
        x[:, :cols] = state["x"][lo:lo + step]
        x = x.view(-1, blocks, 32)
        amax = x.abs().amax(dim=2, keepdim=True)
        unit = torch.exp2((torch.floor(torch.log2(amax.clamp(min=1e-300))) - 2).clamp(min=-127.0))
        a = x.abs() / unit
        v = torch.zeros_like(a)
        # a border itself belongs to the neighbour whose last bit is 0: 0, 1, 2 and 4
        for low, high, even_low in ((0.0, 0.5, True), (0.5, 1.0, False), (1.0, 1.5, True), (1.5, 2.0, False),
                                    (2.0, 3.0, True), (3.0, 4.0, False), (4.0, 6.0, True)):
            border = (low + high) / 2
            v = torch.where(a > border if even_low else a >= border, high, v)
        out[lo:lo + step] = (torch.sign(x) * v * unit).view(-1, 32 * blocks)[:, :cols]
    return out


def _exact_values(codes, scales):
    c = torch.stack([codes % 16, codes // 16], dim=2).flatten(1).double()
    sign, c = torch.where(c >= 8, -1.0, 1.0), c % 8
    e = torch.floor(c / 2)
    v = torch.where(e == 0, c % 2 / 2, torch.exp2(e - 1) * (1 + c % 2 / 2))
    return sign * v * torch.exp2(scales.double() - 127).repeat_interleave(32, dim=1)


def _exact_matmul(case, state):
    x = _exact_values(state["x_codes"], state["x_scales"])
    y = torch.empty(case["rows"], case["out"], dtype=torch.float64, device="cuda")
    step = max(1, (CHUNK_ELEMS >> 1) // case["in"])
    for lo in range(0, case["out"], step):
        w = _exact_values(state["w_codes"][lo:lo + step], state["w_scales"][lo:lo + step])
        y[:, lo:lo + step] = x @ w.t().contiguous()
    return y


def _exact_verify(case, state):
    """Request by request, draft by draft, as the method is told."""
    k, t = case["drafts"], case["temperature"]
    lens, tokens, u = state["lens"].tolist(), state["tokens"].tolist(), state["uniforms"].double().tolist()
    got = {"accepted": [], "tokens": [], "logprobs": []}
    for b in range(case["requests"]):
        out, lps, token = [], [], None
        for i in range(lens[b] + 1):
            lp = torch.log_softmax(state["target"][b * (k + 1) + i].double() / t, dim=0)
            rest = lp.exp()
            if i < lens[b]:
                x = tokens[b][i]
                if case["draft_logits"]:
                    q = torch.softmax(state["draft"][b * k + i].double() / t, dim=0)
                else:
                    q = torch.zeros_like(rest)
                    q[x] = 1.0
                if u[b][i] * float(q[x]) < float(rest[x]):
                    out.append(x)
                    lps.append(float(lp[x]))
                    continue
                rest = (rest - q).clamp(min=0.0)
            total = rest.cumsum(dim=0)
            token = int((total <= u[b][k] * float(total[-1])).sum())
            break
        got["accepted"].append(len(out))
        got["tokens"].append(out + [token] + [-1] * (k - len(out)))
        got["logprobs"].append(lps + [float(lp[token])] + [0.0] * (k - len(out)))
    return {"accepted": torch.tensor(got["accepted"], dtype=torch.int32),
            "tokens": torch.tensor(got["tokens"], dtype=torch.int32),
            "logprobs": torch.tensor(got["logprobs"], dtype=torch.float64)}


def _exact_norm(case, state):
    norm = torch.linalg.vector_norm(state["grad"], dtype=torch.float64)
    scale = torch.minimum(torch.ones_like(norm), MAX_NORM / (norm + 1e-6))
    zero = torch.zeros(1, dtype=torch.int32)
    return {"sumsq": (norm * norm).view(1), "nonfinite": zero, "scale": scale.view(1), "skip": zero}


def _exact_clip_step(case, state):
    out = _exact_norm(case, state)
    h, parts = ADAMW, []
    for g, w, m, v in zip(*(state[name].split(CHUNK_ELEMS >> 1) for name in ("grad", "master", "m", "v"))):
        g = g.double() * out["scale"]
        m1 = m.double() + (1 - h["beta1"]) * (g - m)
        v1 = v.double() + (1 - h["beta2"]) * (g.square() - v)
        root = (v1 / (1 - h["beta2"] ** h["step"])).sqrt() + h["eps"]
        w1 = w.double() - h["lr"] * (h["weight_decay"] * w.double() + m1 / (1 - h["beta1"] ** h["step"]) / root)
        parts.append((w1, m1, v1))
    master, m, v = (torch.cat(p) for p in zip(*parts))
    return {**out, "master": master, "m": m, "v": v, "param": master.clone()}
