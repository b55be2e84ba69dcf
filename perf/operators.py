"""The language-model operators of the library as cases to be timed and checked: products with the quantized gathered
parameters, token log-probabilities with their gradient, and distillation from a teacher's top logits.

`run` computes a case in elementary torch operations in 32 bits, or, with `own` set, with the library's entry points.
`exact` computes the same outputs from the operators' definitions in 64 bits.
"""
import math

import torch

own = False

CHUNK_ELEMS = 1 << 27  # elements of one chunk of the 64-bit computation


def listed():
    return [
        # one token of a rollout through an attention projection of the Llama-7B shape, 8 ranks' payload: the smallest call
        {"name": "matvec4_one_4096", "kind": "matvec", "rows": 1, "out": 4096, "in": 4096, "bits": 4, "block": 128,
         "world": 8, "y": "bf16"},
        # one token through the Llama-70B shape's down projection: the ordinary long product
        {"name": "matvec4_one_down", "kind": "matvec", "rows": 1, "out": 8192, "in": 28672, "bits": 4, "block": 128,
         "world": 8, "y": "bf16"},
        # 16 rollouts side by side through a Qwen2.5-3B up projection, small groups
        {"name": "matvec4_batch16", "kind": "matvec", "rows": 16, "out": 11008, "in": 2048, "bits": 4, "block": 32,
         "world": 4, "y": "bf16"},
        # sizes no group or shard boundary falls in line with (an expert or adapter of odd width), 3 tokens
        {"name": "matvec4_odd", "kind": "matvec", "rows": 3, "out": 5003, "in": 1531, "bits": 4, "block": 64,
         "world": 3, "y": "f32"},
        # the LM head of the Llama-70B shape in 8 bits for 4 tokens, logits in fp32: the largest product
        {"name": "matvec8_head", "kind": "matvec", "rows": 4, "out": 128256, "in": 8192, "bits": 8, "block": 128,
         "world": 8, "y": "f32"},
        # scoring one sampled token of a 32000-token vocabulary with its 5 best alternatives: latency
        {"name": "logprobs_one", "kind": "logprobs", "rows": 1, "vocab": 32000, "dtype": "bf16", "top": 5,
         "temperature": 1.0},
        # a batch of rollouts at one position, fp32 logits of the Qwen2.5-3B vocabulary, 20 alternatives, sampled at 0.7
        {"name": "logprobs_batch_f32", "kind": "logprobs", "rows": 64, "vocab": 151936, "dtype": "f32", "top": 20,
         "temperature": 0.7},
        # scoring whole sequences for an on-policy update, 128256 tokens: the largest forward
        {"name": "logprobs_long", "kind": "logprobs", "rows": 4096, "vocab": 128256, "dtype": "bf16", "top": 8,
         "temperature": 1.0},
        # the update's gradient, with an entropy bonus
        {"name": "logprobs_grad", "kind": "logprobs_grad", "rows": 2048, "vocab": 151936, "dtype": "bf16",
         "temperature": 1.0, "entropy": True},
        # the same in fp32 with a vocabulary that no vector width divides, without the bonus
        {"name": "logprobs_grad_odd", "kind": "logprobs_grad", "rows": 333, "vocab": 50007, "dtype": "f32",
         "temperature": 0.9, "entropy": False},
        # distilling a training micro-batch from a teacher's 64 best logits: loss and gradient in one call
        {"name": "distill_batch", "kind": "distill", "rows": 4096, "vocab": 128256, "dtype": "bf16", "k": 64,
         "temperature": 2.0},
        # fp32 logits, odd vocabulary, more teacher entries, few rows
        {"name": "distill_odd_f32", "kind": "distill", "rows": 301, "vocab": 100003, "dtype": "f32", "k": 200,
         "temperature": 1.0},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["matvec", "matvec", "logprobs", "logprobs_grad", "distill"])
    if kind == "matvec":
        odd = rng.random() < 0.3
        bits = rng.choice([4, 4, 8])
        most = 1 << 27 if odd else 1 << 29
        n_in = _log_int(rng, 512, 28672)
        n_out = _log_int(rng, 256, min(128256, most // n_in))
        if odd:
            n_in, n_out = n_in | 1, n_out | 1
        else:
            n_in, n_out = max(512, n_in // 256 * 256), max(256, n_out // 16 * 16)
        return {"kind": kind, "rows": _log_int(rng, 1, 64), "out": n_out, "in": n_in, "bits": bits,
                "block": rng.choice([16, 32, 64, 128, 128, 256]), "world": rng.choice([1, 2, 3, 4, 8]),
                "y": rng.choice(["bf16", "f32"])}
    vocab = _log_int(rng, 2000, 152000)
    if rng.random() < 0.5:
        vocab = vocab // 128 * 128
    case = {"kind": kind, "rows": _log_int(rng, 1, min(4096, (1 << 28) // vocab)), "vocab": vocab,
            "dtype": rng.choice(["bf16", "f32"]), "temperature": rng.choice([0.6, 0.8, 1.0, 1.0, 1.5, 2.0])}
    if kind == "logprobs":
        case["top"] = rng.choice([0, 1, 5, 8, 20, 32])
    elif kind == "logprobs_grad":
        case["entropy"] = rng.random() < 0.5
    else:
        case["k"] = _log_int(rng, 1, 512)
    return case


# ---------------------------------------------------------------- inputs


def _dtype(name):
    return {"bf16": torch.bfloat16, "f32": torch.float32}[name]


def _layout(case):
    """Flat offset of the matrix, shard length and scales a shard: a unit of a norm's weight and the matrix, tensor
    starts aligned to 128 elements, the length padded to 8 elements a rank."""
    off = -(-case["in"] // 128) * 128
    unit = 8 * case["world"]
    shard = -(-(off + case["out"] * case["in"]) // unit) * 8
    return off, shard, -(-shard // case["block"])


def _matvec_inputs(case, gen):
    off, shard, n_scales = _layout(case)
    n, bits, block, world = case["out"] * case["in"], case["bits"], case["block"], case["world"]
    qmax = 7 if bits == 4 else 127
    codes = torch.empty(world, shard * bits // 8, dtype=torch.uint8, device="cuda")
    scales = torch.empty(world, n_scales, dtype=torch.float32, device="cuda")
    for q in range(world):  # each rank quantizes its shard of weights of standard deviation 0.02
        w = torch.zeros(n_scales * block, device="cuda")
        w[:shard].normal_(0.0, 0.02, generator=gen)
        if off + n < (q + 1) * shard:
            w[max(0, off + n - q * shard):] = 0
        w = w.to(torch.bfloat16).float().view(n_scales, block)
        s = w.abs().amax(dim=1) / qmax
        c = torch.round(w / torch.where(s > 0, s, 1.0)[:, None]).clamp_(-qmax, qmax).to(torch.int32).view(-1)[:shard]
        codes[q] = ((c[0::2] & 15) | ((c[1::2] & 15) << 4) if bits == 4 else c & 255).to(torch.uint8)
        scales[q] = s
    x = torch.empty(case["rows"], case["in"], device="cuda").normal_(0.0, 1.0, generator=gen).to(torch.bfloat16)
    state = {"codes": codes.view(-1), "scales": scales.view(-1), "x": x,
             "y": torch.empty(case["rows"], case["out"], dtype=_dtype(case["y"]), device="cuda")}
    if own:
        import fsdp_sharded_mixed_flatten_amd as zs
        state["plan"] = zs.zs_shard_plan([case["in"], n], world, 0, tensor_align_elems=128)
    return state


def _peaked_logits(case, gen, ids, heights):
    """Logits of a language model: a wide floor and, at `ids` of each row, the tokens it thinks likely."""
    z = torch.empty(case["rows"], case["vocab"], device="cuda").normal_(0.0, 2.0, generator=gen)
    z.scatter_(1, ids, heights)
    return z.to(_dtype(case["dtype"]))


def _distinct_ids(rows, k, vocab, gen):
    step = max(1, vocab // k)
    gaps = torch.randint(1, step + 1, (rows, k), device="cuda", generator=gen)
    return (torch.randint(0, vocab, (rows, 1), device="cuda", generator=gen) + gaps.cumsum(1)) % vocab


def _logprobs_inputs(case, gen):
    rows, vocab = case["rows"], case["vocab"]
    ids = _distinct_ids(rows, 16, vocab, gen)
    heights = torch.empty(rows, 16, device="cuda").normal_(9.0, 3.0, generator=gen)
    state = {"logits": _peaked_logits(case, gen, ids, heights)}
    pick = torch.randint(0, 16, (rows, 1), device="cuda", generator=gen)
    tokens = ids.gather(1, pick).view(-1).to(torch.int32)
    if rows > 8:  # positions behind the end of a finished rollout
        tokens[torch.rand(rows, device="cuda", generator=gen) < 0.06] = -1
    state["tokens"] = tokens
    return state


def _row_stats(z, temperature):
    """Largest logit, log of the sum and entropy of softmax(z / temperature), in z's precision."""
    top = z.amax(dim=1)
    d = (z - top[:, None]) / temperature
    e = torch.exp(d)
    s = e.sum(dim=1)
    return top, torch.log(s), torch.log(s) - (e * d).sum(dim=1) / s


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    kind = case["kind"]
    if kind == "matvec":
        state = _matvec_inputs(case, gen)
    elif kind == "distill":
        rows, k, vocab = case["rows"], case["k"], case["vocab"]
        ids = _distinct_ids(rows, k, vocab, gen)
        teacher = torch.empty(rows, k, device="cuda").normal_(4.0, 3.0, generator=gen).sort(dim=1, descending=True)[0]
        noise = torch.empty(rows, k, device="cuda").normal_(0.0, 1.5, generator=gen)
        kept = torch.randint((k + 1) // 2, k + 1, (rows, 1), device="cuda", generator=gen)
        weight = torch.full((rows,), 1.0 / rows, device="cuda")
        if rows > 8:  # prompt positions carry no loss
            weight[torch.rand(rows, device="cuda", generator=gen) < 0.1] = 0.0
        state = {"logits": _peaked_logits(case, gen, ids, teacher + noise), "weight": weight, "teacher": teacher,
                 "ids": torch.where(torch.arange(k, device="cuda") < kept, ids, -1).to(torch.int32)}
        state["loss"] = torch.empty(rows, device="cuda")
        state["grad"] = torch.empty_like(state["logits"])
    else:
        state = _logprobs_inputs(case, gen)
        rows = case["rows"]
        live = state["tokens"] >= 0
        if kind == "logprobs":
            for name in ("logprob", "entropy"):
                state[name] = torch.empty(rows, device="cuda")
            state["stats"] = torch.empty(rows, 2, device="cuda")
            if case["top"]:
                state["top_ids"] = torch.empty(rows, case["top"], dtype=torch.int32, device="cuda")
                state["top_logprobs"] = torch.empty(rows, case["top"], device="cuda")
        else:  # what the forward pass left, and the gradients that a loss over the rows sends back
            parts = [_row_stats(z.float(), case["temperature"]) for z in state["logits"].split(512)]
            top, logsum, entropy = (torch.cat(p) for p in zip(*parts))
            state["stats"] = torch.where(live[:, None], torch.stack([top, logsum], dim=1), 0.0)
            state["entropy"] = torch.where(live, entropy, 0.0)
            state["grad_logprob"] = torch.empty(rows, device="cuda").normal_(0.0, 1.0 / rows, generator=gen)
            if case["entropy"]:
                state["grad_entropy"] = torch.full((rows,), -0.01 / rows, device="cuda")
            state["grad"] = torch.empty_like(state["logits"])
    state["case"] = dict(case)
    return state


# ---------------------------------------------------------------- one pass


def run(state):
    kind = state["case"]["kind"]
    if own:
        return _OWN[kind](state)
    return _PLAIN[kind](state)


def _plain_matvec(state):
    case = state["case"]
    off, shard, n_scales = _layout(case)
    b = state["codes"]
    if case["bits"] == 4:
        c = torch.stack([b & 15, b >> 4], dim=1).view(case["world"], shard).to(torch.int8)
        c = torch.where(c > 7, c - 16, c)
    else:
        c = b.view(torch.int8).view(case["world"], shard)
    s = state["scales"].view(case["world"], n_scales).repeat_interleave(case["block"], dim=1)[:, :shard]
    w = (c.float() * s).view(-1)[off:off + case["out"] * case["in"]].view(case["out"], case["in"])
    return torch.matmul(state["x"].float(), w.t()).to(state["y"].dtype)


def _plain_logprobs(state):
    case, tokens = state["case"], state["tokens"]
    z, live = state["logits"].float(), tokens >= 0
    top, logsum, entropy = _row_stats(z, case["temperature"])
    at = z.gather(1, tokens.clamp(min=0).long()[:, None])[:, 0]
    out = {"logprob": torch.where(live, (at - top) / case["temperature"] - logsum, 0.0),
           "entropy": torch.where(live, entropy, 0.0),
           "stats": torch.where(live[:, None], torch.stack([top, logsum], dim=1), 0.0)}
    if case["top"]:
        # the largest logits, the lower index first among equals: order by value, then by index, as one integer
        bits = (z + 0.0).view(torch.int32)
        rank = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).long() * (1 << 32)
        rank += torch.arange(case["vocab"] - 1, -1, -1, device=z.device)
        ids = case["vocab"] - 1 - (torch.topk(rank, case["top"], dim=1)[0] & 0xFFFFFFFF)
        lp = (z.gather(1, ids) - top[:, None]) / case["temperature"] - logsum[:, None]
        out["top_ids"] = torch.where(live[:, None], ids, -1).to(torch.int32)
        out["top_logprobs"] = torch.where(live[:, None], lp, 0.0)
    return out


def _plain_logprobs_grad(state):
    case, tokens = state["case"], state["tokens"]
    live = tokens >= 0
    top, logsum = state["stats"][:, :1], state["stats"][:, 1:]
    lp = (state["logits"].float() - top) / case["temperature"] - logsum
    p = torch.exp(lp)
    g = p * -state["grad_logprob"][:, None]
    if case["entropy"]:
        g -= state["grad_entropy"][:, None] * p * (lp + state["entropy"][:, None])
    g.scatter_add_(1, tokens.clamp(min=0).long()[:, None], state["grad_logprob"][:, None])
    return torch.where(live[:, None], g / case["temperature"], 0.0).to(state["logits"].dtype)


def _plain_distill(state):
    case, ids, t = state["case"], state["ids"], state["case"]["temperature"]
    kept = ids >= 0
    q = torch.exp(torch.where(kept, (state["teacher"] - state["teacher"].amax(dim=1, keepdim=True)) / t, -math.inf))
    q = q / q.sum(dim=1, keepdim=True)
    z = state["logits"].float()
    top, logsum, _ = _row_stats(z, t)
    at = ids.clamp(min=0).long()
    lp = (z.gather(1, at) - top[:, None]) / t - logsum[:, None]
    loss = state["weight"] * t * t * torch.where(q > 0, q * (torch.log(q) - lp), 0.0).sum(dim=1)
    g = torch.exp((z - top[:, None]) / t - logsum[:, None])
    g.scatter_add_(1, at, -q)
    return {"loss": loss, "grad": (g * (state["weight"] * t)[:, None]).to(state["logits"].dtype)}


_PLAIN = {"matvec": _plain_matvec, "logprobs": _plain_logprobs, "logprobs_grad": _plain_logprobs_grad,
          "distill": _plain_distill}


def _own_matvec(state):
    import fsdp_sharded_mixed_flatten_amd as zs
    case = state["case"]
    zs.zs_quant_matvec(state["plan"], 1, case["out"], case["in"], case["bits"], case["block"], state["codes"],
                       state["scales"], state["x"], state["y"])
    return state["y"]


def _own_logprobs(state):
    import fsdp_sharded_mixed_flatten_amd as zs
    names = ["logprob", "entropy", "stats"] + (["top_ids", "top_logprobs"] if state["case"]["top"] else [])
    out = {name: state[name] for name in names}
    zs.zs_token_logprobs(state["logits"], state["tokens"], temperature=state["case"]["temperature"], **out)
    return out


def _own_logprobs_grad(state):
    import fsdp_sharded_mixed_flatten_amd as zs
    zs.zs_token_logprobs_backward(state["logits"], state["tokens"], state["stats"], state["grad_logprob"],
                                  state["grad"], temperature=state["case"]["temperature"], entropy=state["entropy"],
                                  grad_entropy=state.get("grad_entropy"))
    return state["grad"]


def _own_distill(state):
    import fsdp_sharded_mixed_flatten_amd as zs
    zs.zs_distill_topk(state["logits"], state["ids"], state["teacher"], state["loss"], grad_logits=state["grad"],
                       temperature=state["case"]["temperature"], row_weight=state["weight"])
    return {"loss": state["loss"], "grad": state["grad"]}


_OWN = {"matvec": _own_matvec, "logprobs": _own_logprobs, "logprobs_grad": _own_logprobs_grad,
        "distill": _own_distill}


# ---------------------------------------------------------------- what a pass cannot do without


def work(case):
    if case["kind"] == "matvec":
        n = case["out"] * case["in"]
        y = 2 if case["y"] == "bf16" else 4
        return {"bytes": n * case["bits"] / 8 + n / case["block"] * 4 + 2 * case["rows"] * case["in"]
                + y * case["rows"] * case["out"], "flops": 2 * n * case["rows"]}
    rows, vocab = case["rows"], case["vocab"]
    esz = 2 if case["dtype"] == "bf16" else 4
    if case["kind"] == "logprobs":
        # tokens in; log-probability, entropy, two statistics and the alternatives out
        return {"bytes": rows * (vocab * esz + 4 + 16 + 8 * case["top"]), "flops": 6 * rows * vocab}
    if case["kind"] == "logprobs_grad":
        return {"bytes": rows * (2 * vocab * esz + 4 + 12 + (4 if case["entropy"] else 0)), "flops": 6 * rows * vocab}
    return {"bytes": rows * (2 * vocab * esz + 8 * case["k"] + 8), "flops": 8 * rows * vocab}


# ---------------------------------------------------------------- the definitions in 64 bits


def exact(case, seed):
    state = prepare(case, seed)
    return {"matvec": _exact_matvec, "logprobs": _exact_logprobs, "logprobs_grad": _exact_logprobs_grad,
            "distill": _exact_distill}[case["kind"]](case, state)


def _exact_matvec(case, state):
    off, shard, n_scales = _layout(case)
    bits, n_in = case["bits"], case["in"]
    x = state["x"].double()
    y = torch.empty(case["rows"], case["out"], dtype=torch.float64, device=x.device)
    step = max(1, CHUNK_ELEMS // n_in)
    for lo in range(0, case["out"], step):
        hi = min(lo + step, case["out"])
        j = torch.arange(off + lo * n_in, off + hi * n_in, device=x.device)
        if bits == 4:
            c = (state["codes"][j // 2].long() >> (j % 2 * 4)) % 16
            c -= (c >= 8).long() * 16
        else:
            c = state["codes"][j].long()
            c -= (c >= 128).long() * 256
        s = state["scales"][j // shard * n_scales + j % shard // case["block"]]
        y[:, lo:hi] = x @ (c.double() * s.double()).view(hi - lo, n_in).t()
    return y


def _chunks(case):
    step = max(1, CHUNK_ELEMS // case["vocab"])
    return [slice(lo, min(lo + step, case["rows"])) for lo in range(0, case["rows"], step)]


def _exact_logprobs(case, state):
    parts = []
    for c in _chunks(case):
        raw, token = state["logits"][c], state["tokens"][c].long()
        z = raw.double() / case["temperature"]
        lp = z - torch.logsumexp(z, dim=1, keepdim=True)
        skip = token < 0
        first = raw.double().max(dim=1)[0]
        out = {"logprob": lp[torch.arange(len(token)), token.clamp(min=0)], "entropy": -(lp.exp() * lp).sum(dim=1),
               "stats": torch.stack([first, -lp.max(dim=1)[0]], dim=1)}
        if case["top"]:
            order = raw.float().sort(dim=1, descending=True, stable=True)[1][:, :case["top"]]
            out["top_ids"] = order.to(torch.int32)
            out["top_logprobs"] = lp.gather(1, order)
        for name, v in out.items():
            v[skip] = -1 if name == "top_ids" else 0
        parts.append(out)
    return {name: torch.cat([p[name] for p in parts]) for name in parts[0]}


def _exact_logprobs_grad(case, state):
    g = torch.empty(case["rows"], case["vocab"], dtype=torch.float64, device="cuda")
    for c in _chunks(case):
        token = state["tokens"][c].long()
        lp = (state["logits"][c].double() - state["stats"][c, :1].double()) / case["temperature"] \
            - state["stats"][c, 1:].double()
        delta = torch.arange(case["vocab"], device="cuda") == token[:, None]
        out = state["grad_logprob"][c].double()[:, None] * (delta.double() - lp.exp())
        if case["entropy"]:
            out -= state["grad_entropy"][c].double()[:, None] * lp.exp() * (lp + state["entropy"][c].double()[:, None])
        g[c] = torch.where(token[:, None] < 0, 0.0, out / case["temperature"])
    return g


def _exact_distill(case, state):
    t = case["temperature"]
    g = torch.empty(case["rows"], case["vocab"], dtype=torch.float64, device="cuda")
    loss = torch.empty(case["rows"], dtype=torch.float64, device="cuda")
    for c in _chunks(case):
        ids, w = state["ids"][c].long(), state["weight"][c].double()
        lp = torch.log_softmax(state["logits"][c].double() / t, dim=1)
        logq = torch.log_softmax(torch.where(ids < 0, -math.inf, state["teacher"][c].double() / t), dim=1)
        q = logq.exp()
        loss[c] = w * t * t * (q * torch.where(ids < 0, 0.0, logq - lp.gather(1, ids.clamp(min=0)))).sum(dim=1)
        dense = torch.zeros_like(lp).scatter_add_(1, ids.clamp(min=0), q)
        g[c] = (w * t)[:, None] * (lp.exp() - dense)
    return {"loss": loss, "grad": g}
