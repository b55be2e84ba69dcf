"""Plain 64-bit implementations of the language-model operators, written from
their definitions: the oracle the tests compare the kernels with. Row by
row in numpy, no vector tricks shared with the library.
"""
import math

import numpy as np


def bf16_to_f64(bits):
    """float64 values of bf16 bit patterns (uint16)."""
    return (np.asarray(bits, np.uint16).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


# ---------------------------------------------------------------- products with the quantized gather


def decode_codes(codes_all, bits):
    """Integers of a payload's code bytes (4 bits: the even element in the low nibble; two's complement)."""
    b = np.asarray(codes_all, np.uint8)
    if bits == 8:
        return b.view(np.int8).astype(np.int64)
    c = np.empty(2 * b.size, np.int64)
    c[0::2] = b & 15
    c[1::2] = b >> 4
    return np.where(c > 7, c - 16, c)


def quant_weights(codes_all, scales_all, bits, block, shard, n_scales, off, n_out, n_in):
    """The weight matrix [n_out, n_in] in float64: code * scale of its own shard's block."""
    j = off + np.arange(n_out * n_in, dtype=np.int64)
    scale = np.asarray(scales_all, np.float32)[j // shard * n_scales + j % shard // block]
    return (decode_codes(codes_all, bits)[j] * scale.astype(np.float64)).reshape(n_out, n_in)


def quant_matvec(w, x):
    """(y, sum of |w x|): [rows, n_out] each; the second is what a rounding bound is relative to."""
    x = np.asarray(x, np.float64)
    with np.errstate(invalid="ignore"):
        return x @ w.T, np.abs(x) @ np.abs(w.T)


# ---------------------------------------------------------------- log-probabilities


def row_softmax(x, temperature):
    """(max, log s, log-probabilities) of one row of float64 logits; a row of -infinity only gives (-inf, 0, -inf ...),
    one that holds a NaN or +infinity NaN."""
    if np.isnan(x).any() or np.isposinf(x).any():
        return math.nan, math.nan, np.full(x.shape, math.nan)
    m = x.max()
    if m == -math.inf:
        return m, 0.0, np.full(x.shape, -math.inf)
    d = (x - m) / temperature
    logs = math.log(math.fsum(np.exp(d)))
    return m, logs, d - logs


def token_logprobs(logits, tokens, temperature=1.0, top=0):
    """dict of logprob, entropy, stats, top_ids, top_logprobs for float64 logits [rows, vocab]."""
    rows, vocab = logits.shape
    out = {"logprob": np.zeros(rows), "entropy": np.zeros(rows), "stats": np.zeros((rows, 2)),
           "top_ids": np.full((rows, top), -1, np.int64), "top_logprobs": np.zeros((rows, top))}
    for r in range(rows):
        if tokens[r] < 0:
            continue
        m, logs, lp = row_softmax(logits[r], temperature)
        p = np.exp(lp)
        out["stats"][r] = m, logs
        out["logprob"][r] = lp[tokens[r]] if tokens[r] < vocab else math.nan
        if m == -math.inf:
            out["entropy"][r] = 0.0
        else:
            seen = ~(p == 0.0)
            out["entropy"][r] = -math.fsum(p[seen] * lp[seen]) if not math.isnan(m) else math.nan
        if math.isnan(m):
            out["top_logprobs"][r] = math.nan
        else:
            order = np.lexsort((np.arange(vocab), -logits[r]))[:top]
            out["top_ids"][r] = order
            out["top_logprobs"][r] = lp[order]
    return out


def token_logprobs_backward(logits, tokens, temperature, grad_logprob, grad_entropy=None):
    """(gradient, magnitude of its terms before they cancel), float64 [rows, vocab]."""
    rows, vocab = logits.shape
    g, mag = np.zeros((rows, vocab)), np.zeros((rows, vocab))
    for r in range(rows):
        if tokens[r] < 0:
            continue
        m, _, lp = row_softmax(logits[r], temperature)
        if m == -math.inf:
            continue
        if math.isnan(m) or tokens[r] >= vocab:
            g[r] = math.nan
            continue
        p = np.exp(lp)
        l = np.where(p == 0.0, 0.0, lp)
        gl = float(grad_logprob[r])
        gh = 0.0 if grad_entropy is None else float(grad_entropy[r])
        h = -math.fsum(p * l)
        g[r] = -p * (gl + gh * (l + h))
        mag[r] = p * (abs(gl) + abs(gh) * (np.abs(l) + h))
        g[r, tokens[r]] += gl
        mag[r, tokens[r]] += abs(gl)
    return g / temperature, mag / temperature


# ---------------------------------------------------------------- distillation


def distill_topk(logits, ids, teacher, temperature=1.0, row_weight=None):
    """(loss [rows], magnitude of the loss's terms, gradient, magnitude of its terms), float64."""
    rows, vocab = logits.shape
    loss, lmag = np.zeros(rows), np.zeros(rows)
    g, mag = np.zeros((rows, vocab)), np.zeros((rows, vocab))
    t2 = temperature * temperature
    for r in range(rows):
        w = 1.0 if row_weight is None else float(row_weight[r])
        used = [(int(i), float(v)) for i, v in zip(ids[r], teacher[r]) if i >= 0]
        bad = any(i >= vocab or math.isnan(v) or v == math.inf for i, v in used)
        if w == 0.0 or (not bad and all(v == -math.inf for _, v in used)):
            continue
        m, _, lp = row_softmax(logits[r], temperature)
        if bad or math.isnan(m):
            loss[r], g[r] = math.nan, math.nan
            continue
        top = max(v for _, v in used)
        e = [math.exp((v - top) / temperature) for _, v in used]
        s = math.fsum(e)
        p = np.exp(lp)
        g[r] = mag[r] = p
        terms = []
        for (i, v), x in zip(used, e):
            q = x / s
            if q == 0.0:
                continue
            logq = (v - top) / temperature - math.log(s)
            terms.append(q * (logq - lp[i]))
            lmag[r] += q * (abs(logq) + abs(lp[i]))
            g[r, i] -= q
            mag[r, i] += q
        loss[r] = w * t2 * (math.inf if any(math.isinf(x) for x in terms) else math.fsum(terms))
        lmag[r] *= abs(w) * t2
        g[r] *= w * temperature
        mag[r] *= abs(w) * temperature
    return loss, lmag, g, mag
