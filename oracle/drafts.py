"""Plain 64-bit implementation of the verification of drafted tokens, request by request and token by token: the oracle
the tests compare the kernels with."""
import math

import numpy as np


def softmax(z, temperature):
    """Probabilities of a row of logits; None where a NaN or +infinity is among them, zeros where all are -infinity."""
    z = np.asarray(z, np.float64)
    if np.isnan(z).any() or np.isposinf(z).any():
        return None
    top = z.max()
    if top == -math.inf:
        return np.zeros_like(z)
    e = np.exp((z - top) / temperature)
    return e / math.fsum(e)


def draw(share, u):
    """The lowest index whose running sum exceeds u times the sum of all, among those with a share; the last of these
    where none does."""
    border = float(u) * math.fsum(share)
    run, last = 0.0, -1
    for j in np.flatnonzero(share > 0):
        run += share[j]
        last = int(j)
        if not run <= border:
            return last
    return last


def verify(target, draft, tokens, lens, uniforms, temperature=1.0):
    """(accepted [requests], tokens, logprobs [requests, drafts + 1]) for target logits [requests, drafts + 1, vocab],
    draft logits [requests, drafts, vocab] or None, and lens or None."""
    requests, places, vocab = target.shape
    k = places - 1
    accepted, out = np.zeros(requests, np.int32), np.full((requests, places), -1, np.int32)
    lps = np.zeros((requests, places))
    for b in range(requests):
        n = k if lens is None else min(int(lens[b]), k)
        for i in range(n + 1 if n >= 0 else 0):
            accepted[b] = i
            p = softmax(target[b, i], temperature)
            if p is None or p.sum() == 0:
                lps[b, i] = math.nan
                break
            share = p
            if i < n:
                x = int(tokens[b, i])
                q = np.zeros(vocab)
                if draft is not None:
                    q = softmax(draft[b, i], temperature)
                    if q is None:
                        lps[b, i] = math.nan
                        break
                elif 0 <= x < vocab:
                    q[x] = 1.0
                if 0 <= x < vocab and float(uniforms[b, i]) * q[x] < p[x]:
                    out[b, i], lps[b, i] = x, math.log(p[x])
                    continue
                share = np.maximum(p - q, 0.0)
                if share.sum() == 0:
                    share = p
            out[b, i] = draw(share, uniforms[b, k])
            lps[b, i] = math.log(p[out[b, i]])
            break
    return accepted, out, lps
