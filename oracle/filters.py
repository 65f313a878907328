"""Oracle of filtered rows of logits, float64: what temperature, top-k, top-p
and min-p keep of a row, drawing from it, and the verification rule between two
filtered distributions.

TEST INFRASTRUCTURE ONLY (same rule as the rest of ``oracle/``).

One row at a time, in numpy.  Beside each result it returns a margin: how far
(relative to the total) the decision is from its border, so that a comparison
can leave out what rounding may decide.
"""
from __future__ import annotations

import numpy as np


def kept(z, T=1.0, k=0, p=1.0, least=0.0):
    """z [V] float64 logits (no NaN, no +inf, not all -inf).  Returns (tokens
    ascending, their probabilities, margin of top-p's and min-p's borders)."""
    z = np.asarray(z, dtype=np.float64) + 0.0
    order = np.argsort(-z, kind="stable")
    if T == 0:
        return order[:1], np.ones(1), 1.0
    margin = 1.0
    if 0 < k < len(z):
        order = order[:k]
    with np.errstate(over="ignore"):
        w = np.exp((z[order] - z[order[0]]) / min(max(T, 2.0 ** -100), 2.0 ** 100))
    n = len(order)
    if p < 1:
        head = np.concatenate([[0.0], np.cumsum(w)[:-1]])
        target = max(p, 0.0) * w.sum()
        n = max(1, int((head < target).sum()))
        # equal weights are summed without rounding here and there
        flat = np.all((w == 1) | (w == 0))
        margin = 1.0 if p <= 0 or flat else float(np.abs(head - target).min() / w.sum())
    if least > 0:
        n = max(1, min(n, int((w >= least).sum())))
        if least < 1:
            margin = min(margin, float(np.abs(w - least).min()))
    order, w = order[:n], w[:n]
    at = np.argsort(order)
    return order[at], w[at] / w.sum(), margin


def pick(tokens, w, v):
    """The first token whose running sum exceeds v times the total, and the margin."""
    c = np.cumsum(w)
    i = min(int((c <= v * c[-1]).sum()), len(w) - 1)
    while w[i] == 0:
        i -= 1
    near = np.abs(c[:-1] - v * c[-1])[(c[:-1] > 0) & (c[:-1] < c[-1])]
    return int(tokens[i]), float(near.min() / c[-1]) if len(near) else 1.0


def bad(z, ask):
    T, k, p, least = ask
    if not (T >= 0 and np.isfinite(T)) or np.isnan(p) or not least <= 1:
        return 1
    z = np.asarray(z, dtype=np.float64)
    return 2 if np.isnan(z).any() or (z == np.inf).any() or not (z > -np.inf).any() else 0


def sample(logits, uniforms, asks):
    """logits [B][K][V], uniforms [B][K], asks[b] = (T, top_k, top_p, min_p).
    Returns tokens, prob, margin, code, each [B][K]."""
    B, K, _ = logits.shape
    tokens, code = np.full((B, K), -1), np.zeros((B, K), dtype=int)
    prob, margin = np.full((B, K), np.nan), np.ones((B, K))
    for b in range(B):
        for i in range(K):
            u = float(uniforms[b, i])
            c = bad(logits[b, i], asks[b])
            code[b, i] = 1 if not 0 <= u < 1 else c
            if code[b, i]:
                continue
            x, w, m0 = kept(logits[b, i], *asks[b])
            tokens[b, i], m1 = pick(x, w, u)
            prob[b, i] = w[list(x).index(tokens[b, i])]
            margin[b, i] = min(m0, m1)
    return tokens, prob, margin, code


def verify(target, draft, drafted, uniforms, asks, draft_asks=None):
    """target [B][K+1][V], draft [B][K][V], drafted [B][K], uniforms [B][K+1][2].
    Returns tokens [B][K+1], accept_len [B], margin [B]."""
    draft_asks = asks if draft_asks is None else draft_asks
    B, K1, V = target.shape
    K = K1 - 1
    tokens, length, margin = np.full((B, K1), -1), np.zeros(B, dtype=int), np.ones(B)
    for b in range(B):
        out = []
        for i in range(K1):
            u, v = (float(y) for y in uniforms[b, i])
            code = bad(target[b, i], asks[b])
            late = bad(draft[b, i], draft_asks[b]) if i < K else 0
            if not 0 <= v < 1 or (i < K and not 0 <= u < 1) or late == 1:
                code = 1
            if code != 1 and i < K and not 0 <= drafted[b, i] < V:
                code = 3
            code = code or late
            if code:
                out, length[b] = [], -code
                break
            x, w, m = kept(target[b, i], *asks[b])
            margin[b] = min(margin[b], m)
            q = np.zeros(V)
            q[x] = w
            p = np.zeros(V)
            if i < K:
                y, w, m = kept(draft[b, i], *draft_asks[b])
                p[y] = w
                d = int(drafted[b, i])
                if q[d] > 0 or p[d] > 0:
                    margin[b] = min(margin[b], m, abs(u * p[d] - q[d]))
                if u * p[d] < q[d]:
                    out.append(d)
                    continue
                margin[b] = min(margin[b], m)
            r = np.clip(q - p, 0, None)
            # what is left is as exact as q and p are: relative to 1, not to its sum
            r = r if r.sum() > 0 else q
            t, m = pick(np.arange(V), r, v)
            margin[b] = min(margin[b], m * r.sum())
            out.append(t)
            length[b] = i
            break
        tokens[b, :len(out)] = out
    return tokens, length, margin
