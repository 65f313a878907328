"""Oracle of the verification pass's attention, float64.

TEST INFRASTRUCTURE ONLY (same rule as the rest of ``oracle/``).

One sequence and one key/value head at a time, over the concatenation of what
the pass's query tokens can see (nextadmin.net lesson "Speculative Decoding",
§ KV cache management; aiengineeringfromscratch.com Phase 10 lesson 25, § Tree
attention verification): the shared prefix, the sequence's cache entries below
its length, and the pass's own entries under the mask (causal without one).
Beside the result it returns what an error bound needs.
"""
from __future__ import annotations

import math

import torch


def attention(q, cache, seq_len, staged=None, mask=None, prefix=None, scale=None):
    """q [B][T][Hq][D], cache [B][L][2][H][D], prefix [P][2][H][D], staged
    [B][T][2][H][D] as values (any float type, any device).  Returns a dict of
    float64 tensors: out [B][T][Hq][D], lse [B][T][Hq], mass [B][T][Hq][D] (the
    weighted mean of |v|), reach [B][T][Hq] (the largest scale * sum_d |q_d k_d|
    over the visible entries), count [B][T][Hq] (visible entries)."""
    B, T, Hq, D = q.shape
    H = cache.shape[3]
    G = Hq // H
    scale = D ** -0.5 if scale is None else scale
    f = dict(dtype=torch.float64, device=q.device)
    res = {"out": torch.zeros((B, T, Hq, D), **f), "mass": torch.zeros((B, T, Hq, D), **f),
           "lse": torch.full((B, T, Hq), -math.inf, **f), "reach": torch.zeros((B, T, Hq), **f),
           "count": torch.zeros((B, T, Hq), **f)}
    for b in range(B):
        n = int(seq_len[b])
        for h in range(H):
            parts = [] if prefix is None else [prefix[:, :, h]]
            parts.append(cache[b, :n, :, h])
            if staged is not None:
                parts.append(staged[b, :, :, h])
            kv = torch.cat([p.double() for p in parts])
            seen = torch.ones((T, len(kv)), dtype=torch.bool, device=q.device)
            if staged is not None:
                seen[:, len(kv) - T:] = (mask[b] != 0 if mask is not None else
                                         torch.ones((T, T), dtype=torch.bool, device=q.device).tril())
            for t in range(T):
                k, v = kv[seen[t], 0], kv[seen[t], 1]
                if not len(k):
                    continue
                x = q[b, t, h * G:(h + 1) * G].double()
                s = scale * (x @ k.T)
                z = torch.logsumexp(s, -1)
                p = torch.exp(s - z[:, None])
                at = (b, t, slice(h * G, (h + 1) * G))
                res["out"][at] = p @ v
                res["mass"][at] = p @ v.abs()
                res["lse"][at] = z
                res["reach"][at] = scale * (x.abs() @ k.abs().T).amax(-1)
                res["count"][at] = len(k)
    return res
