"""Pins for the attention oracle: the formula written out in plain Python, and
what the sharing of a prefix and the tree mask mean."""
from __future__ import annotations

import math

import torch

from oracle.attention import attention
from oracle.tree import tree_mask


def _inputs(B, T, Hq, H, D, P, L, seed):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)   # noqa: E731
    return r(B, T, Hq, D), r(B, L, 2, H, D), r(B, T, 2, H, D), r(P, 2, H, D)


def test_formula_in_plain_python():
    q, cache, staged, prefix = _inputs(2, 3, 4, 2, 5, 2, 6, 1)
    seq_len = [4, 0]
    got = attention(q, cache, seq_len, staged, None, prefix, 0.7)
    for b in range(2):
        for t in range(3):
            for hq in range(4):
                h = hq // 2
                ent = [prefix[j, :, h] for j in range(2)] + [cache[b, j, :, h] for j in range(seq_len[b])]
                ent += [staged[b, j, :, h] for j in range(t + 1)]
                w = [math.exp(0.7 * sum(float(a) * float(c) for a, c in zip(q[b, t, hq], e[0]))) for e in ent]
                for d in range(5):
                    want = sum(x * float(e[1, d]) for x, e in zip(w, ent)) / sum(w)
                    assert abs(float(got["out"][b, t, hq, d]) - want) < 1e-12
                assert abs(float(got["lse"][b, t, hq]) - math.log(sum(w))) < 1e-12
                assert int(got["count"][b, t, hq]) == len(ent)


def test_a_shared_prefix_is_each_sequences_own():
    q, cache, staged, prefix = _inputs(3, 2, 2, 1, 4, 5, 4, 2)
    n = torch.tensor([4, 0, 1])
    got = attention(q, cache, n, staged, None, prefix)
    own = torch.cat([prefix[None].expand(3, -1, -1, -1, -1), cache], 1)
    want = attention(q, own, n + 5, staged)
    for k in ("out", "lse", "mass"):
        assert torch.allclose(got[k], want[k], atol=1e-13)


def test_tree_mask_is_attention_along_each_path():
    par = [-1, 0, 0, 1, 1, 3]
    q, cache, staged, _ = _inputs(1, 6, 2, 2, 4, 1, 3, 3)
    mask = torch.as_tensor(tree_mask(par))[None]
    got = attention(q, cache, [3], staged, mask)
    for n in range(6):
        path = [n]
        while par[path[0]] >= 0:
            path.insert(0, par[path[0]])
        want = attention(q[:, path], cache, [3], staged[:, path])
        assert torch.allclose(got["out"][0, n], want["out"][0, -1], atol=1e-13)


def test_rows_that_see_nothing():
    q, cache, staged, _ = _inputs(1, 2, 1, 1, 4, 1, 3, 4)
    mask = torch.tensor([[[0, 0], [0, 1]]], dtype=torch.uint8)
    got = attention(q, cache, [0], staged, mask)
    assert not got["out"][0, 0].any() and float(got["lse"][0, 0, 0]) == -math.inf
    assert torch.equal(got["out"][0, 1, 0], staged[0, 1, 1, 0])
