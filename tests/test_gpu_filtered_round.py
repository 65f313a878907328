"""Decoding rounds with the filtered calls and the windowed attention together, as
the example runs them: every call of the first and the last round against its
oracle, on what the calls before it have left.  Tolerances are those of
test_gpu_filters.py and test_gpu_attention.py."""
from __future__ import annotations

import os
import sys

import numpy as np
import pytest
import torch

from oracle import filters as oracle
from oracle.attention import window_attention
from test_gpu_attention import _hold, _values

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu
NEAR = 2.0 ** -28


def test_rounds():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import filtered_round
    rounds, K = 5, 3
    calls = dict(sample=0, window=0, verify=0)
    # as the device has them
    exact = lambda asks: [(float(np.float32(a)), k, float(np.float32(c)), float(np.float32(e))) for a, k, c, e in asks]   # noqa: E731
    cpu = lambda *x: [y.double().cpu().numpy() for y in x]   # noqa: E731

    def watch(what, inputs, outputs):
        n = calls[what]
        calls[what] += 1
        per = {"sample": K, "window": K + 1, "verify": 1}[what]
        if per <= n < per * (rounds - 1):
            return
        torch.cuda.synchronize()
        if what == "sample":
            z, u, asks = inputs
            t, p, margin, code = oracle.sample(*cpu(z, u), exact(asks))
            assert not code.any()
            assert ((outputs[0].cpu().numpy() == t) | (margin < NEAR)).all()
        elif what == "window":
            q, cache, scale, length, new, window, sinks = inputs
            ref = window_attention(q, _values(cache, scale), length.tolist(), window, sinks, new)
            _hold(outputs[0], outputs[1], ref, q.shape[-1], f"pass {n}")
        else:
            z, draft, d, u, asks = inputs
            t, length, margin = oracle.verify(*cpu(z, draft), d.cpu().numpy(), *cpu(u), exact(asks))
            same = (outputs[1].cpu().numpy() == length) & (outputs[0].cpu().numpy() == t).all(-1)
            assert (same | (margin < NEAR)).all()
    per_round = filtered_round.main(B=12, K=K, rounds=rounds, V=1500, window=7, sinks=2, watch=watch)
    assert 1 <= per_round <= K + 1
    assert calls == dict(sample=rounds * K, window=rounds * (K + 1), verify=rounds)
