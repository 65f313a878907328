"""How the verification attention is called (CUDA): from threads, on streams that
are not current, under capture, with waits that run out."""
from __future__ import annotations

import threading

import pytest
import torch

import speculative_decoding_verification_sampling_gb300 as sv
from test_gpu_attention import DEV, _case, _device   # noqa: F401

pytestmark = pytest.mark.gpu


def _call(a, **kw):
    keys = ("q", "cache", "seq_len")
    return sv.spec_verify_attention(*(a[k] for k in keys), **{k: v for k, v in a.items() if k not in keys}, **kw)


def test_two_threads_on_one_stream():
    """Each thread's results are those of the same calls alone, bit for bit."""
    shapes = [(3, 5, 8, 2, 128, 300, 400, [400, 31, 260], False, "causal"),
              (2, 9, 16, 4, 64, 0, 3000, [3000, 1999], True, "tree"),
              (64, 8, 4, 1, 64, 515, 20, [(3 * i) % 21 for i in range(64)], True, "causal")]
    cases = [[_case(*s, seed=50 + i + 10 * k) for i, s in enumerate(shapes)] for k in range(2)]
    want = [[tuple(x.clone() for x in _call(a)) for a in mine] for mine in cases]
    torch.cuda.synchronize()
    bad, both = [], threading.Barrier(2)

    def work(k):
        torch.cuda.set_device(DEV)
        both.wait()
        for r in range(200):
            i = (r + k) % 3
            out, lse = _call(cases[k][i])
            if not (torch.equal(out, want[k][i][0]) and torch.equal(lse, want[k][i][1])):
                bad.append((k, r, i))
    threads = [threading.Thread(target=work, args=(k,)) for k in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad, bad[:10]
