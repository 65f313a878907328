"""Refusals of the windowed attention, and pins of its oracle (no GPU needed)."""
from __future__ import annotations

import ctypes

import pytest
import torch

import speculative_decoding_verification_sampling_gb300 as sv
from oracle.attention import attention, window_attention

P = ctypes.c_void_p(256)


def test_window_attention_rejects_bad_arguments():
    f = sv.load().spec_verify_window_attention
    ok = dict(q=P, cache=P, cs=None, quant=0, len=P, staged=P, mask=None, window=4, sinks=1, B=2, T=3, Hq=4, H=2, D=64,
              L=8, scale=0.1, out=P, lse=None, ws=P, wsb=1 << 40, st=None, stream=None)
    n0 = sv.spec_launch_count()
    odd = ctypes.c_void_p(264)
    for bad in (dict(q=None), dict(cache=None), dict(len=None), dict(out=None), dict(ws=None), dict(wsb=0),
                dict(quant=1), dict(staged=None, mask=P), dict(window=0), dict(window=-1), dict(sinks=-1), dict(B=0),
                dict(T=0), dict(T=2049), dict(Hq=0), dict(H=0), dict(Hq=5), dict(D=96), dict(Hq=129, H=1), dict(L=-1),
                dict(scale=0.0), dict(scale=float("nan")), dict(q=odd), dict(cache=odd), dict(staged=odd),
                dict(out=odd), dict(ws=odd), dict(B=300, Hq=1, H=1, L=2 ** 31 - 1)):
        assert f(*{**ok, **bad}.values()) == 1, bad
    assert sv.spec_launch_count() == n0


def test_binding_rejects_what_is_not_a_cuda_tensor_of_the_right_kind():
    q = torch.zeros((1, 1, 1, 64), dtype=torch.bfloat16)
    cache = torch.zeros((1, 4, 2, 1, 64), dtype=torch.bfloat16)
    n = torch.zeros(1, dtype=torch.int32)
    for bad in ((q, cache, n), (q[0], cache, n), (q, cache[0], n)):
        with pytest.raises(TypeError):
            sv.spec_verify_window_attention(*bad, 4)


def test_oracle_sees_the_first_and_the_last():
    g = torch.Generator().manual_seed(1)
    r = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)   # noqa: E731
    q, cache, staged = r(2, 3, 4, 8), r(2, 9, 2, 2, 8), r(2, 3, 2, 2, 8)
    far = window_attention(q, cache, [9, 4], 100, 0, staged)
    ref = attention(q, cache, [9, 4], staged)
    for k in ref:
        torch.testing.assert_close(far[k], ref[k])
    # by hand: token 1 of sequence 0 has eleven entries; it sees 0, 1 and the last three
    got = window_attention(q, cache, [9, 4], 3, 2, staged)
    kv = torch.cat([cache[0], staged[0, :2]])[[0, 1, 8, 9, 10]]
    p = torch.softmax(8 ** -0.5 * q[0, 1, 3] @ kv[:, 0, 1].T, -1)
    torch.testing.assert_close(got["out"][0, 1, 3], p @ kv[:, 1, 1])
    assert got["count"][0, 1, 3] == 5
    assert (window_attention(q, cache, [0, 0], 3, 2)["lse"] == -torch.inf).all()
