"""Refusals of the 8-bit cache calls and the verification attention: argument
errors come back before anything is launched (no GPU needed)."""
from __future__ import annotations

import ctypes

import pytest
import torch

import speculative_decoding_verification_sampling_gb300 as sv

P = ctypes.c_void_p(256)


def test_kv_commit_quant_rejects_bad_arguments():
    f = sv.load().spec_kv_commit_quant
    ok = dict(cache=P, scale=P, staged=P, sdt=1, nodes=None, lead=0, NL=1, B=1, K=4, L=8, H=1, D=64, acc=P, len=P,
              st=None, stream=None)
    n0 = sv.spec_launch_count()
    for bad in (dict(cache=None), dict(scale=None), dict(staged=None), dict(sdt=2), dict(lead=-1), dict(lead=2),
                dict(NL=0), dict(B=0), dict(K=0), dict(L=0), dict(H=0), dict(D=0), dict(D=96), dict(acc=None),
                dict(len=None), dict(cache=ctypes.c_void_p(264)), dict(staged=ctypes.c_void_p(264)),
                dict(NL=1 << 20, B=1 << 20, L=1 << 20)):
        assert f(*{**ok, **bad}.values()) == 1, bad
    assert f(*{**ok, "NL": 1 << 16, "B": 1 << 16}.values()) == 5       # the grid
    assert sv.spec_launch_count() == n0


def test_kv_read_quant_rejects_bad_arguments():
    f = sv.load().spec_kv_read_quant
    ok = dict(cache=P, scale=P, start=None, len=P, NL=1, B=1, L=8, count=4, H=1, D=64, out=P, odt=1, st=None,
              stream=None)
    n0 = sv.spec_launch_count()
    for bad in (dict(cache=None), dict(scale=None), dict(len=None), dict(out=None), dict(odt=3), dict(NL=0),
                dict(B=-1), dict(L=0), dict(count=0), dict(H=0), dict(D=32), dict(cache=ctypes.c_void_p(260)),
                dict(out=ctypes.c_void_p(264)), dict(NL=1 << 20, B=1 << 20, L=1 << 20)):
        assert f(*{**ok, **bad}.values()) == 1, bad
    assert sv.spec_launch_count() == n0


def test_verify_attention_rejects_bad_arguments():
    f = sv.load().spec_verify_attention
    ok = dict(q=P, prefix=P, ps=None, cache=P, cs=None, quant=0, len=P, staged=P, mask=None, B=2, T=3, Hq=4, H=2, D=64,
              P=5, L=8, scale=0.1, out=P, lse=None, ws=P, wsb=1 << 40, st=None, stream=None)
    n0 = sv.spec_launch_count()
    odd = ctypes.c_void_p(264)
    for bad in (dict(q=None), dict(prefix=None), dict(cache=None), dict(len=None), dict(out=None), dict(ws=None),
                dict(wsb=0), dict(quant=1), dict(quant=1, ps=P), dict(quant=1, cs=P), dict(staged=None, mask=P),
                dict(B=0), dict(T=0), dict(T=2049), dict(Hq=0), dict(H=0), dict(Hq=5), dict(D=128 + 64), dict(D=0),
                dict(Hq=129, H=1), dict(P=-1), dict(L=-1), dict(B=1 << 20, T=2048), dict(scale=0.0),
                dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(q=odd), dict(prefix=odd),
                dict(cache=odd), dict(staged=odd), dict(out=odd), dict(ws=odd)):
        assert f(*{**ok, **bad}.values()) == 1, bad
    assert sv.spec_launch_count() == n0


def test_attention_workspace_bytes():
    w = sv.spec_attention_workspace_bytes
    assert 0 < w(1, 1, 1, 1, 64, 0, 0) <= w(64, 5, 32, 8, 128, 8192, 512) < 4 << 30
    for bad in ((0, 1, 1, 1, 64, 0, 0), (1, 0, 1, 1, 64, 0, 0), (1, 1, 3, 2, 64, 0, 0), (1, 1, 1, 1, 65, 0, 0),
                (1, 1, 1, 1, 64, -1, 0), (1, 1, 1, 1, 64, 0, -1), (1, 2049, 1, 1, 64, 0, 0)):
        assert w(*bad) == 0, bad


def test_binding_rejects_what_is_not_a_cuda_tensor_of_the_right_kind():
    q = torch.zeros((1, 1, 1, 64), dtype=torch.bfloat16)
    cache = torch.zeros((1, 4, 2, 1, 64), dtype=torch.bfloat16)
    n = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(TypeError):
        sv.spec_verify_attention(q, cache, n)
    with pytest.raises(TypeError):
        sv.spec_verify_attention(q[0], cache, n)
    with pytest.raises(TypeError):
        sv.spec_verify_attention(q, cache[0], n)
    c8 = torch.zeros((1, 1, 4, 2, 1, 64), dtype=torch.float8_e4m3fn)
    s8 = torch.zeros((1, 1, 4, 2, 1), dtype=torch.uint8)
    with pytest.raises(TypeError):
        sv.spec_kv_commit_quant(c8, s8, cache[None], n, n)
    with pytest.raises(TypeError):
        sv.spec_kv_read_quant(c8, s8, None, n, 4)
    with pytest.raises(TypeError):
        sv.spec_kv_read_quant(c8[0], s8, None, n, 4)
