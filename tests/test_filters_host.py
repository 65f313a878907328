"""Refusals of the filtered calls, and pins of their oracle (no GPU needed)."""
from __future__ import annotations

import ctypes

import numpy as np
import pytest
import torch

import speculative_decoding_verification_sampling_gb300 as sv
from oracle import filters as oracle

P = ctypes.c_void_p(256)


def test_filter_sample_rejects_bad_arguments():
    f = sv.load().spec_filter_sample
    ok = dict(z=P, dt=1, u=P, B=1, K=1, V=8, f=None, out=P, prob=None, st=None, stream=None)
    n0 = sv.spec_launch_count()
    for bad in (dict(z=None), dict(dt=2), dict(u=None), dict(B=0), dict(K=0), dict(V=0), dict(out=None),
                dict(B=1 << 20, K=1 << 10)):
        assert f(*{**ok, **bad}.values()) == 1, bad
    assert f(*{**ok, "V": 524289}.values()) == 5
    assert sv.spec_launch_count() == n0


def test_verify_filtered_rejects_bad_arguments():
    f = sv.load().spec_verify_filtered
    ok = dict(t=P, dt=1, d=P, tok=P, u=P, B=2, K=3, V=8, f=None, df=None, out=P, n=P, ws=P, wsb=1 << 40, st=None,
              stream=None)
    n0 = sv.spec_launch_count()
    for bad in (dict(t=None), dict(dt=2), dict(d=None), dict(tok=None), dict(u=None), dict(B=0), dict(K=0),
                dict(K=32), dict(V=0), dict(out=None), dict(n=None), dict(ws=None), dict(wsb=16),
                dict(ws=ctypes.c_void_p(264)), dict(B=1 << 26)):
        assert f(*{**ok, **bad}.values()) == 1, bad
    assert f(*{**ok, "V": 524289}.values()) == 5
    assert sv.spec_launch_count() == n0
    w = sv.spec_filter_workspace_bytes
    assert 0 < w(1, 1, 1) < w(256, 4, 128256) < 1 << 28
    assert not any((w(0, 1, 1), w(1, 0, 1), w(1, 32, 1), w(1, 1, 0), w(1, 1, 524289), w(1 << 26, 4, 8)))


def test_binding_rejects_what_is_not_a_cuda_tensor_of_the_right_kind():
    z, u = torch.zeros(2, 1, 8), torch.zeros(2, 1)
    for bad in ((z, u), (z[0], u)):
        with pytest.raises(TypeError):
            sv.spec_filter_sample(*bad)
    with pytest.raises(TypeError):
        sv.spec_verify_filtered(z, z, torch.zeros(2, 0, dtype=torch.int32), u)
    with pytest.raises(TypeError):
        sv.Filters(temperature=torch.ones(2))._struct(2, 0, "filters")


def test_oracle_keeps_by_the_definition():
    z = np.log([0.4, 0.05, 0.3, 0.2, 0.05])
    assert oracle.kept(z)[0].tolist() == [0, 1, 2, 3, 4]
    assert oracle.kept(z, k=2)[0].tolist() == [0, 2]
    assert oracle.kept(z, k=4)[0].tolist() == [0, 1, 2, 3]             # the lower index of two equals
    assert oracle.kept(z, p=0.4)[0].tolist() == [0]                    # 0.4 reaches 0.4
    assert oracle.kept(z, p=0.41)[0].tolist() == [0, 2]
    assert oracle.kept(z, p=0.0)[0].tolist() == [0]
    assert oracle.kept(z, k=2, p=0.6)[0].tolist() == [0, 2]            # 4/7 < 0.6 of what top-k left
    assert oracle.kept(z, k=2, p=0.55)[0].tolist() == [0]
    assert oracle.kept(z, least=0.5 - 1e-9)[0].tolist() == [0, 2, 3]
    assert oracle.kept(z, T=0.5, least=0.3)[0].tolist() == [0, 2]      # (3/4)^2 = 0.56, (1/2)^2 = 0.25
    assert oracle.kept(z, T=0)[0].tolist() == [0]
    np.testing.assert_allclose(oracle.kept(z, k=2)[1], [4 / 7, 3 / 7])
    assert [oracle.pick(*oracle.kept(z, k=2)[:2], v)[0] for v in (0.0, 0.57, 0.58, 0.999)] == [0, 0, 2, 2]


def test_oracle_verification_gives_the_target():
    """Drafts from p', verified: the first emitted token follows q' (exactly, over a grid of uniforms)."""
    rng = np.random.default_rng(1)
    zq, zp = rng.normal(size=6), rng.normal(size=6)
    ask, dask = (0.8, 4, 0.9, 0.0), (1.2, 5, 1.0, 0.1)
    x, w, _ = oracle.kept(zq, *ask)
    q = np.zeros(6)
    q[x] = w
    y, w, _ = oracle.kept(zp, *dask)
    p = np.zeros(6)
    p[y] = w
    got, n = np.zeros(6), 400
    for d in y:
        for u in (np.arange(n) + 0.5) / n:
            t, a, _ = oracle.verify(np.stack([zq, zq])[None], zp[None, None], np.array([[d]]),
                                    np.array([[[u, 0.5], [0.5, 0.5]]]), [ask], [dask])
            if a[0] == 1:
                got[d] += p[d] / n
            else:       # integrate the draw: all of (q - p)+
                r = np.clip(q - p, 0, None)
                got += p[d] / n * r / r.sum()
    np.testing.assert_allclose(got, q, atol=2.0 / n)
