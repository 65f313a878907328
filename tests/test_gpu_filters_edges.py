"""Filtered calls where their searches change over: cuts among equal logits, near
zero, at the ends of the weights' range; calls at once.  Oracle and tolerances as in
test_gpu_filters.py."""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import speculative_decoding_verification_sampling_gb300 as sv
from test_gpu_filters import BF, DEV, _filters, _pair, _sample, _verify

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(DEV)
    sv.load()


# top-p, larger top-k, both, with min-p, at temperatures from one end to the other
ASKS = [(T, k, p, m) for T in (1e-3, 0.5, 1.0, 20.0, 1e4, 1e30) for k, p, m in
        ((0, 0.5, 0.0), (0, 0.97, 0.0), (300, 1.0, 0.0), (300, 0.7, 0.0), (1500, 0.9, 0.01))]


def _rows(kind, n, V, dtype, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    z = torch.randn((n, 1, V), generator=g, device=DEV)
    if kind == "near zero":          # bfloat16 values of many octaves, both signs
        z = z * torch.exp2(-12 * torch.rand((n, 1, V), generator=g, device=DEV)) * 0.01
    elif kind == "few values":       # hundreds to thousands of tokens at each
        z = torch.round(2 * z) / 2
    elif kind == "two values":
        z = torch.where(z > 1.0, 0.25, -0.25)
    elif kind == "signed zeros":     # half of the row at zero of either sign, beside others
        z = torch.where(z.abs() < 0.7, 0.0 * z, z)
    elif kind == "one above":        # all weight but 2^-20 in one token
        z = z * 0.1
        z[..., V // 2] = 20.0
    elif kind == "steps":            # equal weights in blocks: borders of top-p between them
        z = torch.floor(torch.arange(V, device=DEV).float() / V * 5).expand(n, 1, V).contiguous()
    elif kind == "falling":          # the last CTAs' parts hold nothing that is kept
        z = torch.linspace(12, -12, V, device=DEV).expand(n, 1, V).contiguous()
    return z.to(dtype)


@pytest.mark.parametrize("kind", ["near zero", "few values", "two values", "signed zeros", "one above", "steps",
                                  "falling"])
@pytest.mark.parametrize("dtype", [torch.float32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("V", [257, 4096, 20011])
def test_sample_changeovers(kind, dtype, V):
    _sample(_rows(kind, len(ASKS), V, dtype, V), ASKS, V, f"{kind} {V}")


@pytest.mark.parametrize("kind", ["few values", "two values", "signed zeros", "falling"])
@pytest.mark.parametrize("dtype", [torch.float32, BF], ids=["f32", "bf16"])
def test_verify_changeovers(kind, dtype):
    """The cut between equal logits, told by whichever CTA has it, reaches the rule."""
    V, K = 9001, 2
    g = torch.Generator(device=DEV).manual_seed(5)
    z = _rows(kind, len(ASKS) * 3, V, torch.float32, 7).view(len(ASKS), 3, V)
    draft = (z[:, :K] + 0.25 * (torch.rand((len(ASKS), K, V), generator=g, device=DEV) < 0.3)).to(dtype).contiguous()
    f, _ = _filters(ASKS)
    drafted, _ = sv.spec_filter_sample(draft, torch.rand((len(ASKS), K), generator=g, device=DEV), f)
    u = torch.rand((len(ASKS), K + 1, 2), generator=g, device=DEV)
    _verify(z.to(dtype), draft, drafted, u, ASKS, None, kind)


@pytest.mark.parametrize("dtype", [torch.float32, BF], ids=["f32", "bf16"])
def test_uniforms_at_the_ends(dtype):
    V = 3000
    z = _rows("few values", 6, V, dtype, 1)
    asks = [(1.0, 0, 1.0, 0.0), (1.0, 0, 0.9, 0.0), (1.0, 40, 1.0, 0.0), (1.0, 500, 0.9, 0.0), (1.0, 0, 1.0, 0.3),
            (0.0, 0, 1.0, 0.0)]
    f, exact = _filters(asks)
    from oracle import filters as oracle
    for v in (0.0, 2.0 ** -149, 1.0 - 2.0 ** -24):
        tokens, prob = sv.spec_filter_sample(z, torch.full((6, 1), v, device=DEV), f)
        for b in range(6):
            x, w, _ = oracle.kept(z[b, 0].double().cpu().numpy(), *exact[b])
            assert int(tokens[b]) == (x[0] if v < 0.5 else x[w > 0][-1]), (v, b)
            assert float(prob[b]) > 0


def test_calls_at_once_on_two_streams():
    B, K, V = 40, 3, 30011
    asks = [ASKS[i % len(ASKS)] for i in range(B)]
    f, _ = _filters(asks)
    inputs = [_pair("zipf", B, K, V, BF, s) for s in (1, 2)]
    drafted = [sv.spec_filter_sample(d, torch.rand((B, K), generator=g, device=DEV), f)[0] for _, d, _, g in inputs]
    want = [sv.spec_verify_filtered(t, d, x, u, f) for (t, d, u, _), x in zip(inputs, drafted)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(6):
        for i, s in enumerate(streams):
            (t, d, u, _), x = inputs[i], drafted[i]
            with torch.cuda.stream(s):
                got[i].append(sv.spec_verify_filtered(t, d, x, u, f))
    torch.cuda.synchronize()
    for i in range(2):
        for tokens, n in got[i]:
            assert torch.equal(tokens, want[i][0]) and torch.equal(n, want[i][1])


def test_outputs_given_and_refusals_on_the_device():
    z = torch.randn((2, 3, 500), device=DEV)
    u = torch.rand((2, 3), device=DEV)
    tokens, prob = torch.empty((2, 3), dtype=torch.int32, device=DEV), torch.empty((2, 3), device=DEV)
    a, b = sv.spec_filter_sample(z, u, out_tokens=tokens, out_prob=prob)
    assert a is tokens and b is prob and torch.equal(a, sv.spec_filter_sample(z, u)[0])
    with pytest.raises(ValueError):
        sv.spec_filter_sample(z[:, :, ::2], u)
    with pytest.raises(ValueError):
        sv.spec_filter_sample(z, u[:1])
    with pytest.raises(TypeError):
        sv.spec_filter_sample(z.half(), u)
    with pytest.raises(TypeError):
        sv.spec_filter_sample(z, u.double())
    with pytest.raises(ValueError):
        sv.spec_filter_sample(z, u, sv.Filters.fill(3, DEV))
    with pytest.raises(TypeError):
        sv.spec_filter_sample(z, u, sv.Filters(top_k=torch.ones(2, device=DEV)))
    with pytest.raises(TypeError):
        sv.spec_filter_sample(z, u, sv.Filters(top_p=torch.ones(2)))
    d = torch.zeros((2, 2), dtype=torch.int32, device=DEV)
    v = torch.rand((2, 3, 2), device=DEV)
    with pytest.raises(sv.SpecVerifyError):
        sv.spec_verify_filtered(z, z[:, :2].contiguous(), d, v, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
    with pytest.raises(ValueError):
        sv.spec_verify_filtered(z, z, d, v)
    with pytest.raises(TypeError):
        sv.spec_verify_filtered(z, z[:, :2].to(BF), d, v)


def test_window_without_a_cache():
    """A pass over nothing but its own entries, windows shorter than it."""
    from oracle.attention import window_attention
    from test_gpu_attention import _hold
    g = torch.Generator(device=DEV).manual_seed(2)
    r = lambda *s: torch.randn(s, generator=g, device=DEV).to(BF)   # noqa: E731
    q, staged = r(2, 9, 8, 64), r(2, 9, 2, 2, 64)
    cache, n = r(2, 0, 2, 2, 64), torch.zeros(2, dtype=torch.int32, device=DEV)
    for window, sinks in ((3, 0), (3, 2), (100, 0), (1, 1)):
        out, lse = sv.spec_verify_window_attention(q, cache, n, window, sinks=sinks, staged=staged)
        _hold(out, lse, window_attention(q, cache, [0, 0], window, sinks, staged), 64, f"{window} {sinks}")
    out, lse = sv.spec_verify_window_attention(q, cache, n, 3, sinks=1)
    assert not out.any() and (lse == -math.inf).all()


def test_window_refusals_on_the_device():
    q = torch.zeros((1, 2, 2, 64), dtype=BF, device=DEV)
    cache = torch.zeros((1, 4, 2, 1, 64), dtype=BF, device=DEV)
    n = torch.zeros(1, dtype=torch.int32, device=DEV)
    for bad in (dict(window=0), dict(window=4, sinks=-1), dict(window=4, cache_scale=torch.zeros((1, 4, 2, 1), dtype=torch.uint8, device=DEV)),
                dict(window=4, staged=cache)):
        with pytest.raises(ValueError):
            sv.spec_verify_window_attention(q, cache, n, **bad)
    with pytest.raises(sv.SpecVerifyError):     # a mask without entries
        sv.spec_verify_window_attention(q, cache, n, 4, mask=torch.ones((1, 2, 2), dtype=torch.uint8, device=DEV))
    with pytest.raises(TypeError):
        sv.spec_verify_window_attention(q.float(), cache, n, 4)
