"""Draws at the borders between the parts of a row: those that the CTAs of a
cluster, and their warps, take.  Oracle and tolerances as in test_gpu_filters.py.
Outputs are filled ahead with what no call returns."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import speculative_decoding_verification_sampling_gb300 as sv
from oracle import filters as oracle
from test_gpu_filters import BF, DEV, NEAR, _filters

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(DEV)
    sv.load()


def _row(V, parts, dtype=BF):
    """[V] with parts = (value, first, end) in turn, the rest far below."""
    z = torch.full((V,), -10000.0, device=DEV)
    for x, first, end in parts:
        z[first:end] = x
    return z.to(dtype)


def _draw(z, ask, uniforms, what):
    """One row [V] drawn from with every uniform, as many sequences of one call."""
    n = len(uniforms)
    f, exact = _filters([ask] * n)
    u = torch.tensor(uniforms, dtype=torch.float32, device=DEV)[:, None]
    tokens = torch.full((n, 1), -7, dtype=torch.int32, device=DEV)
    prob = torch.full((n, 1), -7.0, device=DEV)
    sv.spec_filter_sample(z.expand(n, 1, -1).contiguous(), u, f, out_tokens=tokens, out_prob=prob)
    tokens, prob = tokens[:, 0].cpu().numpy(), prob[:, 0].double().cpu().numpy()
    assert (tokens != -7).all() and (prob != -7).all(), f"{what}: no token for {u[:, 0].cpu().numpy()[tokens == -7]}"
    x, w, m0 = oracle.kept(z.double().cpu().numpy(), *exact[0])
    at = {int(t): float(p) for t, p in zip(x, w)}
    for i, v in enumerate(u[:, 0].double().tolist()):
        t, m = oracle.pick(x, w, v)
        if min(m, m0) < NEAR:
            continue
        assert tokens[i] == t, f"{what}: {tokens[i]} not {t} at {v!r}"
        assert abs(prob[i] - at[t]) <= 1.01 * (2.0 ** -24 + 2.0 ** -30) * at[t] + 2.0 ** -43, what


def _borders(z, ask, steps=2):
    """Uniforms (multiples of 2^-24) at and next to the running sum of what is kept ahead of every 256th token:
    whatever the size of the cluster, a CTA's or a warp's part begins at one of them (32 vectors of 16 bytes)."""
    x, w, _ = oracle.kept(z.double().cpu().numpy(), *_filters([ask])[1][0])
    c = np.concatenate([[0.0], np.cumsum(w)])
    ends = c[np.searchsorted(x, np.arange(0, len(z) + 256, 256))]
    ends = np.unique(np.floor(ends * 2.0 ** 24).astype(np.int64))
    u = np.unique(np.clip(np.concatenate([ends + k for k in range(-steps, steps + 1)]), 0, 2 ** 24 - 1))
    return (u * 2.0 ** -24).tolist()


STEPS = [(6.5, 0, 2048), (12.0, 2048, 2049), (3.5, 4096, 8192)]
LOW = [(-2.0, 0, 2048), (2.9951334e-06, 2048, 2049), (-5.0, 4096, 8192)]   # the largest logit near 0


@pytest.mark.parametrize("parts,T,u", [(STEPS, 0.563560605, 0.105760962), (LOW, 1.0, 0.907368362)], ids=["steps", "low"])
def test_between_the_warps_and_their_cta(parts, T, u):
    """Sums of the warps' parts in floats fell short of their CTA's here, and the uniform between the two."""
    z = _row(16384, parts)
    for n in (1, 3, 40, 700):
        _draw(z, (T, 0, 0.999, 0.0), [u] * n, f"{n} rows")


@pytest.mark.parametrize("kind", ["steps", "low", "zipf", "values", "ties"])
@pytest.mark.parametrize("ask", [(1.0, 0, 0.999, 0.0), (0.7, 0, 0.9, 0.0), (0.9, 3000, 1.0, 0.0), (1.1, 5000, 0.97, 0.001)])
def test_borders_between_parts(kind, ask):
    V = 16384
    g = torch.Generator(device=DEV).manual_seed(3)
    if kind in ("steps", "low"):
        z = _row(V, STEPS if kind == "steps" else LOW)
    elif kind == "zipf":
        z = (12 - 1.5 * torch.log(torch.rand(V, generator=g, device=DEV) * V + 1)).to(BF)
    elif kind == "values":
        z = (torch.round(4 * torch.randn(V, generator=g, device=DEV)) / 8).to(BF)
    else:
        z = torch.full((V,), -3.25, device=DEV).to(BF)
    uniforms = _borders(z, ask)
    _draw(z, ask, uniforms, f"{kind} {ask}")
    for i in range(0, len(uniforms), 7):      # alone: larger clusters
        _draw(z, ask, uniforms[i:i + 1], f"{kind} {ask} alone")


@pytest.mark.parametrize("dtype", [torch.float32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("ask", [(1.0, 0, 1.0, 0.0), (1.0, 0, 0.98, 0.0), (0.5, 700, 1.0, 0.0), (2.0, 700, 0.9, 0.0)])
@pytest.mark.parametrize("V", [2000, 9000])
def test_largest_logit_near_zero(V, ask, dtype):
    """A logit far from 0 less one near 0 needs more bits than a float has: weights keep their 2^-31 all the same.
    Uniforms next to the borders of the largest logit's token, which holds about half of the weight."""
    g = torch.Generator().manual_seed(V)
    B = 300
    z = torch.full((B, 1, V), -10000.0, dtype=torch.float64)
    for b in range(B):
        m = (1.0 if b % 3 else -1.0) * 2.0 ** (-23 + 8 * float(torch.rand((), generator=g)))
        x = -ask[0] * (5.0 + 2.0 * float(torch.rand((), generator=g)))
        z[b, 0, :V // 2] = x
        z[b, 0, V // 4] = m
    z = z.to(dtype)
    u = torch.empty((B, 1))
    f, exact = _filters([ask] * B)
    for b in range(B):
        x, w, _ = oracle.kept(z[b, 0].double().numpy(), *exact[b])
        c = np.concatenate([[0.0], np.cumsum(w)])
        at = int(np.searchsorted(x, V // 4)) + b % 2
        u[b, 0] = min(np.floor(c[at] * 2.0 ** 24) + b // 2 % 2, 2.0 ** 24 - 1) * 2.0 ** -24
    tokens, prob = sv.spec_filter_sample(z.to(DEV), u.to(DEV), f)
    t, p, margin, _ = oracle.sample(z.double().numpy(), u.double().numpy(), exact)
    bad = (tokens.cpu().numpy() != t) & (margin >= NEAR)
    assert (margin >= NEAR).mean() > 0.5
    assert not bad.any(), f"{bad.sum()} of {B}: {tokens.cpu().numpy()[bad][:4]} not {t[bad][:4]}"


def test_parts_of_most_tokens():
    """Rows cut into parts of up to 65536 tokens whose weights' low halves are nearly all ones: sums of them in 32
    bits.  Nearly all tokens are equal and near 0, so their values are not counted; rows begin anywhere in a vector."""
    B, V = 80, 524283
    x = float(torch.tensor(2.0 ** -20).to(BF))
    for T in np.linspace(0.5, 1.0, 4000, dtype=np.float32):
        e = (x - 1.0) / float(T) / np.log(2.0)
        y = np.exp2(e - np.rint(64 * e) / 64) * 2.0 ** 29     # a weight, as its bin has it
        if y % 65536 > 65400 and y % 65536 < 65500:
            break
    else:
        raise AssertionError("no temperature")
    z = torch.full((B, 1, V), x, device=DEV).to(BF)
    z[:, 0, V // 3] = 1.0
    u = torch.full((B, 1), 0.625, device=DEV)
    f, exact = _filters([(float(T), 0, 0.7, 0.0)] * B)
    tokens, prob = sv.spec_filter_sample(z, u, f)
    t, p, margin, _ = oracle.sample(z[:1].double().cpu().numpy(), u[:1].double().cpu().numpy(), exact[:1])
    assert margin[0, 0] >= NEAR
    assert (tokens == int(t[0, 0])).all(), f"{sorted(set(tokens[:, 0].tolist()))} not {t[0, 0]}"
    assert ((prob.double() - p[0, 0]).abs() <= 1.01 * (2.0 ** -24 + 2.0 ** -30) * p[0, 0] + 2.0 ** -43).all()




@pytest.mark.parametrize("dtype,sizes", [(BF, (2100, 4200, 9000, 20000, 40000)), (torch.float32, (1100, 2100, 4300, 9000, 20000))],
                         ids=["bf16", "f32"])
def test_first_exchange_of_short_rows(dtype, sizes):
    """Clusters of 2 to 16 CTAs with little to read ahead of their first exchange, many of them in a row."""
    g = torch.Generator(device=DEV).manual_seed(1)
    for V in sizes:
        for B in (1, 7):
            z = torch.randn((B, 1, V), generator=g, device=DEV).to(dtype)
            z[:, 0, V - 1] = 30.0                     # in the last CTA that has tokens
            f, _ = _filters([(1.0, 0, 1.0, 0.0), (0.0, 0, 1.0, 0.0), (1.0, 9, 1.0, 0.0)][:B] * 3 if B > 1 else [(1.0, 9, 0.9, 0.0)])
            f = sv.Filters(*[getattr(f, n)[:B].clone() for n in sv.Filters.__slots__])
            u = torch.full((B, 1), 0.5, device=DEV)
            out = [torch.full((B, 1), -7, dtype=torch.int32, device=DEV) for _ in range(200)]
            for tokens in out:
                sv.spec_filter_sample(z, u, f, out_tokens=tokens)
            assert all((tokens == V - 1).all() for tokens in out), f"{V} {B}"


def test_a_workspace_with_gaps_is_refused():
    """Its elements do not tell how much memory there is: one repeated element has that of one."""
    B, K, V = 2, 2, 500
    target, draft = torch.randn((B, K + 1, V), device=DEV), torch.randn((B, K, V), device=DEV)
    d, u = torch.zeros((B, K), dtype=torch.int32, device=DEV), torch.rand((B, K + 1, 2), device=DEV)
    n = sv.spec_filter_workspace_bytes(B, K, V)
    with pytest.raises(ValueError):
        sv.spec_verify_filtered(target, draft, d, u, workspace=torch.empty(2 * n, dtype=torch.uint8, device=DEV)[::2])
    q = torch.zeros((1, 2, 2, 64), dtype=BF, device=DEV)
    cache, length = torch.zeros((1, 4, 2, 1, 64), dtype=BF, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
    n = sv.spec_attention_workspace_bytes(1, 2, 2, 1, 64, 0, 4)
    with pytest.raises(ValueError):
        sv.spec_verify_window_attention(q, cache, length, 4, workspace=torch.empty(2 * n, dtype=torch.uint8, device=DEV)[::2])


@pytest.mark.parametrize("ask", [(1.0, 0, 1.0, 0.0), (1.0, 0, 0.97, 0.0), (0.8, 30000, 1.0, 0.0)])
@pytest.mark.parametrize("dtype", [torch.float32, BF], ids=["f32", "bf16"])
def test_equal_logits_alone_and_among_others(dtype, ask):
    """Sums of many equal weights, where roundings would add up: the same probabilities, to the last bit, whatever the
    size of the cluster, and right to half a step of float32."""
    B, V = 96, 100003
    g = torch.Generator(device=DEV).manual_seed(7)
    z = (-4.0 * torch.rand((B, 1, 1), generator=g, device=DEV) - 1.0).expand(B, 1, V).contiguous()
    z[:, 0, V // 2] = 2.0
    z[:, 0, V // 3:V // 3 + 5000] += 0.5
    z = z.to(dtype)
    u = torch.rand((B, 1), generator=g, device=DEV)
    f, exact = _filters([ask] * B)
    one, _ = _filters([ask])
    tokens, prob = sv.spec_filter_sample(z, u, f)
    alone = [sv.spec_filter_sample(z[b:b + 1], u[b:b + 1], one) for b in range(B)]
    assert torch.equal(torch.cat([t for t, _ in alone]), tokens)
    assert torch.equal(torch.cat([p for _, p in alone]), prob)
    t, p, margin, _ = oracle.sample(z[:24].double().cpu().numpy(), u[:24].double().cpu().numpy(), exact[:24])
    near = margin < NEAR
    assert near.sum() <= 2
    assert ((tokens[:24].cpu().numpy() == t) | near).all()
    off = np.abs(prob[:24].double().cpu().numpy() - p)[~near]
    assert (off <= (1.01 * (2.0 ** -24 + 2.0 ** -30) * p + 2.0 ** -43)[~near]).all()
