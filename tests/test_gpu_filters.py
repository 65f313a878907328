"""Filtered sampling and filtered verification (CUDA, through the C ABI) against
the float64 oracle.

What may differ: a weight is right to 2^-31.4 of itself (its exponential's last
factor is float32, 2^-24 relative of at most 0.0055, rounded a few times; the
exponent's rest adds less) and to 2^-44 of the largest, so a sum of them, and a
share of one sum in another, is right to 2^-30.  With V <= 2^18 weights below
half a unit of 2^-43 the total may miss another 2^-26 of the largest in a row
whose whole rest lies there; the rows here do not.  A decision whose distance
from its border (the oracle's margin) is below 2^-28 is left out, and few may be.
A probability is rounded to float32 once more, half a step (2^-24).
"""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import speculative_decoding_verification_sampling_gb300 as sv
from oracle import filters as oracle

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF = torch.bfloat16
NEAR = 2.0 ** -28
ASKS = [(1.0, 0, 1.0, 0.0), (0.0, 0, 1.0, 0.0), (0.7, 20, 0.8, 0.0), (1.0, 0, 0.9, 0.0), (1.0, 0, 1.0, 0.05),
        (0.8, 1, 1.0, 0.0), (1.3, 100, 0.95, 0.02), (0.9, 3000, 1.0, 0.0), (0.6, 700, 0.999, 0.0), (1.0, 0, 0.5, 0.01),
        (1.0, 0, 0.0, 0.0), (50.0, 7, 1.0, 0.0), (0.01, 0, 0.99, 0.0), (1.0, 2 ** 30, 2.0, -1.0), (1.0, 0, 1.0, 1.0),
        (1e30, 50, 0.3, 0.0), (1e-30, 50, 0.3, 0.0), (200.0, 0, 0.7, 0.5), (1.0, -3, -0.5, 0.3), (2.0, 256, 0.9999999, 0.0)]


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(DEV)
    sv.load()


def _filters(asks):
    kinds = (torch.float32, torch.int32, torch.float32, torch.float32)
    cols = [torch.tensor([a[i] for a in asks], dtype=kinds[i], device=DEV) for i in range(4)]
    exact = [tuple(float(c[b]) for c in cols) for b in range(len(asks))]     # as the device has them
    return sv.Filters(*cols), [(t, int(a[1]), p, m) for (t, _, p, m), a in zip(exact, asks)]


def _logits(kind, shape, dtype, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    V = shape[-1]
    z = 2.5 * torch.randn(shape, generator=g, device=DEV)
    if kind == "zipf":
        z = 12 - 1.5 * torch.log(torch.rand(shape, generator=g, device=DEV) * V + 1)
    elif kind == "ties":
        z = torch.round(z)
    elif kind == "equal":
        z = torch.full(shape, -3.25, device=DEV)
    elif kind == "peak":
        z = z.clamp(max=3)
        z[..., V // 3] = 40.0
    elif kind == "masked":
        z[torch.rand(shape, generator=g, device=DEV) < 0.97] = -math.inf
        z[..., V // 2] = 1.5
    elif kind == "lowest":
        z[torch.rand(shape, generator=g, device=DEV) < 0.97] = torch.finfo(dtype).min
        z[..., V - 1] = 0.5
    elif kind == "zeros":
        z = torch.where(torch.rand(shape, generator=g, device=DEV) < 0.5, 0.0, -0.0)
    elif kind == "far":
        z = 300.0 * z
    return z.to(dtype)


def _sample(logits, asks, seed, what, **kw):
    B, K, V = logits.shape
    g = torch.Generator(device=DEV).manual_seed(seed + 1)
    u = torch.rand((B, K), generator=g, device=DEV)
    f, exact = _filters(asks)
    st = torch.full((1,), -5, dtype=torch.int32, device=DEV)
    tokens, prob = sv.spec_filter_sample(logits, u, f, device_status=st, **kw)
    torch.cuda.synchronize()
    assert int(st) == 0, what
    t, p, margin, _ = oracle.sample(logits.double().cpu().numpy(), u.double().cpu().numpy(), exact)
    near = margin < NEAR
    assert near.sum() <= 2 + 0.02 * near.size, what
    tokens, prob = tokens.cpu().numpy(), prob.double().cpu().numpy()
    bad = (tokens != t) & ~near
    assert not bad.any(), f"{what}: {tokens[bad][:4]} not {t[bad][:4]}, asked {[exact[b] for b in np.nonzero(bad)[0][:4]]}"
    off = np.abs(prob - p)[~near & (tokens == t)]
    tol = 1.01 * (2.0 ** -24 + 2.0 ** -30) * p[~near & (tokens == t)] + 2.0 ** -43
    assert (off <= tol).all(), f"{what}: probability"


@pytest.mark.parametrize("kind", ["normal", "zipf", "ties", "equal", "peak", "masked", "lowest", "zeros", "far"])
@pytest.mark.parametrize("dtype", [torch.float32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("V", [1, 2, 7, 31, 1000, 1025, 5003, 32003])
def test_sample(kind, dtype, V):
    z = _logits(kind, (len(ASKS), 2, V), dtype, V)
    _sample(z, ASKS, V, f"{kind} {V}")


@pytest.mark.parametrize("kind", ["normal", "zipf", "ties", "equal"])
@pytest.mark.parametrize("dtype,V", [(torch.float32, 152064), (BF, 128256), (BF, 262147), (torch.float32, 524288)])
def test_sample_large(kind, dtype, V):
    _sample(_logits(kind, (6, 1, V), dtype, V), [ASKS[i] for i in (2, 3, 4, 0, 7, 8)], V, f"{kind} {V}")


def test_sample_many_rows():
    """More rows than CTAs fit at once."""
    asks = [ASKS[i % len(ASKS)] for i in range(700)]
    _sample(_logits("zipf", (700, 2, 3001), BF, 5), asks, 5, "700 x 2 rows")


@pytest.mark.parametrize("dtype", [torch.float32, BF], ids=["f32", "bf16"])
def test_sample_any_alignment(dtype):
    for off in range(1, 8):
        V = 4001 + off
        buf = _logits("zipf", (1, 1, 4 * V + 8), dtype, off).flatten()
        _sample(buf[off:off + 4 * V].view(2, 2, V), [ASKS[2], ASKS[3]], off, f"offset {off}")


def test_sample_without_filters_and_in_part():
    z = _logits("zipf", (3, 2, 999), torch.float32, 1)
    u = torch.rand((3, 2), device=DEV)
    off = [(1.0, 0, 1.0, 0.0)] * 3
    t, p, m, _ = oracle.sample(z.double().cpu().numpy(), u.double().cpu().numpy(), off)
    for f in (None, sv.Filters(), sv.Filters.fill(3, DEV)):
        tokens, _ = sv.spec_filter_sample(z, u, f)
        assert ((tokens.cpu().numpy() == t) | (m < NEAR)).all()
    t, p, m, _ = oracle.sample(z.double().cpu().numpy(), u.double().cpu().numpy(), [(1.0, 5, 1.0, 0.0)] * 3)
    tokens, _ = sv.spec_filter_sample(z, u, sv.Filters(top_k=torch.full((3,), 5, dtype=torch.int32, device=DEV)))
    assert ((tokens.cpu().numpy() == t) | (m < NEAR)).all()


@pytest.mark.parametrize("ask", [ASKS[0], ASKS[2], ASKS[3], ASKS[1]])
@pytest.mark.parametrize("V", [50, 5003])
def test_sample_bad_rows_are_told_and_leave_the_others(ask, V):
    z = _logits("normal", (6, 1, V), torch.float32, 3)
    z[0, 0, V - 1] = math.nan
    z[1, 0, 3] = math.inf
    z[2, 0] = -math.inf
    u = torch.rand((6, 1), device=DEV)
    u[4, 0] = 1.0
    f, exact = _filters([ask] * 6)
    st = torch.zeros((1,), dtype=torch.int32, device=DEV)
    tokens, prob = sv.spec_filter_sample(z, u, f, device_status=st)
    t, p, m, code = oracle.sample(z.double().cpu().numpy(), u.double().cpu().numpy(), exact)
    assert code[:, 0].tolist() == [2, 2, 2, 0, 1, 0]
    assert int(st) in (1, 2)
    assert ((tokens.cpu().numpy() == t) | (m < NEAR)).all()
    assert (torch.isnan(prob).cpu().numpy() == (code > 0)).all()


def test_sample_bad_filters():
    nan = math.nan
    asks = [(nan, 0, 1.0, 0.0), (-1.0, 0, 1.0, 0.0), (math.inf, 0, 1.0, 0.0), (1.0, 0, nan, 0.0), (1.0, 0, 1.0, nan),
            (1.0, 0, 1.0, 1.5), (1.0, 0, 1.0, 0.5)]
    z = _logits("normal", (7, 1, 3000), BF, 3)
    tokens, prob = sv.spec_filter_sample(z, torch.full((7, 1), 0.5, device=DEV), _filters(asks)[0])
    assert (tokens[:6] == -1).all() and torch.isnan(prob[:6]).all() and int(tokens[6]) >= 0


def _verify(target, draft, drafted, u, asks, draft_asks, what, **kw):
    f, exact = _filters(asks)
    df, dexact = _filters(draft_asks) if draft_asks is not None else (None, None)
    st = torch.full((1,), -5, dtype=torch.int32, device=DEV)
    tokens, n = sv.spec_verify_filtered(target, draft, drafted, u, f, draft_filters=df, device_status=st, **kw)
    torch.cuda.synchronize()
    t, want, margin = oracle.verify(target.double().cpu().numpy(), draft.double().cpu().numpy(),
                                    drafted.cpu().numpy(), u.double().cpu().numpy(), exact, dexact)
    assert int(st) == max(0, int(st)) and (int(st) != 0) == (want < 0).any(), what
    near = margin < NEAR
    assert near.sum() <= 2 + 0.03 * near.size, what
    n, tokens = n.cpu().numpy(), tokens.cpu().numpy()
    bad = ((n != want) | (tokens != t).any(-1)) & ~near
    assert not bad.any(), f"{what}: sequences {np.nonzero(bad)[0][:5]}, {n[bad][:5]} not {want[bad][:5]}, {tokens[bad][:3]} not {t[bad][:3]}"
    return want


def _pair(kind, B, K, V, dtype, seed, noise=0.4):
    g = torch.Generator(device=DEV).manual_seed(seed)
    target = _logits(kind, (B, K + 1, V), torch.float32, seed)
    draft = target[:, :K] + noise * torch.randn((B, K, V), generator=g, device=DEV)
    return target.to(dtype), draft.to(dtype).contiguous(), torch.rand((B, K + 1, 2), generator=g, device=DEV), g


@pytest.mark.parametrize("kind", ["normal", "zipf", "ties", "equal", "masked"])
@pytest.mark.parametrize("dtype", [torch.float32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("V,K", [(1, 1), (3, 31), (40, 3), (1500, 4), (6007, 2)])
def test_verify(kind, dtype, V, K):
    B = 2 * len(ASKS)
    asks = ASKS + ASKS
    target, draft, u, g = _pair(kind, B, K, V, dtype, V + K)
    f, _ = _filters(asks)
    drafted, _ = sv.spec_filter_sample(draft, torch.rand((B, K), generator=g, device=DEV), f)
    want = _verify(target, draft, drafted, u, asks, None, f"{kind} {V}")
    assert V == 1 or len(set(want.tolist())) > 1
    # other filters on the draft, and drafts from nowhere
    other = asks[7:] + asks[:7]
    drafted = torch.randint(0, V, (B, K), generator=g, device=DEV, dtype=torch.int32)
    _verify(target, draft, drafted, u, asks, other, f"{kind} {V}, other filters")


@pytest.mark.parametrize("dtype,V", [(BF, 128256), (torch.float32, 32003), (BF, 262144)])
def test_verify_large(dtype, V):
    asks = [ASKS[i] for i in (0, 1, 2, 3, 4, 8)]
    target, draft, u, g = _pair("zipf", 6, 2, V, dtype, V)
    drafted, _ = sv.spec_filter_sample(draft, torch.rand((6, 2), generator=g, device=DEV), _filters(asks)[0])
    _verify(target, draft, drafted, u, asks, None, f"{V}")


def test_verify_equal_rows_accept_everything_and_strangers_nothing():
    target, _, u, g = _pair("zipf", 8, 3, 4000, torch.float32, 9)
    draft = target[:, :3].contiguous()
    asks = [(1.0, 0, 0.9, 0.0)] * 4 + [(0.8, 40, 0.95, 0.0)] * 4
    f, _ = _filters(asks)
    drafted, _ = sv.spec_filter_sample(draft, torch.rand((8, 3), generator=g, device=DEV), f)
    assert (_verify(target, draft, drafted, u, asks, None, "equal rows") == 3).all()
    # a token that neither keeps is rejected, and what is left of q beside p = q is q
    drafted = target[:, :3].argmin(-1).to(torch.int32)
    assert (_verify(target, draft, drafted, u, asks, None, "strangers") == 0).all()


def test_verify_errors_where_the_rule_reaches_them():
    B, K, V = 8, 3, 2000
    target, draft, u, g = _pair("zipf", B, K, V, torch.float32, 4, noise=0.0)
    draft = target[:, :K].contiguous()
    asks = [(1.0, 0, 0.95, 0.0)] * B
    asks[7] = (1.0, 0, math.nan, 0.0)
    f, _ = _filters(asks)
    drafted = target[:, :K].argmax(-1).to(torch.int32)
    drafted[0, 1] = V
    drafted[1, 0] = -1
    target[2, 3, 5] = math.nan
    draft[3, 2, 5] = math.inf
    drafted[4, 0] = int(target[4, 0].argmin())       # rejected ahead of the bad row
    target[4, 1] = -math.inf
    u[5, 1, 0] = 1.5
    u[6, 3, 1] = -0.25
    want = _verify(target, draft, drafted, u, asks, None, "errors")
    assert want.tolist() == [-3, -3, -2, -2, 0, -1, -1, -1]


def test_streams_graphs_and_workspaces():
    B, K, V = 16, 3, 5000
    asks = [ASKS[i % len(ASKS)] for i in range(B)]
    target, draft, u, g = _pair("zipf", B, K, V, BF, 11)
    f, _ = _filters(asks)
    v = torch.rand((B, K), generator=g, device=DEV)
    drafted, prob = sv.spec_filter_sample(draft, v, f)
    tokens, n = sv.spec_verify_filtered(target, draft, drafted, u, f)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    d2, p2 = sv.spec_filter_sample(draft, v, f, stream=s)
    t2, n2 = sv.spec_verify_filtered(target, draft, d2, u, f, stream=s)
    with torch.cuda.stream(s):
        ws = torch.full((sv.spec_filter_workspace_bytes(B, K, V),), 255, dtype=torch.uint8, device=DEV)
        t3, n3 = sv.spec_verify_filtered(target, draft, d2, u, f, workspace=ws)
    s.synchronize()
    for a, b in ((d2, drafted), (p2, prob), (t2, tokens), (n2, n), (t3, tokens), (n3, n)):
        assert torch.equal(a, b)
    graphs, outs = [], []
    for _ in range(2):                 # two graphs with memory of their own, replayed in turn
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            d = sv.spec_filter_sample(draft, v, f)[0]
            outs.append((d, *sv.spec_verify_filtered(target, draft, d, u, f)))
        graphs.append(gr)
    for _ in range(3):
        for gr, (d, t, m) in zip(graphs, outs):
            for x in (d, t, m):
                x.fill_(-7)
            gr.replay()
        torch.cuda.synchronize()
        for d, t, m in outs:
            assert torch.equal(d, drafted) and torch.equal(t, tokens) and torch.equal(m, n)
    draft.copy_(target[:, :K])         # a replay reads what is there then
    graphs[0].replay()
    torch.cuda.synchronize()
    again = sv.spec_verify_filtered(target, draft, sv.spec_filter_sample(draft, v, f)[0], u, f)
    assert torch.equal(outs[0][1], again[0]) and torch.equal(outs[0][2], again[1])


def test_results_do_not_depend_on_the_batch():
    """The same row alone and among others: other cluster sizes, the same sums."""
    V = 20011
    asks = [ASKS[i % len(ASKS)] for i in range(400)]
    z = _logits("zipf", (400, 1, V), BF, 2)
    u = torch.rand((400, 1), device=DEV)
    f, _ = _filters(asks)
    tokens, prob = sv.spec_filter_sample(z, u, f)
    for b in range(0, 400, 37):
        one = sv.Filters(*[getattr(f, x)[b:b + 1].clone() for x in sv.Filters.__slots__])
        t, p = sv.spec_filter_sample(z[b:b + 1].contiguous(), u[b:b + 1].contiguous(), one)
        assert int(t) == int(tokens[b]) and float(p) == float(prob[b])
