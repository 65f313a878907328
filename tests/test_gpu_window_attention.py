"""The verification attention under a sliding window with sinks (CUDA, through the
C ABI) against the float64 oracle, with spec_verify_attention's tolerances: the
same arithmetic on other entries (test_gpu_attention.py derives them).
"""
from __future__ import annotations

import math

import pytest
import torch

import speculative_decoding_verification_sampling_gb300 as sv
from oracle.attention import window_attention
from test_gpu_attention import _case, _hold, _values

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(DEV)
    sv.load()


def _call(a, window, sinks, sm_scale=None, **kw):
    return sv.spec_verify_window_attention(a["q"], a["cache"], a["seq_len"], window, sinks=sinks,
                                           staged=a.get("staged"), mask=a.get("mask"),
                                           cache_scale=a.get("cache_scale"), sm_scale=sm_scale, **kw)


def _run(a, window, sinks, what, sm_scale=None, **kw):
    st = torch.full((1,), -5, dtype=torch.int32, device=DEV)
    out, lse = _call(a, window, sinks, sm_scale, device_status=st, **kw)
    torch.cuda.synchronize()
    assert int(st.item()) == 0, what
    ref = window_attention(a["q"], _values(a["cache"], a.get("cache_scale")), a["seq_len"].tolist(), window, sinks,
                           a.get("staged"), a.get("mask"), sm_scale)
    _hold(out, lse, ref, a["q"].shape[-1], what)
    return out, lse


SHAPES = [
    # B, T, Hq, H, D, L, window, sinks, lens
    (1, 1, 1, 1, 64, 1, 1, 0, [0]),
    (1, 1, 1, 1, 128, 1, 1, 1, [1]),
    (2, 1, 8, 2, 128, 300, 1, 0, [300, 299]),            # the token alone
    (2, 1, 8, 2, 128, 300, 128, 4, [300, 130]),
    (3, 5, 8, 2, 128, 300, 4, 2, [300, 7, 1]),           # shorter than the pass
    (3, 5, 32, 8, 128, 700, 133, 4, [700, 129, 0]),      # one unit, and edges
    (4, 5, 32, 8, 64, 700, 132, 17, [700, 129, 150, 3]), # sinks of their own unit, and part of a unit
    (4, 5, 8, 2, 128, 900, 300, 130, [900, 129, 435, 436]),   # two units of sinks; where window and sinks meet
    (5, 3, 20, 4, 64, 400, 77, 130, [400, 7, 0, 131, 207]),
    (2, 32, 10, 2, 128, 500, 200, 16, [500, 213]),       # 160 rows to a key head
    (2, 61, 16, 2, 128, 300, 100, 5, [300, 41]),         # 488 rows to a key head
    (7, 9, 12, 12, 128, 150, 10 ** 10, 0, [0, 0, 0, 150, 1, 2, 3]),   # the window holds everything
    (3, 4, 8, 2, 64, 150, 3, 10 ** 10, [150, 1, 60]),    # the sinks do
    (1, 2, 256, 2, 128, 190, 50, 3, [177]),              # 128 query heads to a key head
    (1, 3, 129, 3, 64, 190, 90, 0, [190]),
    (70, 4, 8, 2, 128, 300, 140, 4, [(11 * i) % 301 for i in range(70)]),
    (33, 8, 4, 1, 64, 60, 20, 7, [(3 * i) % 61 for i in range(33)]),
    (2, 1, 8, 8, 128, 5000, 2048, 4, [5000, 4111]),
    (3, 9, 8, 2, 128, 2500, 2100, 64, [2500, 1300, 2225]),   # long stretches
    (300, 2, 8, 2, 128, 200, 64, 4, [(13 * i) % 201 for i in range(300)]),
]


@pytest.mark.parametrize("quant", [False, True], ids=["bf16", "q8"])
@pytest.mark.parametrize("kind", ["none", "causal", "tree", "holes"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, s[:8])))
def test_window(shape, kind, quant):
    B, T, Hq, H, D, L, window, sinks, lens = shape
    a = _case(B, T, Hq, H, D, 0, L, lens, quant, kind)
    _run(a, window, sinks, f"{shape[:8]} {kind} {quant}")


@pytest.mark.parametrize("quant", [False, True], ids=["bf16", "q8"])
@pytest.mark.parametrize("T,window,sinks", [(1, 40, 4), (5, 200, 4), (5, 200, 20), (9, 3, 0)])
def test_entries_outside_hold_nan(T, window, sinks, quant):
    """What no token of a sequence sees, and what some do not: a token that does not see a NaN has none."""
    lens = [700, 450, 333]
    a = _case(3, T, 8, 2, 128, 0, 700, lens, quant, "causal", seed=3)
    clean, _ = _call(a, window, sinks)
    if quant:
        def spoil(b, e):
            a["cache_scale"][b, e] = 255
    else:
        def spoil(b, e):
            a["cache"][b, e] = math.nan
    for b, n in enumerate(lens):
        spoil(b, slice(sinks, n + 1 - window))           # ahead of every window
    _run(a, window, sinks, "NaN ahead of the windows")
    if T > 1 and window > T:
        for b, n in enumerate(lens):
            spoil(b, n + 1 - window)                     # the first token's window alone reaches it
        out, lse = _call(a, window, sinks)
        assert torch.isnan(out[:, 0]).all() and torch.isnan(lse[:, 0]).all()
        assert torch.equal(out[:, 1:], clean[:, 1:])


def test_everything_in_reach_is_the_other_call():
    """With a window or sinks over everything, the entries are those of spec_verify_attention."""
    a = _case(4, 5, 8, 2, 128, 0, 600, [600, 0, 129, 511], False, "tree", seed=4)
    want = sv.spec_verify_attention(a["q"], a["cache"], a["seq_len"], staged=a["staged"], mask=a["mask"])
    for window, sinks in ((10 ** 6, 0), (10 ** 6, 5), (1, 10 ** 6)):
        got = _call(a, window, sinks)
        # both sides off by half a step of the output and of each weight, a weight's value at most the largest;
        # lse by 2 (D + 4) 2^-24 of a score's magnitudes, which are below 20 here, on either side
        most = max(float(a["cache"][b, :n].abs().max()) for b, n in enumerate([600, 0, 129, 511]) if n)
        most = max(most, float(a["staged"].abs().max()))
        assert ((got[0].float() - want[0].float()).abs() <= 2.0 ** -7 * 1.01 * (want[0].abs().float() + most)).all()
        assert ((got[1] - want[1]).abs() <= 4 * 132 * 2.0 ** -24 * 20 + 1e-5).all()


def test_long_cache_offsets_past_32_bits():
    """A cache of more than 2^32 elements, the window at its far end."""
    B, L, H, D = 2, 1 << 21, 8, 128
    cache = torch.zeros((B, L, 2, H, D), dtype=BF, device=DEV)
    assert cache.numel() > 2 ** 32
    g = torch.Generator(device=DEV).manual_seed(1)
    n = [L, L - 77]
    for b in range(B):
        cache[b, n[b] - 400:n[b]] = torch.randn((400, 2, H, D), generator=g, device=DEV).to(BF)
        cache[b, :8] = torch.randn((8, 2, H, D), generator=g, device=DEV).to(BF)
    a = dict(q=torch.randn((B, 3, 32, D), generator=g, device=DEV).to(BF), cache=cache,
             seq_len=torch.tensor(n, dtype=torch.int32, device=DEV),
             staged=torch.randn((B, 3, 2, H, D), generator=g, device=DEV).to(BF))
    out, lse = _call(a, 300, 4)
    # the same entries in a short cache
    short = torch.stack([torch.cat([cache[b, :4], cache[b, n[b] - 300:n[b]]]) for b in range(B)])
    ref = window_attention(a["q"], short, [304, 304], 300, 4, a["staged"])
    _hold(out, lse, ref, D, "long cache")


def test_bad_lengths_scales_and_outputs_given():
    a = _case(4, 3, 8, 2, 64, 0, 200, [200, 5, 17, 90], False, "causal", seed=5)
    good = _call(a, 50, 4, 0.3)
    a["seq_len"][1], a["seq_len"][2] = 201, -1
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    out, lse = torch.empty_like(good[0]), torch.empty_like(good[1])
    ws = torch.full((sv.spec_attention_workspace_bytes(4, 3, 8, 2, 64, 0, 200),), 255, dtype=torch.uint8, device=DEV)
    res = _call(a, 50, 4, 0.3, device_status=st, out=out, lse=lse, workspace=ws)
    assert res[0] is out and res[1] is lse and int(st) == 1
    assert torch.isnan(out[1:3]).all() and torch.isnan(lse[1:3]).all()
    for b in (0, 3):
        assert torch.equal(out[b], good[0][b]) and torch.equal(lse[b], good[1][b])


@pytest.mark.parametrize("kind", ["causal", "tree"])
def test_streams_and_graphs(kind):
    a = _case(6, 5, 8, 2, 128, 0, 500, [500, 3, 250, 0, 411, 140], True, kind, seed=6)
    want = _call(a, 130, 20)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = _call(a, 130, 20, stream=s)
    s.synchronize()
    assert torch.equal(other[0], want[0]) and torch.equal(other[1], want[1])
    graphs, outs = [], []
    for w in (130, 60):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(_call(a, w, 20))
        graphs.append(gr)
    wants = [want, _call(a, 60, 20)]
    for _ in range(3):
        for gr in graphs:
            gr.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, wants):
            assert torch.equal(o[0], w[0]) and torch.equal(o[1], w[1])
            o[0].fill_(7)
    a["seq_len"].copy_(torch.tensor([100, 500, 13, 499, 0, 333], dtype=torch.int32))
    graphs[0].replay()
    torch.cuda.synchronize()
    again = _call(a, 130, 20)
    # longer sequences reach what was beyond their ends, NaN: the same there, too
    for x, y in zip(outs[0], again):
        assert torch.equal(torch.isnan(x), torch.isnan(y)) and torch.equal(x.nan_to_num(nan=7.0), y.nan_to_num(nan=7.0))
