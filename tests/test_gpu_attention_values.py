"""Attention of the verification pass (CUDA, through the C ABI): what NaN, scores
and scales far from the ordinary do, against the float64 oracle.

Tolerances are those of test_gpu_attention.py: they count roundings of weights and
outputs (2^-8 each, relative to the weighted mean of |v|) and of scores and sums.
"""
from __future__ import annotations

import pytest
import torch

import speculative_decoding_verification_sampling_gb300 as sv
from test_gpu_attention import BF, DEV, _case, _device, _hold, _reference, _run   # noqa: F401

pytestmark = pytest.mark.gpu


def _call(a):
    keys = ("q", "cache", "seq_len")
    return sv.spec_verify_attention(*(a[k] for k in keys), **{k: v for k, v in a.items() if k not in keys})


# (shape, lens): rows with 16 warps, four warps and eight lanes each in the finishing
# kernel; long stretches (12 units and more of one set of rows); a prefix under 1024 rows
NAN_SHAPES = [
    (2, 3, 4, 2, 64, 40, 300, [300, 170]),
    (6, 5, 16, 4, 128, 200, 300, [300, 0, 7, 128, 129, 255]),
    (20, 9, 16, 2, 128, 70, 140, [(7 * i) % 141 for i in range(20)]),
    (16, 9, 8, 2, 128, 0, 30000, [30000 - 100 * i for i in range(16)]),
    (64, 8, 8, 2, 64, 300, 60, [(7 * i) % 61 for i in range(64)]),
]


@pytest.mark.parametrize("kind", ["causal", "none"])
@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("shape", NAN_SHAPES, ids=lambda s: "x".join(map(str, s[:7])))
def test_a_nan_in_a_query_is_its_rows_result(shape, quant, kind):
    """Every score of the row is NaN: so are its output and lse; the other rows keep their bits."""
    B, T, Hq, H, D, P, L, lens = shape
    a = _case(B, T, Hq, H, D, P, L, lens, quant, kind, seed=31)
    out, lse = _call(a)
    at = [(0, 0, 0), (0, T - 1, Hq - 1), (B - 1, 1, Hq // 2)]
    for i in at:
        a["q"][i][5] = float("nan")
    got, got_lse = _call(a)
    for i in at:
        assert bool(got[i].isnan().all()) and bool(got_lse[i].isnan()), i
        got[i], got_lse[i] = out[i], lse[i]
    assert torch.equal(got, out) and torch.equal(got_lse, lse)


@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("B,P,L,n", [(12, 300, 200, 150), (180, 300, 200, 150), (180, 0, 9000, 8000)])
def test_a_nan_value_stays_beside_larger_weights(B, P, L, n, quant):
    """A value that is NaN reaches the row however small its weight is: its column is NaN."""
    T, Hq, H, D = 3, 4, 2, 64
    a = _case(B, T, Hq, H, D, P, L, [n] * B, quant, "causal", seed=32)
    a["staged"][:, 0, 0, :] = 400 * a["q"][:, 0, ::2] / a["q"][:, 0, ::2].float().norm(dim=-1, keepdim=True)
    a["q"][:] = a["q"][:, :1, ::2].repeat_interleave(2, 2)    # scores of staged entry 0: 400 and more above the rest
    out, lse = _call(a)
    assert not bool(out.isnan().any())
    if quant:
        a["cache_scale"][3, n - 1, 1, 1] = 255
    else:
        a["cache"][3, n - 1, 1, 1, 7] = float("nan")
    got, got_lse = _call(a)
    hit = got[3, :, 2:] if quant else got[3, :, 2:, 7]
    assert bool(hit.isnan().all())
    hit.copy_(out[3, :, 2:] if quant else out[3, :, 2:, 7])
    assert torch.equal(got, out) and torch.equal(got_lse, lse)


# ------------------------------------------------------------------ 8-bit entries: scales and scores
def _scored(B, T, Hq, H, D, lens, score, seed, prefix=None):
    """8-bit entries whose scores are given: q has element 0 alone, and so have the keys.  score [L]
    (and prefix [P]): multiples of 1 / 8 that e4m3 holds; values are random, with scale bytes 117 .. 121."""
    L = len(score)
    P = 0 if prefix is None else len(prefix)
    a = _case(B, T, Hq, H, D, P, L, lens, True, "none", seed=seed)
    a["sm_scale"] = 0.125
    a["q"].zero_()
    a["q"][..., 0] = 1.0
    for name, s in (("cache", score), ("prefix", prefix)):
        if s is None:
            continue
        k = (8 * s).to(torch.float8_e4m3fn)
        assert torch.equal(k.double(), 8 * s), "scores that e4m3 holds"
        x, sc = a[name], a[name + "_scale"]
        x[..., 0, :, :] = 0.0
        x[..., 0, :, 0] = k[:, None]
        if name == "cache":
            for b, n in enumerate(lens):
                sc[b, :n, 0] = 127
                x[b, n:] = 448.0
        else:
            sc[:, 0] = 127
    return a


def _hold_scored(a, what):
    scale = a["sm_scale"]
    out, lse = _call(a)
    _hold(out, lse, _reference({k: v for k, v in a.items() if k != "sm_scale"}, scale), a["q"].shape[-1], what)


@pytest.mark.parametrize("kind", ["causal", "none"])
@pytest.mark.parametrize("first", [200, 60])
@pytest.mark.parametrize("B,T,P,L", [(2, 3, 0, 256), (3, 5, 256, 512), (40, 3, 256, 4096), (2, 61, 512, 300)])
@pytest.mark.parametrize("D", [64, 128])
def test_units_whose_value_scales_lie_far_apart(B, T, P, L, D, first, kind):
    """Values of 2^73 beside values of 2^-67, 128 entries each in turn: every entry has its weight,
    in the output and in lse."""
    lens = [L - 7 * b for b in range(B)]
    a = _case(B, T, 4, 2, D, P, L, lens, True, kind, seed=41)
    for name, dim in (("cache", 1), ("prefix", 0)):
        if name in a:
            n = a[name].shape[dim]
            byte = torch.where(torch.arange(n, device=DEV) // 128 % 2 == 0, first, 260 - first).to(torch.uint8)
            a[name + "_scale"][..., 1, :] = byte[:, None]
    for b, n in enumerate(lens):
        a["cache_scale"][b, n:] = 255
    _run(a, f"{first} first")


@pytest.mark.parametrize("low,high", [(60, 200), (60, 180), (100, 122), (2, 120)])
def test_the_weight_lies_on_the_small_values(low, high):
    """The entries with small values have the larger scores: what is left of the others is in range."""
    for order in (0, 1):
        score = torch.zeros(512, dtype=torch.float64, device=DEV)
        unit = torch.arange(512, device=DEV) // 128 % 2 == order
        score[unit] = -(min(high - low, 70) * 0.75 // 8 * 8)     # in nats: further than the values are apart, or 48
        a = _scored(2, 5, 8, 2, 128, [512, 300], score, 42)
        byte = torch.where(unit, high, low).to(torch.uint8)
        a["cache_scale"][0, :, 1] = byte[:, None]
        a["cache_scale"][1, :300, 1] = byte[:300, None]
        _hold_scored(a, f"{low} {high} {order}")


@pytest.mark.parametrize("D", [64, 128])
def test_the_weight_lies_on_a_small_head_of_a_unit(D):
    """One entry of a unit has nearly all of the weight and values 2^20 below its neighbours'."""
    score = torch.full((300,), -36.0, dtype=torch.float64, device=DEV)
    score[[5, 140, 290]] = 0.0
    a = _scored(3, 5, 8, 2, D, [300, 291, 128], score, 43)
    a["cache_scale"][:, :, 1] = torch.where(a["cache_scale"][:, :, 1] == 255, 255, 125)
    for i in (5, 140, 290):
        for b in range(3):
            if i < [300, 291, 128][b]:
                a["cache_scale"][b, i, 1] = 105
    _hold_scored(a, "small heads")


@pytest.mark.parametrize("gap", [11.0, 12.0, 13.0, 14.0])
@pytest.mark.parametrize("sink", ["zero", "small", "large"])
@pytest.mark.parametrize("D", [64, 128])
def test_a_dominant_entry_and_a_flat_tail(D, sink, gap):
    """One entry 2^16 to 2^20 above thousands of equal ones, whose values all agree: zeros (whose scale
    byte is 127), or values of the neighbours' scale, or small ones."""
    B, L = 40, 8193
    score = torch.full((L,), -gap, dtype=torch.float64, device=DEV)
    score[0] = 0.0
    a = _scored(B, 5, 8, 2, D, [L - 130 * b for b in range(B)], score, 44)
    a["cache"][:, :, 1] = 128.0
    for b in range(B):
        a["cache_scale"][b, :L - 130 * b, 1] = 120       # 1
    a["cache"][:, 0, 1] = 0.0 if sink == "zero" else 0.125 if sink == "small" else 128.0
    a["cache_scale"][:, 0, 1] = 127 if sink == "zero" else 120
    a["cache"][:, 1::2, 1] = torch.where(torch.rand((B, L // 2, 1, D), device=DEV,
                                                    generator=torch.Generator(device=DEV).manual_seed(3)) < 0.1,
                                         -128.0, 128.0).to(torch.float8_e4m3fn)
    if sink == "zero":
        a["cache"][:, 0, 1, :, ::3] = -0.0
    _hold_scored(a, f"{sink} {gap}")


@pytest.mark.parametrize("T", [5, 61])
@pytest.mark.parametrize("sm_scale", [1e-3, 0.5, 4.0])
def test_peaked_rows_8_bits(T, sm_scale):
    a = _case(3, T, 8, 2, 128, 600, 2500, [2500, 0, 257], True, "causal", seed=4)
    a["q"][0] *= 4
    _run(a, f"scale {sm_scale}", sm_scale)


@pytest.mark.parametrize("B,T", [(2, 5), (2, 61), (40, 3)])
@pytest.mark.parametrize("down", [False, True])
def test_rising_scores_8_bits(B, T, down):
    """Each run of entries scores higher than the ones before: the running maximum moves all along."""
    grid = torch.arange(256, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn).double() / 8
    grid = grid[~grid.isnan()].sort().values
    up = grid[(torch.arange(2900, device=DEV) * len(grid)) // 2900]
    up = up.flip(0) if down else up
    a = _scored(B, T, 8, 2, 64, [2000 - 40 * b for b in range(B)], up[900:], 45, prefix=up[:900])
    a["q"][..., 0] = torch.rand((B, T, 8), device=DEV, generator=torch.Generator(device=DEV).manual_seed(6)).to(BF) + 0.5
    a["sm_scale"] = 1.0
    _hold_scored(a, "rising")


def test_scores_of_minus_infinity_8_bits():
    """Products below float32's lowest number: no weight."""
    score = torch.zeros(300, dtype=torch.float64, device=DEV)
    a = _scored(2, 3, 4, 2, 64, [300, 129], score, 46)
    want, want_lse = _call({**a, "seq_len": torch.tensor([2, 2], dtype=torch.int32, device=DEV)})
    a["cache"][:, 2:, 0, :, 0] = -448.0
    a["cache_scale"][0, 2:, 0] = a["cache_scale"][1, 2:129, 0] = 254
    ref = _reference({**{k: v for k, v in a.items() if k != "sm_scale"}, "seq_len": torch.tensor([2, 2])}, 0.125)
    ref["count"] += 298
    _hold(*_call(a), ref, 64, "minus infinity")
    _hold(want, want_lse, ref, 64, "without them")


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("below", [22, 23, 27, 31, 32, 33, 60])
def test_values_far_below_their_units(below, D):
    """A head 2^22 below its unit's scale is exact; further down it loses 2^-40 of the unit's range,
    and from 2^32 below on it counts as 0, 2^-32 of that."""
    top, n = 127, 300
    score = torch.full((n,), -48.0, dtype=torch.float64, device=DEV)
    score[[5, 140, 290]] = 0.0
    a = _scored(2, 5, 8, 2, D, [n, 291], score, 47)
    a["cache_scale"][..., 1, :] = torch.where(a["cache_scale"][..., 1, :] == 255, 255, top)
    for i in (5, 140, 290):
        a["cache_scale"][:, i, 1] = top - below
    scale = a["sm_scale"]
    out, lse = _call(a)
    ref = _reference({k: v for k, v in a.items() if k != "sm_scale"}, scale)
    lost = 0.0 if below <= 22 else 2.0 ** -40 if below < 32 else 2.0 ** -32
    tol = 1.01 * (2.0 ** -8 * ref["out"].abs() + (2.0 ** -8 + 2.0 ** -19) * ref["mass"]) + lost * 448.0
    err = (out.double() - ref["out"]).abs()
    assert bool((err <= tol).all()), float((err / tol).max())
    _hold(ref["out"].to(BF), lse, ref, D, "lse")
