"""Attention of the verification pass (CUDA, through the C ABI): what NaN, scores
and scales far from the ordinary do, against the float64 oracle.
"""
from __future__ import annotations

import pytest
import torch

import speculative_decoding_verification_sampling_gb300 as sv
from test_gpu_attention import _case, _device   # noqa: F401

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

