"""The windowed attention over passes of many tokens (parts of a prompt), up to
2048: windows shorter than the pass, about as long, and longer.  Oracle and
tolerances as in test_gpu_window_attention.py."""
from __future__ import annotations

import pytest
import torch

import speculative_decoding_verification_sampling_gb300 as sv
from oracle.attention import window_attention
from test_gpu_attention import _case, _hold, _values

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(DEV)
    sv.load()


CASES = [
    # B, T, Hq, H, D, L, window, sinks, lens, kind, quant
    (2, 64, 8, 2, 128, 300, 63, 4, [300, 40], "tree", False),
    (2, 64, 8, 2, 128, 300, 63, 4, [300, 40], "causal", True),
    (2, 130, 4, 1, 64, 400, 129, 0, [400, 77], "holes", False),
    (2, 130, 4, 1, 64, 400, 129, 0, [400, 77], "causal", True),
    (1, 512, 4, 2, 128, 700, 100, 4, [640], "causal", False),    # every window ends in the pass
    (1, 512, 4, 2, 128, 700, 100, 4, [640], "tree", True),
    (2, 512, 2, 1, 64, 1500, 513, 130, [1500, 90], "causal", False),
    (1, 512, 4, 4, 128, 1500, 900, 4, [1500], "holes", False),   # windows from the cache, edges of up to 511 entries
    (1, 512, 4, 4, 128, 1500, 900, 4, [1500], "causal", True),
    (1, 2048, 2, 1, 128, 500, 300, 4, [500], "causal", False),
    (1, 2048, 2, 2, 64, 2600, 2300, 16, [2600], "causal", True),
]


@pytest.mark.parametrize("case", CASES, ids=lambda s: "-".join(map(str, s[:8] + s[9:])))
def test_long_pass(case):
    B, T, Hq, H, D, L, window, sinks, lens, kind, quant = case
    a = _case(B, T, Hq, H, D, 0, L, lens, quant, kind, seed=T + window)
    st = torch.full((1,), -5, dtype=torch.int32, device=DEV)
    out, lse = sv.spec_verify_window_attention(a["q"], a["cache"], a["seq_len"], window, sinks=sinks,
                                               staged=a["staged"], mask=a.get("mask"), cache_scale=a.get("cache_scale"),
                                               device_status=st)
    torch.cuda.synchronize()
    assert int(st) == 0
    mask = a["mask"].cpu() if "mask" in a else None
    ref = window_attention(a["q"], _values(a["cache"], a.get("cache_scale")), lens, window, sinks, a["staged"], mask)
    _hold(out, lse, ref, D, f"{case}")


def test_longest_pass_under_its_causal_mask():
    """2048 tokens under the mask that a call without one has."""
    a = _case(1, 2048, 2, 1, 64, 0, 900, [900], False, "causal", seed=1)
    mask = torch.ones((2048, 2048), dtype=torch.uint8, device=DEV).tril()[None].contiguous()
    for window in (200, 1500, 2500):
        kw = dict(sinks=4, staged=a["staged"])
        want = sv.spec_verify_window_attention(a["q"], a["cache"], a["seq_len"], window, **kw)
        got = sv.spec_verify_window_attention(a["q"], a["cache"], a["seq_len"], window, mask=mask, **kw)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
