"""Attention of the verification pass (CUDA, through the C ABI) against the
float64 oracle.

Tolerances, from the roundings on the way (half a step of bfloat16 is 2^-8
relative, of float32 2^-24):
  - a score is off by at most `ds`: the bfloat16 products are exact, and the sum of D
    of them and the scaling round to float32 (D + 4 times at most, each relative
    to the sum of magnitudes, `reach`); 2^x and the subtraction of the maximum
    add 2^-20 of a weight at most;
  - a weight is rounded to bfloat16 where it meets the values (2^-8 of it), the sums
    of n weighted values round n times; both are relative to `mass`, the weighted
    mean of |v|; the normalisation and the output round once more (2^-8 of it);
  - lse takes a relative error of the sum as an absolute one, and rounds itself.
"""
from __future__ import annotations

import math

import pytest
import torch

import speculative_decoding_verification_sampling_gb300 as sv
from oracle.attention import attention

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(DEV)
    sv.load()


def _values(x, scale):
    return x.double() if scale is None else x.double() * torch.exp2(scale.double() - 127)[..., None]


def _hold(out, lse, ref, D, what):
    n = ref["count"]
    ds = (D + 4) * 2.0 ** -24 * ref["reach"]
    rel = 2 * ds + 2.0 ** -20 + n * 2.0 ** -24
    tol = 1.01 * (2.0 ** -8 * ref["out"].abs() + (2.0 ** -8 + rel)[..., None] * ref["mass"]) + 1e-37
    err = (out.double() - ref["out"]).abs()
    assert bool((err <= tol).all()), f"{what}: out off by {float((err / tol).max()):.3g} of its tolerance"
    none = n == 0
    assert bool((lse[none] == -math.inf).all()), f"{what}: lse of rows that see nothing"
    tol = 1.01 * (rel + 2.0 ** -22 * (ref["lse"].abs() + ref["reach"]))
    err = (lse.double() - ref["lse"]).abs()[~none]
    assert bool((err <= tol[~none]).all()), f"{what}: lse off by {float((err / tol[~none]).max()):.3g} of its tolerance"


def _codes(g, *shape):
    z = torch.randn(shape, generator=g, device=DEV)
    z *= 447.0 / z.abs().amax(-1, keepdim=True)
    return z.to(torch.float8_e4m3fn), torch.randint(117, 122, shape[:-1], generator=g, device=DEV, dtype=torch.uint8)


def _tree(g, B, T):
    par = torch.tensor([[-1] + [int(torch.randint(0, n, (1,), generator=g)) for n in range(1, T)] for _ in range(B)],
                       dtype=torch.int32, device=DEV)
    return sv.spec_tree_mask(par)


def _case(B, T, Hq, H, D, P, L, lens, quant, kind, seed=0, stale=float("nan")):
    """Inputs whose invisible places hold `stale`: entries past a sequence's
    length, and (kind "holes") staged entries that no row sees."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device=DEV).to(BF)   # noqa: E731
    a = dict(q=r(B, T, Hq, D), seq_len=torch.tensor(lens, dtype=torch.int32, device=DEV))
    if quant:
        a["cache"], a["cache_scale"] = _codes(g, B, L, 2, H, D)
        if P:
            a["prefix"], a["prefix_scale"] = _codes(g, P, 2, H, D)
    else:
        a["cache"] = r(B, L, 2, H, D)
        if P:
            a["prefix"] = r(P, 2, H, D)
    if kind != "none":
        a["staged"] = r(B, T, 2, H, D)
    if kind == "tree":
        a["mask"] = _tree(torch.Generator().manual_seed(seed), B, T)
    if kind == "holes":
        a["mask"] = (torch.rand((B, T, T), generator=g, device=DEV) < 0.4).to(torch.uint8) * 255
        a["mask"][:, 0] = 0                    # a row that sees no staged entry
        a["mask"][:, :, T // 2] = 0            # an entry that no row sees
        a["staged"][:, T // 2] = stale
    for b, n in enumerate(lens):
        if quant:
            a["cache_scale"][b, n:] = 255      # NaN
            a["cache"][b, n:] = 448.0
        else:
            a["cache"][b, n:] = stale
    return a


def _reference(a, sm_scale=None):
    clean = {k: v for k, v in a.items()}
    pre = a.get("prefix")
    return attention(a["q"], _values(clean["cache"], a.get("cache_scale")), a["seq_len"].tolist(), a.get("staged"),
                     a.get("mask"), None if pre is None else _values(pre, a.get("prefix_scale")), sm_scale)


def _run(a, what, sm_scale=None, **kw):
    st = torch.full((1,), -5, dtype=torch.int32, device=DEV)
    out, lse = sv.spec_verify_attention(a["q"], a["cache"], a["seq_len"], staged=a.get("staged"), mask=a.get("mask"),
                                        prefix=a.get("prefix"), cache_scale=a.get("cache_scale"),
                                        prefix_scale=a.get("prefix_scale"), sm_scale=sm_scale, device_status=st, **kw)
    torch.cuda.synchronize()
    assert int(st.item()) == 0, what
    _hold(out, lse, _reference(a, sm_scale), a["q"].shape[-1], what)
    return out, lse


SHAPES = [
    # B, T, Hq, H, D, P, L, lens
    (1, 1, 1, 1, 64, 0, 1, [0]),                     # nothing at all but the token itself
    (1, 1, 1, 1, 128, 0, 1, [1]),
    (2, 1, 8, 2, 128, 1, 3, [0, 3]),
    (3, 5, 8, 2, 128, 127, 300, [128, 129, 300]),
    (3, 5, 32, 8, 128, 128, 257, [0, 255, 256]),
    (4, 5, 32, 8, 64, 129, 130, [1, 127, 0, 130]),
    (5, 3, 20, 4, 64, 333, 400, [400, 7, 0, 1, 129]),
    (2, 32, 10, 2, 128, 500, 200, [200, 13]),        # 160 rows to a key head
    (2, 61, 16, 2, 128, 70, 300, [300, 41]),         # 488 rows to a key head
    (7, 9, 12, 12, 128, 1000, 150, [0, 0, 0, 150, 1, 2, 3]),
    (1, 2, 256, 2, 128, 40, 90, [77]),               # 128 query heads to a key head
    (1, 3, 129, 3, 64, 40, 90, [90]),
    (33, 4, 4, 1, 128, 260, 30, list(range(0, 31)) + [30, 0]),
    (40, 5, 8, 2, 64, 2100, 60, [(7 * i) % 61 for i in range(40)]),   # 800 rows over the prefix
    (70, 4, 8, 2, 128, 1000, 300, [(11 * i) % 301 for i in range(70)]),   # 1120 rows over the prefix
    (33, 8, 4, 1, 64, 515, 20, [(3 * i) % 21 for i in range(33)]),        # 1056
    (2, 1, 8, 8, 128, 0, 5000, [5000, 4111]),
    (3, 9, 8, 2, 128, 0, 2500, [2500, 1300, 1025]),  # 36 rows to a key head, long stretches
    (2, 20, 8, 2, 64, 300, 3000, [3000, 1025]),      # 80
]


@pytest.mark.parametrize("kind", ["causal", "tree", "holes", "none"])
@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s[:7])))
def test_matches_oracle(shape, quant, kind):
    B, T, Hq, H, D, P, L, lens = shape
    a = _case(B, T, Hq, H, D, P, L, lens, quant, kind, seed=B * 31 + T)
    _run(a, f"{shape} {quant} {kind}")


@pytest.mark.parametrize("quant", [False, True])
def test_a_prefix_and_no_cache(quant):
    g = torch.Generator(device=DEV).manual_seed(21)
    r = lambda *s: torch.randn(s, generator=g, device=DEV).to(BF)   # noqa: E731
    for B in (2, 300):
        a = dict(q=r(B, 4, 4, 64), cache=r(B, 0, 2, 1, 64),
                 seq_len=torch.zeros(B, dtype=torch.int32, device=DEV), staged=r(B, 4, 2, 1, 64))
        if quant:
            a["cache"] = a["cache"].to(torch.float8_e4m3fn)
            a["cache_scale"] = torch.zeros((B, 0, 2, 1), dtype=torch.uint8, device=DEV)
            a["prefix"], a["prefix_scale"] = _codes(g, 700, 2, 1, 64)
        else:
            a["prefix"] = r(700, 2, 1, 64)
        _run(a, f"prefix alone, {B}")


def test_no_prefix_no_cache():
    """A capacity of 0: the pass's own entries alone."""
    g = torch.Generator(device=DEV).manual_seed(1)
    r = lambda *s: torch.randn(s, generator=g, device=DEV).to(BF)   # noqa: E731
    a = dict(q=r(2, 4, 4, 64), cache=r(2, 0, 2, 2, 64), seq_len=torch.zeros(2, dtype=torch.int32, device=DEV),
             staged=r(2, 4, 2, 2, 64))
    _run(a, "no cache")
    a.pop("staged")
    out, lse = _run(a, "nothing")
    assert not out.any() and bool((lse == -math.inf).all())


@pytest.mark.parametrize("sm_scale", [1e-3, 0.5, 4.0])
def test_scales_and_peaked_rows(sm_scale):
    """At scale 4 a row's weight sits on one entry; its score is far from the first entries'."""
    a = _case(3, 5, 8, 2, 128, 600, 500, [500, 0, 257], False, "causal", seed=4)
    a["q"][0] *= 4
    _run(a, f"scale {sm_scale}", sm_scale)


def test_rising_scores():
    """Each entry scores higher than the ones before: the running maximum moves all along."""
    a = _case(2, 5, 8, 2, 64, 700, 400, [400, 130], False, "causal", seed=5)
    up = torch.linspace(0.01, 3, 700, device=DEV)[:, None, None]
    a["q"][:] = a["q"][:1, :1, :1].abs()
    a["prefix"][:, 0] = (a["q"][0, 0, 0] * up).to(BF)
    a["cache"][:, :, 0] = torch.where(a["cache"][:, :, 0].isnan(), a["cache"][:, :, 0],
                                      (a["q"][0, 0, 0] * torch.linspace(3, 6, 400, device=DEV)[:, None, None]).to(BF))
    _run(a, "rising", 0.5)


def test_infinite_and_nan_entries_where_seen():
    """A NaN that a row sees is its result; rows that do not see it keep theirs."""
    a = _case(2, 3, 4, 2, 64, 10, 20, [5, 20], False, "causal", seed=6)
    clean_out, clean_lse = _run(a, "clean")
    a["staged"][0, 1, 1, 0, 7] = float("nan")      # seen by tokens 1, 2 of sequence 0, heads 0, 1; a value
    a["cache"][1, 3, 0, 1, 5] = float("inf")       # seen by all of sequence 1, heads 2, 3; a key
    a["q"][1, :, 2:, 5] = 1.0
    out, lse = sv.spec_verify_attention(a["q"], a["cache"], a["seq_len"], staged=a["staged"], prefix=a["prefix"])
    assert torch.equal(out[0, 0], clean_out[0, 0]) and torch.equal(lse[0], clean_lse[0])
    assert bool(out[0, 1:, :2, 7].isnan().all()) and torch.equal(out[0, 1:, 2:], clean_out[0, 1:, 2:])
    assert bool(out[1, :, 2:].isnan().all()) and torch.equal(out[1, :, :2], clean_out[1, :, :2])


def test_a_score_of_minus_infinity_has_no_weight():
    a = _case(1, 2, 2, 1, 64, 6, 300, [300], False, "causal", seed=7)
    a["q"][..., 0] = 1.0
    keep = a["cache"].clone()
    a["cache"][0, 2:, 0, 0, 0] = float("-inf")
    a["cache"][0, 2:, 1] = 3.0
    out, lse = sv.spec_verify_attention(a["q"], a["cache"], a["seq_len"], staged=a["staged"], prefix=a["prefix"])
    a["cache"] = keep
    a["seq_len"].fill_(2)
    ref = _reference(a)
    ref["count"] += 298
    _hold(out, lse, ref, 64, "minus infinity")


def test_bad_lengths_are_reported_and_the_rest_is_right():
    a = _case(4, 5, 8, 2, 128, 200, 60, [60, 10, 0, 33], False, "causal", seed=8)
    want, want_lse = _run(a, "before")
    a["seq_len"][1], a["seq_len"][2] = 61, -1
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    out, lse = sv.spec_verify_attention(a["q"], a["cache"], a["seq_len"], staged=a["staged"], prefix=a["prefix"],
                                        device_status=st)
    assert int(st.item()) == 1
    assert bool(out[1:3].isnan().all()) and bool(lse[1:3].isnan().all())
    ref = {k: v[[0, 3]] for k, v in _reference({**a, "seq_len": torch.tensor([60, 0, 0, 33])}).items()}
    _hold(out[[0, 3]], lse[[0, 3]], ref, 128, "the rest")


def test_offsets_past_32_bits():
    """The last sequences of a cache of 5 GB, and of one of 5 G codes."""
    L, H, D = 300_000, 8, 128
    for quant in (False, True):
        B = 9 if quant else 5
        g = torch.Generator(device=DEV).manual_seed(9)
        lens = [0] * (B - 1) + [700]
        a = dict(q=torch.randn((B, 2, 16, D), generator=g, device=DEV).to(BF),
                 seq_len=torch.tensor(lens, dtype=torch.int32, device=DEV),
                 staged=torch.randn((B, 2, 2, H, D), generator=g, device=DEV).to(BF))
        if quant:
            a["cache"] = torch.empty((B, L, 2, H, D), dtype=torch.float8_e4m3fn, device=DEV)
            a["cache_scale"] = torch.full((B, L, 2, H), 255, dtype=torch.uint8, device=DEV)
            a["cache"][-1, :700], a["cache_scale"][-1, :700] = _codes(g, 700, 2, H, D)
            small = dict(a, cache=a["cache"][:, :700].clone(), cache_scale=a["cache_scale"][:, :700].clone())
        else:
            a["cache"] = torch.empty((B, L, 2, H, D), dtype=BF, device=DEV)
            a["cache"][-1, :700] = torch.randn((700, 2, H, D), generator=g, device=DEV).to(BF)
            small = dict(a, cache=a["cache"][:, :700].clone())
        out, lse = sv.spec_verify_attention(a["q"], a["cache"], a["seq_len"], staged=a["staged"],
                                            cache_scale=a.get("cache_scale"))
        _hold(out, lse, _reference(small), D, f"quant {quant}")
        del a, small


def test_one_layer_of_a_cache_and_given_outputs_on_a_side_stream():
    g = torch.Generator(device=DEV).manual_seed(10)
    a = _case(3, 4, 8, 2, 64, 90, 50, [50, 3, 20], False, "causal", seed=10)
    layers = torch.randn((3, 3, 50, 2, 2, 64), generator=g, device=DEV).to(BF)
    layers[1] = a["cache"]
    a["cache"] = layers[1]
    out = torch.empty_like(a["q"])
    lse = torch.empty((3, 4, 8), device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = sv.spec_verify_attention(a["q"], a["cache"], a["seq_len"], staged=a["staged"], prefix=a["prefix"], out=out,
                                   lse=lse, stream=side)
    side.synchronize()
    assert got[0] is out and got[1] is lse
    _hold(out, lse, _reference(a), 64, "side stream")


def test_repeatable_and_captured():
    """Two calls give the same bits, and so does a replay of a captured call on changed inputs."""
    a = _case(6, 5, 16, 4, 128, 1500, 700, [700, 0, 5, 256, 511, 90], True, "causal", seed=11)
    call = lambda: sv.spec_verify_attention(   # noqa: E731
        a["q"], a["cache"], a["seq_len"], staged=a["staged"], prefix=a["prefix"], cache_scale=a["cache_scale"],
        prefix_scale=a["prefix_scale"])
    one, two = call(), call()
    assert torch.equal(one[0], two[0]) and torch.equal(one[1], two[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = call()
    a["q"].copy_(a["q"].flip(0))
    a["seq_len"].copy_(torch.tensor([3, 0, 5, 200, 500, 90], dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    _hold(*held, _reference(a), 128, "replay")


def test_the_round_with_an_8_bit_cache():
    """Attention over the 8-bit cache is attention over what it reads back as."""
    g = torch.Generator(device=DEV).manual_seed(12)
    B, T, H, D, L = 4, 5, 2, 64, 40
    c = torch.zeros((1, B, L, 2, H, D), dtype=torch.float8_e4m3fn, device=DEV)
    s = torch.full((1, B, L, 2, H), 127, dtype=torch.uint8, device=DEV)
    n = torch.zeros(B, dtype=torch.int32, device=DEV)
    for step in range(4):
        staged = torch.randn((1, B, T, 2, H, D), generator=g, device=DEV).to(BF)
        q = torch.randn((B, T, 8, D), generator=g, device=DEV).to(BF)
        back = sv.spec_kv_read_quant(c, s, None, n, L)
        x = sv.spec_verify_attention(q, c[0], n, staged=staged[0], cache_scale=s[0])
        y = sv.spec_verify_attention(q, back[0], n, staged=staged[0])
        ref = attention(q, back[0], n.tolist(), staged[0])
        _hold(*x, ref, D, f"8 bits, step {step}")
        _hold(*y, ref, D, f"16 bits, step {step}")
        sv.spec_kv_commit_quant(c, s, staged, torch.tensor([4, 0, -2, step], dtype=torch.int32, device=DEV), n, lead=1)
    assert n.tolist() == [20, 4, 0, 10]


def test_many_rows_with_bad_lengths():
    """More rows than get a CTA each in the finishing kernel."""
    lens = [(13 * i) % 41 for i in range(90)]
    a = _case(90, 5, 8, 2, 64, 150, 40, lens, False, "tree", seed=13)
    _run(a, "before")
    a["seq_len"][7], a["seq_len"][89] = 41, -3
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    out, lse = sv.spec_verify_attention(a["q"], a["cache"], a["seq_len"], staged=a["staged"], mask=a["mask"],
                                        prefix=a["prefix"], device_status=st)
    assert int(st.item()) == 1
    keep = [b for b in range(90) if b not in (7, 89)]
    assert bool(out[[7, 89]].isnan().all()) and bool(lse[[7, 89]].isnan().all())
    lens[7] = lens[89] = 0
    ref = {k: v[keep] for k, v in _reference({**a, "seq_len": torch.tensor(lens)}).items()}
    _hold(out[keep], lse[keep], ref, 64, "the rest")


def test_scales_far_apart_within_a_unit():
    """Heads of very different magnitudes side by side: what a unit's largest scale leaves of the others."""
    for big in (20, 60):
        a = _case(2, 3, 8, 2, 128, 200, 300, [300, 170], True, "causal", seed=14)
        a["cache_scale"][:, 5::7] -= big          # 2^-20, 2^-60 of the others
        a["prefix_scale"][::3] -= big
        _run(a, f"2^-{big}")
        a["cache_scale"][:, :170] = a["cache_scale"][:, :170].clamp(min=60) - 50   # and everything small
        a["prefix_scale"].clamp_(min=60).sub_(50)
        a["staged"] *= 2.0 ** -50
        _run(a, f"2^-{big}, small")


def test_heads_that_read_back_as_nan():
    """Scale byte 255 where a row sees it, in a key and in a value."""
    a = _case(2, 2, 4, 2, 64, 10, 400, [200, 400], True, "causal", seed=15)
    clean = _run(a, "clean")
    a["cache_scale"][0, 130, 0, 1] = 255     # a key: the whole row
    a["cache_scale"][1, 300, 1, 0] = 255     # a value: every column
    out, lse = sv.spec_verify_attention(a["q"], a["cache"], a["seq_len"], staged=a["staged"], prefix=a["prefix"],
                                        cache_scale=a["cache_scale"], prefix_scale=a["prefix_scale"])
    assert bool(out[0, :, 2:].isnan().all()) and bool(lse[0, :, 2:].isnan().all())
    assert bool(out[1, :, :2].isnan().all()) and torch.equal(lse[1], clean[1][1])
    assert torch.equal(out[0, :, :2], clean[0][0, :, :2]) and torch.equal(out[1, :, 2:], clean[0][1, :, 2:])


def test_the_example_runs():
    import os
    import sys
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import verification_round
    assert 1.0 <= verification_round.main(rounds=3) <= 5.0


@pytest.mark.parametrize("quant", [False, True])
def test_workspace_at_any_16_bytes_and_launches(quant):
    """The workspace lies where the caller has room: 16-byte aligned, no further."""
    a = _case(3, 5, 8, 2, 128, 150, 300, [300, 0, 131], quant, "tree", seed=16)
    keys = ("q", "cache", "seq_len")
    args = [a[k] for k in keys]
    kw = {k: v for k, v in a.items() if k not in keys and isinstance(v, torch.Tensor)}
    want = sv.spec_verify_attention(*args, **kw)
    need = sv.spec_attention_workspace_bytes(3, 5, 8, 2, 128, 150, 300)
    room = torch.full((need + 512,), 0xff, dtype=torch.uint8, device=DEV)
    for at in (16, 48, 240):
        before = sv.spec_launch_count()
        got = sv.spec_verify_attention(*args, workspace=room[at:at + need], **kw)
        assert sv.spec_launch_count() - before == 2
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        assert bool((room[:at] == 0xff).all()) and bool((room[at + need:] == 0xff).all())


@pytest.mark.parametrize("B,T,Hq,H,D,P,L,quant", [
    (1, 1, 32, 1, 128, 0, 90001, False),    # one pair over every CTA: hundreds of partial results to a row
    (1, 2, 48, 1, 64, 1000, 60000, True),
    (2, 3, 86, 2, 128, 700, 20000, False),  # just past the rows that have 16 warps each
])
def test_few_rows_over_long_caches(B, T, Hq, H, D, P, L, quant):
    a = _case(B, T, Hq, H, D, P, L, [L - 77 * b for b in range(B)], quant, "causal", seed=17)
    _run(a, f"{B * T * Hq} rows over {L} entries")


@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("kind", ["causal", "holes"])
@pytest.mark.parametrize("B,T,Hq,H,D,P,L", [(2, 62, 4, 1, 64, 130, 300), (2, 129, 4, 2, 128, 70, 140), (1, 512, 8, 2, 64, 300, 129),
                                            (1, 513, 2, 2, 128, 0, 0), (1, 2048, 2, 1, 64, 129, 257)])
def test_many_tokens(B, T, Hq, H, D, P, L, kind, quant):
    """Passes longer than a draft tree's, to the most that a call takes."""
    a = _case(B, T, Hq, H, D, P, L, [L - 100 * b for b in range(B)], quant, kind, seed=18)
    _run(a, f"{T} tokens")
