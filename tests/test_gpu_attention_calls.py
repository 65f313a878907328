"""How the verification attention is called (CUDA): from threads, on streams that
are not current, under capture, with waits that run out."""
from __future__ import annotations

import threading

import pytest
import torch

import speculative_decoding_verification_sampling_gb300 as sv
from test_gpu_attention import DEV, _case, _device   # noqa: F401

pytestmark = pytest.mark.gpu


def _call(a, **kw):
    keys = ("q", "cache", "seq_len")
    return sv.spec_verify_attention(*(a[k] for k in keys), **{k: v for k, v in a.items() if k not in keys}, **kw)


def test_two_threads_on_one_stream():
    """Each thread's results are those of the same calls alone, bit for bit."""
    shapes = [(3, 5, 8, 2, 128, 300, 400, [400, 31, 260], False, "causal"),
              (2, 9, 16, 4, 64, 0, 3000, [3000, 1999], True, "tree"),
              (64, 8, 4, 1, 64, 515, 20, [(3 * i) % 21 for i in range(64)], True, "causal")]
    cases = [[_case(*s, seed=50 + i + 10 * k) for i, s in enumerate(shapes)] for k in range(2)]
    want = [[tuple(x.clone() for x in _call(a)) for a in mine] for mine in cases]
    torch.cuda.synchronize()
    bad, both = [], threading.Barrier(2)

    def work(k):
        torch.cuda.set_device(DEV)
        both.wait()
        for r in range(200):
            i = (r + k) % 3
            out, lse = _call(cases[k][i])
            if not (torch.equal(out, want[k][i][0]) and torch.equal(lse, want[k][i][1])):
                bad.append((k, r, i))
    threads = [threading.Thread(target=work, args=(k,)) for k in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad, bad[:10]


def test_capture_on_a_stream_that_is_not_current():
    """The graph has scratch of its own: a replay neither writes nor reads what the stream's other
    calls keep, which a larger call has replaced meanwhile."""
    a = _case(3, 5, 8, 2, 128, 300, 400, [400, 31, 260], True, "causal", seed=61)
    big = _case(8, 61, 8, 2, 128, 300, 400, [400, 31, 260, 5, 6, 7, 8, 9], True, "causal", seed=62)
    want = _call(a)
    out, lse = torch.zeros_like(want[0]), torch.zeros_like(want[1])
    side, other, graph = torch.cuda.Stream(), torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    _call(a, stream=side, out=out, lse=lse)
    side.synchronize()
    out.zero_()
    torch.cuda.synchronize()
    kept = sv._kept.scratch[(0, side.cuda_stream)]
    kept.fill_(0x55)
    with torch.cuda.graph(graph, stream=side), torch.cuda.stream(other):
        _call(a, stream=side, out=out, lse=lse)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    assert bool((kept == 0x55).all())
    _call(big, stream=side)
    side.synchronize()
    assert sv._kept.scratch[(0, side.cuda_stream)].numel() > kept.numel()
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


def test_streams_by_handle():
    """A stream's handle serves as the stream does; 0 is the default stream."""
    a = _case(3, 5, 8, 2, 128, 300, 400, [400, 31, 260], False, "causal", seed=63)
    want = _call(a)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for s in (side.cuda_stream, 0, torch.cuda.default_stream()):
        with sv._on(DEV, s):
            assert torch.cuda.current_stream().cuda_stream == (s if isinstance(s, int) else 0)
        got = _call(a, stream=s)
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def _spin(stream, ms=30):
    """Keeps a stream busy for a while."""
    with torch.cuda.stream(stream):
        torch.cuda._sleep(int(ms * 1.5e6))


def _side_calls():
    from speculative_decoding_verification_sampling_gb300 import synth
    a = _case(3, 5, 8, 2, 128, 300, 400, [400, 31, 260], False, "causal", seed=64)
    codes = torch.full((1, 3, 40, 2, 2, 64), 56, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
    scale = torch.full((1, 3, 40, 2, 2), 127, dtype=torch.uint8, device=DEV)
    n = torch.tensor([40, 7, 0], dtype=torch.int32, device=DEV)
    cfg = synth.stochastic_gaussian(6, 4, 5000, torch.bfloat16, 1.0, seed=3)
    tgt, drf, tok = (cfg[k].to(DEV) for k in ("target", "draft", "draft_tokens"))
    par = torch.tensor([[-1, 0, 0, 1, 1, 3]], dtype=torch.int32, device=DEV)
    toks = torch.zeros_like(par)
    tree = torch.randn((1, 6, 5000), generator=torch.Generator().manual_seed(1)).to(DEV)
    return {
        "attention": lambda **kw: _call(a, **kw),
        "read": lambda **kw: (sv.spec_kv_read_quant(codes, scale, None, n, 40, **kw),),
        "verify": lambda **kw: sv.spec_verify(tgt, drf, tok, 1.0, 7, **kw),
        "draft": lambda **kw: sv.spec_draft_sample(drf, 1.0, 7, **kw),
        "tree": lambda **kw: sv.spec_verify_tree_greedy(tree, toks, par, **kw),
        "mask": lambda **kw: (sv.spec_tree_mask(par, **kw),),
        "philox": lambda **kw: (sv.spec_philox_words(7, 0, 64, 64, device=DEV, **kw),),
    }


@pytest.mark.parametrize("name", ["attention", "read", "verify", "draft", "tree", "mask", "philox"])
def test_outputs_of_a_call_on_another_stream_are_its_own(name):
    """A result whose memory the current stream has work pending on, or that is dropped before the
    other stream has written it, is nobody else's meanwhile."""
    call = _side_calls()[name]
    want = [x.clone() for x in call()]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    # blocks of the outputs' sizes, freed on the current stream with a late write pending
    _spin(torch.cuda.current_stream())
    for x in [torch.empty_like(w) for w in want for _ in range(4)]:
        x.view(torch.uint8).fill_(0xee)
    del x
    got = call(stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(g, w) for g, w in zip(got, want))
    # dropped at once: what the current stream allocates next is not written any more
    del got
    _spin(side)
    got = call(stream=side)
    del got
    mine = [torch.full_like(w.view(torch.uint8), 0x33) for w in want for _ in range(4)]
    torch.cuda.synchronize()
    assert all(bool((x == 0x33).all()) for x in mine)


@pytest.mark.parametrize("kernel", [None, "cluster", "general", "rows"])
def test_a_captured_verification_has_its_own_workspace(kernel, monkeypatch):
    """Replays between eager calls of other sizes on the same stream, one of which replaces the
    workspace that the stream's calls share."""
    from speculative_decoding_verification_sampling_gb300 import synth
    if kernel:
        monkeypatch.setenv("SPECVERIFY_KERNEL", kernel)

    def inputs(B, K, V, seed):
        cfg = synth.stochastic_gaussian(B, K, V, torch.bfloat16, 1.0, seed=seed)
        return [cfg[k].to(DEV) for k in ("target", "draft", "draft_tokens")]
    small, wide, large = inputs(6, 4, 8192, 3), inputs(3, 7, 16384, 4), inputs(24, 4, 32768, 5)
    want = [[x.clone() for x in sv.spec_verify(*a, 1.0, 7)] for a in (small, wide, large)]
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        sv.spec_verify(*small, 1.0, 7)
        side.synchronize()
        kept = sv._kept.workspaces[(0, side.cuda_stream)][0]
        before = kept.clone()
        with torch.cuda.graph(graph, stream=side):
            held = sv.spec_verify(*small, 1.0, 7)
        for i, a in enumerate((None, wide, large)):
            if a is not None:
                got = sv.spec_verify(*a, 1.0, 7)
                assert all(torch.equal(g, w) for g, w in zip(got, want[i]))
            for x in held:
                x.zero_()
            graph.replay()
            side.synchronize()
            assert all(torch.equal(g, w) for g, w in zip(held, want[0]))
            if a is None:
                assert torch.equal(kept, before)


@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("B,T,Hq,H,D,P,L,lens", [
    (5, 5, 8, 2, 128, 0, 6000, [6000, 0, 31, 4100, 2048]),              # one set of rows, results joined
    (4, 5, 8, 2, 64, 700, 300, [300, 0, 128, 7]),
    (3, 61, 16, 2, 128, 300, 900, [900, 0, 129]),                      # two sets of rows
    (64, 8, 8, 2, 128, 400, 60, [(7 * i) % 61 for i in range(64)]),    # an 8-bit prefix read back: two lines
])
def test_waits_run_out_then_recover(B, T, Hq, H, D, P, L, lens, quant, monkeypatch):
    """A spin limit of 1: the softmax's first wait for scores runs out.  The CTA winds down (its copies
    and products land, its TMEM is freed), its rows are NaN, the status is SPEC_ERR_TIMEOUT; rows that
    see no prefix and no cache are right.  The next call is right again."""
    a = _case(B, T, Hq, H, D, P, L, lens, quant, "causal", seed=71)
    want, want_lse = _call(a)
    for _ in range(3):
        monkeypatch.setenv("SPECVERIFY_SPIN_LIMIT", "1")
        st = torch.full((1,), -5, dtype=torch.int32, device=DEV)
        out, lse = _call(a, device_status=st)
        torch.cuda.synchronize()
        gone = lse.isnan()
        assert int(st.item()) == 7 and bool(gone.any())
        assert bool(out[gone].isnan().all())
        assert torch.equal(out[~gone], want[~gone]) and torch.equal(lse[~gone], want_lse[~gone])
        if P == 0:
            assert not bool(gone[[b for b in range(B) if lens[b] == 0]].any())
        monkeypatch.delenv("SPECVERIFY_SPIN_LIMIT")
        st.fill_(-5)
        out, lse = _call(a, device_status=st)
        torch.cuda.synchronize()
        assert int(st.item()) == 0 and torch.equal(out, want) and torch.equal(lse, want_lse)
