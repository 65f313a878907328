"""Memory that the binding keeps between calls, without a GPU: whose it is."""
from __future__ import annotations

import threading

import torch

import speculative_decoding_verification_sampling_gb300 as sv

CPU = torch.device("cpu")


def test_threads_on_one_stream_share_no_memory(monkeypatch):
    """The launches of two threads' calls may interleave on their stream."""
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)

    def hold():
        return [sv._scratch(1 << 12, CPU, 77), sv._workspace(CPU, 77, 1 << 12, (1, 2, 3, 0))]
    here, there = hold(), []
    t = threading.Thread(target=lambda: there.extend(hold()))
    t.start()
    t.join()
    assert [x.data_ptr() for x in hold()] == [x.data_ptr() for x in here]
    assert len(there) == 2 and not {x.data_ptr() for x in here} & {x.data_ptr() for x in there}


def test_attention_sizes_just_below_2_to_31():
    """Units of 128 entries are counted without overflow: what does not fit is refused, the rest is not."""
    w, top = sv.spec_attention_workspace_bytes, 2 ** 31 - 1
    for P, L in ((top, 0), (0, top), (top - 126, 0), (0, top - 127)):
        assert w(1, 1, 1, 1, 64, P, L) >= w(1, 1, 1, 1, 64, min(P, 2 ** 30), min(L, 2 ** 30)) > 0
        assert w(1, 1, 512, 512, 64, P, L) == 0       # 512 pairs of 2^24 units: past the line
        assert w(1, 1, 256, 256, 64, P, L) == 0
    assert w(300, 1, 1, 1, 64, 0, top) == 0
    assert w(1, 1, 512, 512, 64, 2 ** 26, 0) > 0
