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
