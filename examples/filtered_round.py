"""Speculative decoding of requests with filters of their own, on a toy target
with a sliding window and sinks, on the GPU.

Every round, for every sequence of a batch:

  1. drafts, one token at a time, drawn under the sequence's temperature, top-k,
     top-p and min-p (spec_filter_sample) from the target's logits, disturbed;
  2. the target's pass over the last emitted token and the K drafts: attention to
     the first tokens of the sequence and the last ones before each token
     (spec_verify_window_attention) over an 8-bit cache, and logits;
  3. accept / reject between the filtered distributions (spec_verify_filtered);
  4. the accepted entries enter the cache (spec_kv_commit_quant).

    python examples/filtered_round.py
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import speculative_decoding_verification_sampling_gb300 as sv   # noqa: E402


def main(B=12, K=4, rounds=8, V=4096, Hq=8, Hkv=2, D=64, window=11, sinks=4, seed=7, watch=None):
    """watch(what, inputs, outputs): told of every call of step 1 to 3."""
    dev = torch.device("cuda:0")
    bf = torch.bfloat16
    g = torch.Generator(device=dev).manual_seed(seed)
    T, L = K + 1, rounds * (K + 1)

    def weights(*s):
        return (torch.randn(s, generator=g, device=dev) / s[0] ** 0.5).to(bf)
    embed = torch.randn((V, Hq * D), generator=g, device=dev).to(bf)
    wq, wkv, head = weights(Hq * D, Hq * D), weights(Hq * D, 2 * Hkv * D), weights(Hq * D, V)
    # what the requests ask for, in turn: greedy, top-k and top-p, top-p alone, min-p
    asks = [((0.0, 0, 1.0, 0.0), (0.8, 40, 0.95, 0.0), (1.0, 0, 0.9, 0.0), (1.2, 0, 1.0, 0.1))[b % 4] for b in range(B)]
    kinds = (torch.float32, torch.int32, torch.float32, torch.float32)
    filters = sv.Filters(*[torch.tensor([a[i] for a in asks], dtype=kinds[i], device=dev) for i in range(4)])
    cache = torch.zeros((1, B, L, 2, Hkv, D), dtype=torch.float8_e4m3fn, device=dev)
    scale = torch.full((1, B, L, 2, Hkv), 127, dtype=torch.uint8, device=dev)
    length = torch.zeros(B, dtype=torch.int32, device=dev)

    def told(what, inputs, outputs):
        if watch is not None:
            watch(what, inputs, outputs)
        return outputs

    def target(tokens):
        """Logits [B][T][V] of the pass over tokens [B][T], and their entries."""
        x = embed[tokens.long()]
        new = (x @ wkv).view(*tokens.shape, 2, Hkv, D)
        q = (x @ wq).view(B, tokens.shape[1], Hq, D)
        out, _ = told("window", (q, cache[0], scale[0], length, new, window, sinks), sv.spec_verify_window_attention(
            q, cache[0], length, window, sinks=sinks, staged=new, cache_scale=scale[0]))
        return ((out.view(B, tokens.shape[1], Hq * D) + x) @ head).float(), new

    last = torch.randint(0, V, (B, 1), generator=g, device=dev, dtype=torch.int32)
    made = 0
    for _ in range(rounds):
        drafted, logits = last, []
        for _ in range(K):
            z = target(drafted)[0][:, -1:]
            z = (z + 0.3 * torch.randn(z.shape, generator=g, device=dev)).contiguous()
            u = torch.rand((B, 1), generator=g, device=dev)
            logits.append(z)
            drafted = torch.cat([drafted, told("sample", (z, u, asks), sv.spec_filter_sample(z, u, filters))[0]], 1)
        z, new = target(drafted)
        draft, u = torch.cat(logits, 1), torch.rand((B, T, 2), generator=g, device=dev)
        d = drafted[:, 1:].contiguous()
        tokens, accepted = told("verify", (z, draft, d, u, asks), sv.spec_verify_filtered(z, draft, d, u, filters))
        sv.spec_kv_commit_quant(cache, scale, new[None].contiguous(), accepted, length, lead=1)
        last = tokens.gather(1, accepted[:, None].long())
        made += int((accepted + 1).sum())
    assert int(length.sum()) == made, "cache lengths"
    print(f"{B} sequences, {rounds} rounds of K = {K}: {made / (B * rounds):.2f} tokens per round and sequence")
    return made / (B * rounds)


if __name__ == "__main__":
    main()
