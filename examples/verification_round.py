"""Speculative decoding rounds with a toy one-layer target on the GPU.

Every round, for every sequence of a batch behind one shared prompt:

  1. the drafter's tokens (here: the target's own distribution, disturbed);
  2. the target's pass over the last emitted token and the K drafts: attention
     over the shared prompt, the sequence's own 8-bit cache and the new entries
     (spec_verify_attention), and logits;
  3. accept / reject (spec_verify);
  4. the accepted entries enter the 8-bit cache (spec_kv_commit_quant).

At the end the cache is read back (spec_kv_read_quant) and held against the
entries of the emitted tokens computed anew.

    python examples/verification_round.py
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import speculative_decoding_verification_sampling_gb300 as sv   # noqa: E402


def main(B=16, K=4, rounds=8, prompt=300, V=4096, Hq=8, Hkv=2, D=64, seed=7):
    dev = torch.device("cuda:0")
    bf = torch.bfloat16
    g = torch.Generator(device=dev).manual_seed(seed)
    T, L = K + 1, rounds * (K + 1)

    def weights(*s):
        return (torch.randn(s, generator=g, device=dev) / s[0] ** 0.5).to(bf)
    embed = torch.randn((V, Hq * D), generator=g, device=dev).to(bf)
    wq, wkv, head = weights(Hq * D, Hq * D), weights(Hq * D, 2 * Hkv * D), weights(Hq * D, V)

    def entries(tokens):
        """Keys and values of tokens [...]: [...][2][Hkv][D]."""
        return (embed[tokens.long()] @ wkv).view(*tokens.shape, 2, Hkv, D)

    prefix = entries(torch.randint(0, V, (prompt,), generator=g, device=dev))
    # the shared prompt in 8 bits, by the same commit: one sequence whose entries are all accepted
    p8 = torch.empty((1, 1, prompt, 2, Hkv, D), dtype=torch.float8_e4m3fn, device=dev)
    ps = torch.empty((1, 1, prompt, 2, Hkv), dtype=torch.uint8, device=dev)
    sv.spec_kv_commit_quant(p8, ps, prefix[None, None].contiguous(),
                            torch.tensor([prompt], dtype=torch.int32, device=dev),
                            torch.zeros(1, dtype=torch.int32, device=dev))
    cache = torch.zeros((1, B, L, 2, Hkv, D), dtype=torch.float8_e4m3fn, device=dev)
    scale = torch.full((1, B, L, 2, Hkv), 127, dtype=torch.uint8, device=dev)
    length = torch.zeros(B, dtype=torch.int32, device=dev)

    def target(tokens):
        """Logits [B][T][V] of the pass over tokens [B][T], and their entries."""
        x = embed[tokens.long()]
        new = entries(tokens)
        out, _ = sv.spec_verify_attention((x @ wq).view(B, tokens.shape[1], Hq, D), cache[0], length, staged=new,
                                          prefix=p8[0, 0], cache_scale=scale[0], prefix_scale=ps[0, 0])
        return ((out.view(B, tokens.shape[1], Hq * D) + x) @ head).float(), new

    last = torch.randint(0, V, (B, 1), generator=g, device=dev, dtype=torch.int32)
    emitted = [[int(t)] for t in last[:, 0].tolist()]
    for r in range(rounds):
        # drafts, one token at a time: the target's logits with noise
        drafted, logits = last, []
        for _ in range(K):
            z = target(drafted)[0][:, -1]
            z = z + 0.5 * torch.randn(z.shape, generator=g, device=dev)
            logits.append(z)
            drafted = torch.cat([drafted, sv.spec_draft_sample(z[:, None].contiguous(), 1.0, seed + r)[0]], 1)
        z, new = target(drafted)
        tokens, accepted = sv.spec_verify(z, torch.stack(logits, 1), drafted[:, 1:].contiguous(), 1.0, seed + r)
        sv.spec_kv_commit_quant(cache, scale, new[None].contiguous(), accepted, length, lead=1)
        last = tokens.gather(1, accepted[:, None].long())
        for b, (t, a) in enumerate(zip(tokens.tolist(), accepted.tolist())):
            emitted[b] += t[:a + 1]

    # every emitted token but the last has its entry in the cache, off by at most half a step of e4m3
    back = sv.spec_kv_read_quant(cache, scale, None, length, L, dtype=torch.float32)[0]
    for b, n in enumerate(length.tolist()):
        assert n == len(emitted[b]) - 1, "cache length"
        want = entries(torch.tensor(emitted[b][:-1], device=dev)).float()
        step = want.abs().amax(-1, keepdim=True) * 2.0 ** -9    # of the smallest codes, at most
        assert bool(((back[b, :n] - want).abs() <= 2.0 ** -4 * want.abs() + step).all()), "cache entries"
        assert not back[b, n:].any()
    made = sum(map(len, emitted)) - B
    print(f"{B} sequences, {rounds} rounds of K = {K}: {made / (B * rounds):.2f} tokens per round and sequence")
    return made / (B * rounds)


if __name__ == "__main__":
    main()
