"""The quantising KV commit and reading back (CUDA, through the C ABI) against
their oracle: codes, scale bytes, lengths and read-back values all bit for bit
(a code is the nearest one, so there is nothing to tolerate)."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import speculative_decoding_verification_sampling_gb300 as sv
from oracle import kv_quant as kq

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(DEV)
    sv.load()


def _cache(NL, B, L, H, D, seed):
    """A cache full of arbitrary bytes: what is not committed must not move."""
    g = torch.Generator().manual_seed(seed)
    codes = torch.randint(0, 256, (NL, B, L, 2, H, D), generator=g, dtype=torch.int32).to(torch.uint8)
    scale = torch.randint(0, 256, (NL, B, L, 2, H), generator=g, dtype=torch.int32).to(torch.uint8)
    return codes, scale


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _check_commit(codes, scale, staged, acc, ln, nodes=None, lead=0):
    c, s = codes.to(DEV).view(torch.float8_e4m3fn), scale.to(DEV)
    n, st = _i32(ln), torch.full((1,), -5, dtype=torch.int32, device=DEV)
    ret = sv.spec_kv_commit_quant(c, s, staged.to(DEV), _i32(acc), n, nodes=_i32(nodes) if nodes is not None else None,
                                  lead=lead, device_status=st)
    oc, os_, on, ost = kq.commit(codes.numpy(), scale.numpy(), staged.double().numpy(), acc, ln, nodes, lead)
    bad = os_ == 255     # a head that reads back as NaN: its codes say nothing
    got = c.view(torch.uint8).cpu().numpy()
    np.testing.assert_array_equal(s.cpu().numpy(), os_)
    np.testing.assert_array_equal(got[~bad], oc[~bad])
    np.testing.assert_array_equal(n.cpu().numpy(), on)
    assert ret is n and int(st.item()) == (1 if ost.any() else 0)
    return c, s, n


@pytest.mark.parametrize("NL,B,L,K,H,D,dtype", [
    (3, 7, 40, 5, 8, 64, torch.bfloat16),
    (2, 33, 70, 9, 2, 128, torch.bfloat16),
    (1, 5, 9, 4, 1, 128, torch.float32),
    (1, 1, 1, 1, 1, 64, torch.float32),
    (4, 64, 300, 6, 8, 128, torch.bfloat16),
    (2, 3, 90, 61, 3, 64, torch.float32),
])
@pytest.mark.parametrize("lead", [0, 1])
def test_commit_matches_oracle(NL, B, L, K, H, D, dtype, lead):
    g = torch.Generator().manual_seed(NL * 100 + B)
    staged = (torch.randn((NL, B, K, 2, H, D), generator=g) *
              torch.exp2(torch.randint(-20, 20, (NL, B, K, 2, H, 1), generator=g).float())).to(dtype)
    ln = torch.randint(0, L + 1, (B,), generator=g).tolist()
    acc = torch.randint(-2, K + 2, (B,), generator=g).tolist()     # errors, overflows, above K
    _check_commit(*_cache(NL, B, L, H, D, 7), staged, acc, ln, None, lead)


def test_edges_of_the_format():
    """Largest magnitudes around 448 * 2^e, ties, subnormal codes and numbers,
    zeros of both signs, infinities and NaN in one head of an entry."""
    H, D = 9, 64
    x = torch.zeros((1, 1, 4, 2, H, D))
    v = torch.from_numpy(kq.e4m3_numbers()).float()
    mid = (v[1:] + v[:-1]) / 2
    for i, t in enumerate((448.0, 448.00003, 447.99997, 224.0, 1.75, 1.7500001, 2.0 ** -9, 3.0e38, 1.0e-44)):
        x[0, 0, 0, 0, i, 0] = t
        x[0, 0, 0, 1, i, 5] = -t
        x[0, 0, 0, 1, i, 6] = t / 448
    for i in range(8):   # every midpoint, with 448 beside it so that e = 0
        x[0, 0, 1, 0, i, :16] = mid[16 * i:16 * i + 16] if i < 7 else torch.cat([mid[112:], mid[:2]])
        x[0, 0, 1, 0, i, 63] = 448.0
        x[0, 0, 1, 1, i] = -x[0, 0, 1, 0, i]
    x[0, 0, 2, 0, 0, 3] = float("nan")
    x[0, 0, 2, 0, 1, 3] = float("inf")
    x[0, 0, 2, 1, 2, 3] = float("-inf")
    x[0, 0, 3] = torch.randn((2, H, D), generator=torch.Generator().manual_seed(1)) * 1e-38
    x[0, 0, 3, 0, 0, 1] = -0.0
    _check_commit(*_cache(1, 1, 6, H, D, 1), x, [4], [1])
    _check_commit(*_cache(1, 1, 6, H, D, 1), x.to(torch.bfloat16), [4], [1])


def test_tree_paths():
    NL, B, K, L, H, D = 2, 6, 7, 20, 2, 128
    g = torch.Generator().manual_seed(3)
    staged = torch.randn((NL, B, K, 2, H, D), generator=g).to(torch.bfloat16)
    nodes = [[1, 4, 6, -1, -1, -1, -1], [2, 5, -1, -1, -1, -1, -1], [-1] * 7, [1, 7, 2, 0, 0, 0, 0],
             [3, -1, 2, 0, 0, 0, 0], [6, 6, 6, 6, 6, 6, 6]]
    acc, ln = [3, 2, 0, 3, 2, 6], [0, 17, 19, 2, 3, 13]     # nodes 7 and -1 are refused
    for lead in (0, 1):
        _check_commit(*_cache(NL, B, L, H, D, 4), staged, acc, ln, nodes, lead)


@pytest.mark.parametrize("NL,B,L,count,H,D,dtype", [
    (3, 7, 40, 5, 8, 64, torch.bfloat16), (1, 4, 33, 40, 1, 128, torch.float32), (2, 5, 1, 1, 3, 64, torch.float32),
    (1, 9, 700, 700, 2, 128, torch.bfloat16)])
def test_read_matches_oracle(NL, B, L, count, H, D, dtype):
    codes, scale = _cache(NL, B, L, H, D, 11)
    scale = scale.clamp(min=20)
    # the smallest bytes, NaN, and the largest whose heads stay finite
    scale[:, :, 0, 0, 0] = torch.tensor([0, 1, 255, 246], dtype=torch.uint8).repeat(B)[:B]
    g = torch.Generator().manual_seed(2)
    ln = torch.randint(0, L + 1, (B,), generator=g)
    start = torch.randint(0, L + 2, (B,), generator=g)
    ln[0], start[0] = L, 0
    for s in (start, None):
        st = torch.full((1,), -5, dtype=torch.int32, device=DEV)
        got = sv.spec_kv_read_quant(codes.to(DEV).view(torch.float8_e4m3fn), scale.to(DEV),
                                    _i32(s.tolist()) if s is not None else None, _i32(ln.tolist()), count, dtype=dtype,
                                    device_status=st)
        want, _ = kq.read(codes.numpy(), scale.numpy(), s, ln, count)
        with np.errstate(over="ignore"):
            want = torch.from_numpy(want).to(dtype)      # overflows to infinity past the type's range
        assert got.dtype == dtype and torch.equal(got.cpu().nan_to_num(nan=3e38), want.nan_to_num(nan=3e38))
        assert int(st.item()) == 0


def test_read_reports_bad_lengths_and_reads_the_rest():
    codes, scale = _cache(1, 4, 8, 2, 64, 5)
    scale.clamp_(20, 250)
    ln, start = [8, 9, -1, 5], [0, 0, 0, -1]
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = sv.spec_kv_read_quant(codes.to(DEV).view(torch.float8_e4m3fn), scale.to(DEV), _i32(start), _i32(ln), 8,
                                dtype=torch.float32, device_status=st)
    want, bad = kq.read(codes.numpy(), scale.numpy(), start, ln, 8)
    assert bad.tolist() == [0, 1, 1, 1] and int(st.item()) == 1
    assert torch.equal(got.cpu().nan_to_num(nan=3e38), torch.from_numpy(want).float().nan_to_num(nan=3e38))


def test_verify_then_commit_on_another_stream():
    from speculative_decoding_verification_sampling_gb300 import synth
    cfg = synth.stochastic_gaussian(16, 4, 5000, torch.bfloat16, 1.0, seed=3)
    g = torch.Generator().manual_seed(9)
    staged = torch.randn((2, 16, 5, 2, 2, 64), generator=g).to(torch.bfloat16)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        _, acc = sv.spec_verify(cfg["target"].to(DEV), cfg["draft"].to(DEV), cfg["draft_tokens"].to(DEV), 1.0, 11)
        c = torch.zeros((2, 16, 64, 2, 2, 64), dtype=torch.float8_e4m3fn, device=DEV)
        s = torch.full((2, 16, 64, 2, 2), 127, dtype=torch.uint8, device=DEV)
        n0 = torch.arange(16, dtype=torch.int32, device=DEV)
        n = n0.clone()
        sv.spec_kv_commit_quant(c, s, staged.to(DEV), acc, n, lead=1)
        x = sv.spec_kv_read_quant(c, s, n0, n, 5, dtype=torch.float32)
    side.synchronize()
    a = acc.cpu()
    assert torch.equal(n.cpu(), n0.cpu() + a + 1)
    for b in range(16):
        want = torch.from_numpy(kq.values(*kq.quantise(staged[:, b].double().numpy()))).float()
        assert torch.equal(x[:, b, :a[b] + 1].cpu(), want[:, :a[b] + 1])
        assert not x[:, b, a[b] + 1:].any()


def test_launch_counts():
    c = torch.zeros((1, 2, 8, 2, 1, 64), dtype=torch.float8_e4m3fn, device=DEV)
    s = torch.zeros((1, 2, 8, 2, 1), dtype=torch.uint8, device=DEV)
    staged = torch.ones((1, 2, 3, 2, 1, 64), device=DEV)
    n0 = sv.spec_launch_count()
    n = _i32([0, 0])
    sv.spec_kv_commit_quant(c, s, staged, _i32([1, 2]), n)
    assert sv.spec_launch_count() == n0 + 2
    sv.spec_kv_read_quant(c, s, None, n, 3)
    assert sv.spec_launch_count() == n0 + 3


@pytest.mark.parametrize("NL,B,K,H,D", [(1, 1, 2100, 2, 64), (2, 3, 701, 3, 128), (1, 1, 1, 1, 64), (3, 1, 150, 8, 128)])
@pytest.mark.parametrize("nodes", [False, True])
def test_commit_of_many_entries_by_few_sequences(NL, B, K, H, D, nodes):
    """A prompt at once: more CTAs than (layer, sequence) pairs, each with a part of the pieces."""
    codes, scale = _cache(NL, B, K + 7, H, D, K)
    staged = torch.randn((NL, B, K, 2, H, D), generator=torch.Generator().manual_seed(K)).to(torch.bfloat16)
    order = [[(7 * i + b) % K for i in range(K)] for b in range(B)] if nodes else None
    _check_commit(codes, scale, staged, [max(K - 11 * b, 0) for b in range(B)], [(5 * b) % 8 for b in range(B)], order)


def test_every_code_at_every_byte():
    """Which elements reading back gives exactly: float32 up to byte 246, bfloat16 from byte 3 on as
    well.  Below that bfloat16 has no such number for some, and rounds; above, the largest are infinite."""
    codes = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(1, 1, 1, 2, 2, 64).repeat(1, 1, 255, 1, 1, 1)
    byte = torch.arange(255, dtype=torch.int32).to(torch.uint8).view(1, 1, 255, 1, 1).repeat(1, 1, 1, 2, 2)
    exact = torch.from_numpy(kq.values(codes.numpy(), byte.numpy()))
    code = torch.from_numpy(kq.decode(codes[0, 0, 0].numpy()))
    for dtype, low in ((torch.float32, 0), (torch.bfloat16, 3)):
        got = sv.spec_kv_read_quant(codes.to(DEV).view(torch.float8_e4m3fn), byte.to(DEV), None, _i32([255]), 255,
                                    dtype=dtype).cpu().double()
        assert torch.equal(got.isnan(), exact.isnan())
        inside = slice(low, 247)
        assert torch.equal(got[:, :, inside].nan_to_num(), exact[:, :, inside].nan_to_num())
        assert bool(got[0, 0, 247][code.abs() == 448].isinf().all())
        if low:
            near = (got[:, :, :low] - exact[:, :, :low]).abs().nan_to_num()
            assert bool((near <= 2.0 ** -134).all()) and bool((near > 0).any())     # half a step of 2^-133
