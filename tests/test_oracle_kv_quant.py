"""Pins for the 8-bit cache oracle: the format against torch's float8 type, the
scale against its definition, and the commit against hand-made cases."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import kv_quant as kq


def test_numbers_of_the_format():
    v = kq.e4m3_numbers()
    assert v[0] == 0 and v[1] == 2.0 ** -9 and v[8] == 2.0 ** -6 and v[126] == 448
    codes = torch.arange(256, dtype=torch.uint8)
    want = codes.view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(kq.decode(codes.numpy()), want)


def test_encode_matches_torch_at_and_around_every_midpoint():
    v = kq.e4m3_numbers()
    mid = (v[1:] + v[:-1]) / 2
    y = np.concatenate([v, mid, np.nextafter(mid.astype(np.float32), np.float32(0)).astype(np.float64),
                        np.nextafter(mid.astype(np.float32), np.float32(1e9)).astype(np.float64)])
    y = np.concatenate([y, -y])
    want = torch.tensor(y, dtype=torch.float32).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    np.testing.assert_array_equal(kq.encode(y), want)


@pytest.mark.parametrize("top,e", [(448.0, 0), (np.nextafter(448.0, 500), 1), (1.0, -8), (1.75, -8), (1.76, -7),
                                   (0.0, 0), (2.0 ** -133, -126), (2.0 ** 127 * 1.99, 120), (2.0 ** -119, -126)])
def test_scale_is_the_least_that_fits(top, e):
    codes, byte = kq.quantise(np.array([[0.0, -top, top / 3]]))
    assert byte[0] == e + 127
    if top > 2.0 ** -110:
        assert abs(kq.values(codes, byte)[0, 1] + top) <= 2.0 ** -4 * top


def test_non_finite_heads_read_back_as_nan():
    codes, byte = kq.quantise(np.array([[1.0, np.nan], [np.inf, 0.0], [1.0, 2.0]]))
    assert byte.tolist() == [255, 255, 120]      # 2 <= 448 * 2^-7 = 3.5, 2 > 448 * 2^-8
    v = kq.values(codes, byte)
    assert np.isnan(v[:2]).all() and v[2].tolist() == [1.0, 2.0]


def test_commit_lead_nodes_and_errors():
    rng = np.random.default_rng(5)
    NL, B, K, L, H, D = 2, 6, 4, 9, 1, 4
    staged = rng.standard_normal((NL, B, K, 2, H, D))
    cache = np.zeros((NL, B, L, 2, H, D), dtype=np.uint8)
    scale = np.full((NL, B, L, 2, H), 127, dtype=np.uint8)
    nodes = np.array([[1, 3, -1, -1], [2, -1, -1, -1], [4, 0, 0, 0], [1, 2, 3, 0], [0, 0, 0, 0], [3, 3, 3, 3]])
    acc, ln = [2, 1, 1, 3, -2, 3], [0, 8, 0, 5, 3, 6]
    c, s, n, st = kq.commit(cache, scale, staged, acc, ln, nodes, lead=1)
    assert st.tolist() == [0, 1, 1, 0, 0, 1]      # past the capacity, a bad node, past the capacity
    assert n.tolist() == [3, 8, 0, 9, 3, 6]
    for b, src in ((0, [0, 1, 3]), (3, [0, 1, 2, 3])):
        want, byte = kq.quantise(staged[:, b, src])
        np.testing.assert_array_equal(c[:, b, ln[b]:n[b]], want)
        np.testing.assert_array_equal(s[:, b, ln[b]:n[b]], byte)
    for b in (1, 2, 4, 5):
        assert not c[:, b].any() and (s[:, b] == 127).all()
    got, st = kq.read(c, s, np.array([1, 0, 0, 5, 0, 0]), n, 3)
    np.testing.assert_array_equal(got[:, 0, :2], kq.values(c[:, 0, 1:3], s[:, 0, 1:3]))
    assert not got[:, 0, 2:].any() and not st.any()
    assert kq.read(c, s, None, np.array([10, 0, 0, 0, 0, -1]), 2)[1].tolist() == [1, 0, 0, 0, 0, 1]
