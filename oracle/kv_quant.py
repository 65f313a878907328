"""Oracle of the 8-bit KV cache: the quantising commit and reading back.

TEST INFRASTRUCTURE ONLY (same rule as the rest of ``oracle/``).

The format, from its definition: a head's D elements share 2^e with e the least
integer >= -126 such that the largest magnitude is at most 448 * 2^e; a code is
the e4m3 number (1 sign, 4 exponent bits with bias 7, 3 mantissa bits, no
infinity, largest 448) nearest to x * 2^-e, ties to the even mantissa.  The
codes come from a table of the format's 127 non-negative numbers, not from a
conversion instruction or a float8 type.  A head with a NaN or an infinity has
byte 255 and reads back as NaN.

What is committed is the rule of ``oracle/kv_commit.py`` with two additions:
``lead`` staged entries go ahead of the accepted ones, and ``nodes`` names the
staged entries of an accepted tree path.
"""
from __future__ import annotations

import numpy as np

ERR_CAPACITY = 1


def e4m3_numbers():
    """The format's non-negative numbers, code 0 .. 126."""
    v = []
    for code in range(127):
        e, m = code >> 3, code & 7
        v.append(m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10))
    return np.array(v)


_TABLE = e4m3_numbers()


def encode(y):
    """Codes of float64 numbers with |y| <= 448: the nearest, ties to an even code."""
    a = np.abs(y)
    hi = np.searchsorted(_TABLE, a)                  # first number >= a
    lo = np.maximum(hi - 1, 0)
    up = _TABLE[hi] - a
    down = a - _TABLE[lo]
    pick = np.where(up < down, hi, np.where(down < up, lo, np.where(lo % 2 == 0, lo, hi)))
    return (pick | np.where(np.signbit(y), 128, 0)).astype(np.uint8)


def decode(codes):
    codes = np.asarray(codes)
    full = np.concatenate([_TABLE, [np.nan]])
    v = full[codes & 127]
    return np.where(codes & 128, -v, v)


def quantise(x):
    """(codes, byte) of heads x [..., D] in float64."""
    x = np.asarray(x, dtype=np.float64)
    top = np.abs(x).max(-1)
    bad = ~np.isfinite(x).all(-1)
    t = np.where(bad | (top == 0), 1.0, top)
    e = np.floor(np.log2(t)).astype(np.int64) - 9    # below the answer, then upwards
    for _ in range(3):
        e = np.where(t > np.ldexp(448.0, e), e + 1, e)
    e = np.where(top == 0, 0, np.maximum(e, -126))
    codes = encode(np.ldexp(np.where(bad[..., None], 0.0, x), -e[..., None]))
    return codes, np.where(bad, 255, e + 127).astype(np.uint8)


def values(codes, byte):
    """What codes [..., D] with bytes [...] stand for."""
    byte = np.asarray(byte).astype(np.int64)
    v = np.ldexp(decode(codes), byte[..., None] - 127)
    return np.where(byte[..., None] == 255, np.nan, v)


def commit(cache, scale, staged, accept_len, seq_len, nodes=None, lead=0):
    """Returns (codes, bytes, seq_len, status [B]); staged [NL][B][K][2][H][D] in float64."""
    cache, scale = np.array(cache, copy=True), np.array(scale, copy=True)
    seq_len = np.array(seq_len, dtype=np.int64, copy=True)
    K, L = staged.shape[2], cache.shape[2]
    status = np.zeros(len(seq_len), dtype=np.int32)
    for b, a in enumerate(np.asarray(accept_len).tolist()):
        if a < 0:
            continue
        n, at = lead + a, int(seq_len[b])
        if n > K or at < 0 or at + n > L:
            status[b] = ERR_CAPACITY
            continue
        src = list(range(n)) if nodes is None else list(range(lead)) + [int(x) for x in nodes[b][:a]]
        if any(s < 0 or s >= K for s in src):
            status[b] = ERR_CAPACITY
            continue
        if n:
            cache[:, b, at:at + n], scale[:, b, at:at + n] = quantise(staged[:, b, src])
        seq_len[b] = at + n
    return cache, scale, seq_len.astype(np.int32), status


def read(cache, scale, start, seq_len, count):
    """(entries [NL][B][count][2][H][D] in float64, status [B])."""
    NL, B, L = cache.shape[:3]
    out = np.zeros((NL, B, count) + cache.shape[3:])
    status = np.zeros(B, dtype=np.int32)
    for b in range(B):
        s, n = int(start[b]) if start is not None else 0, int(seq_len[b])
        if n < 0 or n > L or s < 0:
            status[b] = ERR_CAPACITY
            continue
        m = max(0, min(count, n - s))
        out[:, b, :m] = values(cache[:, b, s:s + m], scale[:, b, s:s + m])
    return out, status
