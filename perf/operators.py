"""The verification pass's cache operators: what is measured, on which cases.

Three operators around a verification round:

  attention  the target's attention for the round's query tokens (K + 1 tokens of a sequence, or the nodes of a
             draft tree) over a prefix that every sequence shares, the sequence's own cache and the new entries;
  commit     the accepted entries quantised to 8 bits as they enter the cache, and that window read back;
  read       a stretch of an 8-bit cache read back in 16 or 32 bits.

Each has a plain form in elementary torch operations (``own`` false), the framework's entry points (``own`` true)
and a definition in 64 bits (``exact``).  An 8-bit cache holds e4m3 codes and one exponent byte for each (entry, key
or value, head): value = code * 2^(byte - 127).
"""
import math
import random

import torch

own = False

DEV = "cuda:0"
SPANS = {"long": (0.25, 1.0), "full": (1.0, 1.0), "any": (0.0, 1.0)}


# ------------------------------------------------------------------ cases
def _attn(name, B, T, Hq, Hkv, D, P, L, span, quant, tree, staged=True):
    return {"name": name, "op": "attention", "B": B, "T": T, "Hq": Hq, "Hkv": Hkv, "D": D, "P": P, "L": L,
            "span": span, "quant": quant, "tree": tree, "staged": staged}


def _commit(name, NL, B, T, L, Hkv, D, wide, tree):
    return {"name": name, "op": "commit", "NL": NL, "B": B, "T": T, "L": L, "Hkv": Hkv, "D": D, "wide": wide,
            "tree": tree}


def _read(name, NL, B, L, count, Hkv, D, wide, span):
    return {"name": name, "op": "read", "NL": NL, "B": B, "L": L, "count": count, "Hkv": Hkv, "D": D, "wide": wide,
            "span": span}


def listed():
    return [
        # one sequence decoding one token, its entry already in the cache: the smallest call, latency counts
        _attn("attn_one_token", 1, 1, 32, 8, 128, 0, 512, "long", False, False, staged=False),
        # a few sequences behind a system prompt, K = 4 drafts
        _attn("attn_few", 8, 5, 32, 8, 128, 1024, 512, "any", False, False),
        # a serving batch behind a long shared prompt, K = 4 drafts
        _attn("attn_shared", 64, 5, 32, 8, 128, 8192, 512, "any", False, False),
        # the throughput batch behind a longer shared prompt, cache in 8 bits
        _attn("attn_shared_q8", 256, 5, 32, 8, 128, 16384, 512, "any", True, False),
        # long conversations of different lengths with nothing shared, K = 4 drafts
        _attn("attn_long", 64, 5, 32, 8, 128, 0, 16384, "long", False, False),
        # the same with K = 8 drafts and the cache in 8 bits
        _attn("attn_long_q8", 128, 9, 32, 8, 128, 0, 8192, "long", True, False),
        # draft trees of 61 nodes (branching 4, 2, 2, 1, 1) under their mask, eight query heads to a key head
        _attn("attn_tree", 32, 61, 64, 8, 128, 2048, 1021, "any", False, True),
        # five query heads to a key head, heads of 64, nothing a multiple of a tile
        _attn("attn_odd", 7, 3, 20, 4, 64, 333, 1021, "any", False, False),
        # the accepted drafts of the throughput batch, every layer
        _commit("commit_layers", 32, 256, 5, 512, 8, 128, False, False),
        # the accepted paths of a few draft trees, float32 entries of two layers
        _commit("commit_tree", 2, 3, 61, 257, 4, 64, True, True),
        # whole 8-bit caches handed to a 16-bit consumer
        _read("read_all", 32, 16, 512, 512, 8, 128, False, "long"),
        # a short window of one layer in float32
        _read("read_window", 1, 5, 1021, 37, 8, 128, True, "any"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    kind = rng.choice(["attention", "attention", "attention", "commit", "read"])
    D = rng.choice([64, 128, 128])
    Hkv = rng.choice([1, 2, 4, 8, 8])
    while True:
        if kind == "attention":
            tree = rng.random() < 0.25
            G = rng.choice([1, 2, 3, 4, 4, 5, 8])
            T = rng.randint(2, 61) if tree else rng.choice([1, 2, 3, 5, 5, 9, 17, 32])
            c = _attn("", _log(rng, 1, 256), T, G * Hkv, Hkv, D, rng.choice([0, _log(rng, 1, 16384)]),
                      _log(rng, 1, 16384), rng.choice(sorted(SPANS)), rng.random() < 0.5, tree,
                      staged=tree or rng.random() < 0.85)
        elif kind == "commit":
            tree = rng.random() < 0.4
            T = rng.randint(2, 61) if tree else rng.randint(1, 32)
            c = _commit("", _log(rng, 1, 32), _log(rng, 1, 256), T, T + _log(rng, 1, 1024), Hkv, D,
                        rng.random() < 0.3, tree)
        else:
            L = _log(rng, 1, 4096)
            c = _read("", _log(rng, 1, 32), _log(rng, 1, 256), L, _log(rng, 1, L), Hkv, D, rng.random() < 0.3,
                      rng.choice(sorted(SPANS)))
        del c["name"]
        # within the largest listed cases: work, and the memory of the plain form
        w = work(c)
        if kind == "attention":
            rows = c["B"] * c["T"] * c["Hq"]
            fits = (w["bytes"] <= 1.6e9 and w["flops"] <= 3.6e11 and rows * (c["P"] + c["L"]) <= 1e9
                    and c["B"] * c["L"] * c["Hkv"] * c["D"] <= 1.1e9)
        elif kind == "commit":
            fits = w["bytes"] <= 5e8 and c["NL"] * c["B"] * c["L"] * c["Hkv"] * c["D"] <= 6e8
        else:
            fits = w["bytes"] <= 1.5e9 and c["NL"] * c["B"] * c["L"] * c["Hkv"] * c["D"] <= 6e8
        if fits:
            return c


def _lengths(c):
    """The cache length of each sequence: part of the case, so that its work is known."""
    r = random.Random(c["B"] * 7919 + c["L"])
    lo, hi = SPANS[c["span"]]
    n = [int(round(c["L"] * r.uniform(lo, hi))) for _ in range(c["B"])]
    if c["span"] == "any" and c["B"] > 2:
        n[0], n[1] = 0, c["L"]
    return n


def _accepted(c):
    """The accepted drafts of each sequence, -2 for a sequence that the verification reported in error."""
    r = random.Random(c["B"] * 104729 + c["T"])
    depth = _depth(c["T"]) if c["tree"] else c["T"] - 1
    a = [r.randint(0, depth) for _ in range(c["B"])]
    if c["B"] > 4:
        a[3] = -2
    return a


def _parents(n):
    """The parents of a tree of n nodes: branching 4, 2, 2, 1, 1, cut to n nodes, longer trees a chain."""
    par, level = [-1], [0]
    for k in (4, 2, 2, 1, 1):
        nxt = []
        for p in level:
            for _ in range(k):
                if len(par) < n:
                    par.append(p)
                    nxt.append(len(par) - 1)
        level = nxt or level
    while len(par) < n:
        par.append(len(par) - 1)
    return par


def _path(par, n):
    out = []
    while n > 0:
        out.append(n)
        n = par[n]
    return out[::-1]


def _depth(n):
    par = _parents(n)
    return max(len(_path(par, i)) for i in range(n))


# ------------------------------------------------------------------ inputs
def _codes(g, shape):
    """e4m3 codes and exponent bytes as a quantising commit leaves them: each head's largest value in (224, 448]."""
    z = torch.randn(shape, generator=g, device=DEV)
    z *= 447.0 / z.abs().amax(-1, keepdim=True)
    e = torch.randint(118, 121, shape[:-1], generator=g, device=DEV, dtype=torch.uint8)
    return z.to(torch.float8_e4m3fn), e


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV).manual_seed(seed)
    s = {"case": c}
    if c["op"] == "attention":
        B, T, Hq, Hkv, D, P, L = (c[k] for k in ("B", "T", "Hq", "Hkv", "D", "P", "L"))
        bf = torch.bfloat16
        s["q"] = torch.randn((B, T, Hq, D), generator=g, device=DEV, dtype=bf)
        s["seq_len"] = torch.tensor(_lengths(c), dtype=torch.int32, device=DEV)
        if c["quant"]:
            s["cache"], s["cache_scale"] = _codes(g, (B, L, 2, Hkv, D))
            if P:
                s["prefix"], s["prefix_scale"] = _codes(g, (P, 2, Hkv, D))
        else:
            s["cache"] = torch.randn((B, L, 2, Hkv, D), generator=g, device=DEV, dtype=bf)
            if P:
                s["prefix"] = torch.randn((P, 2, Hkv, D), generator=g, device=DEV, dtype=bf)
        if c["staged"]:
            s["staged"] = torch.randn((B, T, 2, Hkv, D), generator=g, device=DEV, dtype=bf)
        if c["tree"]:
            par = _parents(T)
            m = torch.zeros((T, T), dtype=torch.uint8)
            for n in range(T):
                m[n, [0] + _path(par, n)] = 1
            s["mask"] = m.to(DEV).expand(B, T, T).contiguous()
    elif c["op"] == "commit":
        NL, B, T, L, Hkv, D = (c[k] for k in ("NL", "B", "T", "L", "Hkv", "D"))
        s["staged"] = torch.randn((NL, B, T, 2, Hkv, D), generator=g, device=DEV)
        s["staged"] *= torch.exp(torch.randn((NL, B, T, 2, Hkv, 1), generator=g, device=DEV))
        s["staged"] = s["staged"].to(torch.float32 if c["wide"] else torch.bfloat16)
        s["cache"] = torch.zeros((NL, B, L, 2, Hkv, D), dtype=torch.float8_e4m3fn, device=DEV)
        s["scale"] = torch.full((NL, B, L, 2, Hkv), 127, dtype=torch.uint8, device=DEV)
        s["seq_len"] = torch.randint(0, L - T + 1, (B,), generator=g, device=DEV, dtype=torch.int32)
        s["accept_len"] = torch.tensor(_accepted(c), dtype=torch.int32, device=DEV)
        if c["tree"]:
            par = _parents(T)
            rows = []
            for a in _accepted(c):
                p = next(p for p in (_path(par, n) for n in range(T)) if len(p) >= max(a, 0))[:max(a, 0)]
                rows.append(p + [-1] * (T - len(p)))
            s["nodes"] = torch.tensor(rows, dtype=torch.int32, device=DEV)
    else:
        NL, B, L, Hkv, D = (c[k] for k in ("NL", "B", "L", "Hkv", "D"))
        s["cache"], s["scale"] = _codes(g, (NL, B, L, 2, Hkv, D))
        n = torch.tensor(_lengths(c), dtype=torch.int32)
        s["seq_len"] = n.to(DEV)
        s["start"] = (n - c["count"]).clamp(min=0).to(DEV)
    return s


# ------------------------------------------------------------------ one pass
def _pow2(e):
    """2^e in float32 from its bits (exact), e in [-126, 127]."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _values(codes, scale):
    """What 8-bit entries stand for, in float32 (exact)."""
    return codes.float() * _pow2(scale.int() - 127)[..., None]


def _entries(x, scale):
    return x.float() if scale is None else _values(x, scale)


def _plain_attention(s):
    c = s["case"]
    B, T, Hq, Hkv, D, P, L = (c[k] for k in ("B", "T", "Hq", "Hkv", "D", "P", "L"))
    G = Hq // Hkv
    sc = 1.0 / math.sqrt(D)
    # rows of a key head together: [B, Hkv, T * G, D]
    q = s["q"].float().view(B, T, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, T * G, D)
    parts, vals = [], []
    if P:
        kv = _entries(s["prefix"], s.get("prefix_scale"))
        qf = q.transpose(0, 1).reshape(Hkv, B * T * G, D)
        x = torch.matmul(qf, kv[:, 0].permute(1, 2, 0)) * sc
        parts.append(x.view(Hkv, B, T * G, P).transpose(0, 1))
        vals.append(("prefix", kv[:, 1].transpose(0, 1)))
    if L:
        kv = _entries(s["cache"], s.get("cache_scale"))
        seen = torch.arange(L, device=DEV)[None, :] < s["seq_len"][:, None]
        x = torch.matmul(q, kv[:, :, 0].permute(0, 2, 3, 1)) * sc
        parts.append(x.masked_fill(~seen[:, None, None, :], -math.inf))
        vals.append(("own", torch.where(seen[:, :, None, None], kv[:, :, 1], 0.0).transpose(1, 2)))
    if c["staged"]:
        kv = s["staged"].float()
        if c["tree"]:
            seen = s["mask"] != 0
        else:
            seen = (torch.arange(T, device=DEV)[None, :] <= torch.arange(T, device=DEV)[:, None]).expand(B, T, T)
        x = torch.matmul(q, kv[:, :, 0].permute(0, 2, 3, 1)) * sc
        hide = ~seen[:, None, :, None, :].expand(B, Hkv, T, G, T).reshape(B, Hkv, T * G, T)
        parts.append(x.masked_fill(hide, -math.inf))
        vals.append(("own", kv[:, :, 1].transpose(1, 2)))
    m = torch.stack([p.amax(-1) for p in parts]).amax(0)
    ref = torch.where(torch.isinf(m), torch.zeros_like(m), m)[..., None]
    total = torch.zeros_like(m)
    o = torch.zeros((B, Hkv, T * G, D), device=DEV)
    while parts:
        w = torch.exp(parts.pop(0) - ref)
        kind, v = vals.pop(0)
        total += w.sum(-1)
        if kind == "prefix":
            n = v.shape[1]
            y = torch.matmul(w.transpose(0, 1).reshape(Hkv, B * T * G, n), v)
            o += y.view(Hkv, B, T * G, D).transpose(0, 1)
        else:
            o += torch.matmul(w, v)
    o = torch.where(total[..., None] > 0, o / total[..., None], 0.0)
    lse = ref[..., 0] + torch.log(total)
    out = o.view(B, Hkv, T, G, D).permute(0, 2, 1, 3, 4).reshape(B, T, Hq, D).to(torch.bfloat16)
    return out, lse.view(B, Hkv, T, G).permute(0, 2, 1, 3).reshape(B, T, Hq)


def _plain_read(cache, scale, start, seq_len, count, dtype):
    NL, B, L = cache.shape[:3]
    pos = start.long()[:, None] + torch.arange(count, device=DEV)
    fine = pos < seq_len.long()[:, None]
    at = pos.clamp(max=L - 1)
    b = torch.arange(B, device=DEV)[:, None]
    x = _values(cache.view(torch.uint8)[:, b, at].view(torch.float8_e4m3fn), scale[:, b, at])
    return torch.where(fine[None, :, :, None, None, None], x, 0.0).to(dtype)


def _plain_commit(s):
    c = s["case"]
    T, L = c["T"], c["L"]
    old = s["seq_len"]
    acc = s["accept_len"].long()
    n = torch.where(acc >= 0, acc + 1, 0)                       # the last emitted token's entry, then the drafts'
    i = torch.arange(T, device=DEV)[None, :].expand(c["B"], T)
    src = i
    if c["tree"]:
        src = torch.cat([torch.zeros_like(s["nodes"][:, :1]), s["nodes"][:, : T - 1]], 1).long()
    b, k = torch.nonzero(i < n[:, None], as_tuple=True)
    x = s["staged"][:, b, src[b, k]].float()
    top = x.abs().amax(-1)
    mant, ex = torch.frexp(top)                                 # top = mant * 2^ex, mant in [0.5, 1)
    e = torch.where(mant <= 0.875, ex - 9, ex - 8)              # top <= 448 * 2^e, 448 = 0.875 * 2^9
    e = torch.where(top > 0, e, torch.zeros_like(e)).clamp(min=-126)
    code = (x * _pow2(-e)[..., None]).to(torch.float8_e4m3fn)
    at = old.long()[b] + k
    s["cache"].view(torch.uint8)[:, b, at] = code.view(torch.uint8)
    s["scale"][:, b, at] = (e + 127).to(torch.uint8)
    return (old + n).to(torch.int32)


def run(state):
    s, c = state, state["case"]
    dtype = torch.float32 if c.get("wide") else torch.bfloat16
    if own:
        import speculative_decoding_verification_sampling_gb300 as sv
    if c["op"] == "attention":
        if own:
            out, lse = sv.spec_verify_attention(
                s["q"], s["cache"], s["seq_len"], staged=s.get("staged"), mask=s.get("mask"),
                prefix=s.get("prefix"), cache_scale=s.get("cache_scale"), prefix_scale=s.get("prefix_scale"))
        else:
            out, lse = _plain_attention(s)
        return {"out": out, "lse": lse}
    if c["op"] == "commit":
        if own:
            n = s["seq_len"].clone()
            sv.spec_kv_commit_quant(s["cache"], s["scale"], s["staged"], s["accept_len"], n, nodes=s.get("nodes"),
                                    lead=1)
            x = sv.spec_kv_read_quant(s["cache"], s["scale"], s["seq_len"], n, c["T"], dtype=dtype)
        else:
            n = _plain_commit(s)
            x = _plain_read(s["cache"], s["scale"], s["seq_len"], n, c["T"], dtype)
        return {"entries": x, "seq_len": n}
    if own:
        return {"entries": sv.spec_kv_read_quant(s["cache"], s["scale"], s["start"], s["seq_len"], c["count"],
                                                 dtype=dtype)}
    return {"entries": _plain_read(s["cache"], s["scale"], s["start"], s["seq_len"], c["count"], dtype)}


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    c = case
    Hkv, D = c["Hkv"], c["D"]
    if c["op"] == "attention":
        B, T, Hq, P = c["B"], c["T"], c["Hq"], c["P"]
        n = sum(_lengths(c))
        entry = 2 * Hkv * (D + 1 if c["quant"] else 2 * D)
        b = 2 * B * T * Hq * D * 2 + B * T * Hq * 4 + 4 * B + entry * (P + n)
        pairs = B * T * P + T * n
        if c["staged"]:
            b += B * T * 2 * Hkv * D * 2
            if c["tree"]:
                par = _parents(T)
                pairs += B * sum(len(_path(par, i)) + 1 for i in range(T))
                b += B * T * T
            else:
                pairs += B * T * (T + 1) // 2
        return {"bytes": b, "flops": 4 * Hq * D * pairs}
    es = 4 if c["wide"] else 2
    if c["op"] == "commit":
        n = sum(a + 1 for a in _accepted(c) if a >= 0) * c["NL"] * 2 * Hkv
        window = c["B"] * c["T"] * c["NL"] * 2 * Hkv
        # accepted entries read and written in 8 bits, then read back into the whole window
        return {"bytes": n * (D * es + D + 1) + n * (D + 1) + window * D * es + 12 * c["B"], "flops": 0}
    n = sum(min(m, c["count"]) for m in _lengths(c)) * c["NL"] * 2 * Hkv
    window = c["B"] * c["count"] * c["NL"] * 2 * Hkv
    return {"bytes": n * (D + 1) + window * D * es + 8 * c["B"], "flops": 0}


# ------------------------------------------------------------------ the definition, in 64 bits
def _e4m3_values():
    """The value of each of the 256 codes, from the format: 1 sign, 4 exponent (bias 7), 3 mantissa bits."""
    v = []
    for code in range(256):
        e, f = (code >> 3) & 15, code & 7
        x = math.ldexp(f, -9) if e == 0 else math.ldexp(8 + f, e - 10)
        if e == 15 and f == 7:
            x = math.nan
        v.append(-x if code & 128 else x)
    return torch.tensor(v, dtype=torch.float64, device=DEV)


def _two_to(e):
    """2^e in 64 bits from its bits, e in [-1022, 1023]."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _stands_for(codes, scale):
    return _e4m3_values()[codes.view(torch.uint8).long()] * _two_to(scale.long() - 127)[..., None]


def _exact_attention(c, s):
    B, T, Hq, Hkv, D, P = (c[k] for k in ("B", "T", "Hq", "Hkv", "D", "P"))
    G = Hq // Hkv
    out = torch.zeros((B, T, Hq, D), dtype=torch.float64, device=DEV)
    lse = torch.zeros((B, T, Hq), dtype=torch.float64, device=DEV)
    n = s["seq_len"].tolist()
    for h in range(Hkv):
        heads = slice(h * G, (h + 1) * G)
        if P:
            if c["quant"]:
                pk = _stands_for(s["prefix"][:, 0, h], s["prefix_scale"][:, 0, h])
                pv = _stands_for(s["prefix"][:, 1, h], s["prefix_scale"][:, 1, h])
            else:
                pk, pv = s["prefix"][:, 0, h].double(), s["prefix"][:, 1, h].double()
        for b in range(B):
            k = [pk] if P else []
            v = [pv] if P else []
            if c["quant"]:
                k.append(_stands_for(s["cache"][b, : n[b], 0, h], s["cache_scale"][b, : n[b], 0, h]))
                v.append(_stands_for(s["cache"][b, : n[b], 1, h], s["cache_scale"][b, : n[b], 1, h]))
            else:
                k.append(s["cache"][b, : n[b], 0, h].double())
                v.append(s["cache"][b, : n[b], 1, h].double())
            old = sum(len(x) for x in k)
            if c["staged"]:
                k.append(s["staged"][b, :, 0, h].double())
                v.append(s["staged"][b, :, 1, h].double())
            k, v = torch.cat(k), torch.cat(v)
            if not len(k):
                lse[b, :, heads] = -math.inf
                continue
            x = torch.einsum("tgd,jd->tgj", s["q"][b, :, heads].double(), k) / D ** 0.5
            if c["staged"]:
                for t in range(T):
                    if c["tree"]:
                        x[t, :, old:][:, s["mask"][b, t] == 0] = -math.inf
                    else:
                        x[t, :, old + t + 1:] = -math.inf
            z = torch.logsumexp(x, -1)
            lse[b, :, heads] = z
            out[b, :, heads] = torch.einsum("tgj,jd->tgd", torch.exp(x - z[..., None]), v)
    return {"out": out, "lse": lse}


def _exact_commit(c, s):
    NL, B, T = c["NL"], c["B"], c["T"]
    acc = s["accept_len"].tolist()
    x = torch.zeros((NL, B, T, 2, c["Hkv"], c["D"]), dtype=torch.float64, device=DEV)
    n = s["seq_len"].clone()
    for b, a in enumerate(acc):
        if a < 0:
            continue
        src = [0] + (s["nodes"][b, :a].tolist() if c["tree"] else list(range(1, a + 1)))
        x[:, b, : a + 1] = s["staged"][:, b, src].double()
        n[b] += a + 1
    # the exponent: the least e with the largest value at most 448 * 2^e
    top = x.abs().amax(-1, keepdim=True)
    e = torch.ceil(torch.log2(top / 448.0))
    e = torch.where(top > 0, e, 0.0)
    e = torch.where(top > 448.0 * _two_to(e), e + 1, e)
    e = torch.where((top > 0) & (top <= 448.0 * _two_to(e - 1)), e - 1, e).clamp(min=-126)
    y = x * _two_to(-e)
    # the nearest code: steps of 2^(k - 3) in the binade [2^k, 2^(k + 1)), of 2^-9 below 2^-6; ties to even
    _, k = torch.frexp(y)
    step = _two_to((k - 1).clamp(min=-6) - 3)
    return {"entries": torch.round(y / step) * step * _two_to(e), "seq_len": n}


def exact(case, seed):
    c = case
    if c["op"] == "attention" and c["B"] * c["Hkv"] * (c["T"] if c["staged"] else 1) > 40000:
        return None     # too long, one head of one sequence at a time
    s = prepare(c, seed)
    if c["op"] == "attention":
        return _exact_attention(c, s)
    if c["op"] == "commit":
        return _exact_commit(c, s)
    NL, B, count = c["NL"], c["B"], c["count"]
    x = torch.zeros((NL, B, count, 2, c["Hkv"], c["D"]), dtype=torch.float64, device=DEV)
    for b, (a, n) in enumerate(zip(s["start"].tolist(), s["seq_len"].tolist())):
        m = max(0, min(count, n - a))
        x[:, b, :m] = _stands_for(s["cache"][:, b, a : a + m], s["scale"][:, b, a : a + m])
    return {"entries": x}
