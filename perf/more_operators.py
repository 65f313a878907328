"""Sampling filters and windowed attention of a verification round: what is measured, on which cases.

Three operators around a verification round of requests that ask for temperature, top-k, top-p and min-p, on a
target whose layers attend to a sliding window and a few first tokens:

  sample   draft (or plain) tokens drawn from filtered rows of logits, by given uniforms;
  verify   the accept / reject rule where target and draft are both filtered, by given uniforms;
  window   the target's attention for the round's query tokens: each sees the first tokens of its sequence (the
           sinks) and the last ones before itself (the window).

Each has a plain form in elementary torch operations (``own`` false), the framework's entry points (``own`` true)
and a definition in 64 bits (``exact``).

A filtered row: its tokens in descending order of the logits z (the lowest index first among equals) have the
weights w = exp((z - max z) / T).  top-k keeps the first k; top-p keeps, of those, a token if the weights before it
sum up to less than p times the sum of what top-k left; min-p keeps w >= min-p.  The first token always stays.  What
all three keep is normalised.  T = 0 is the first token alone.  Drawing takes the first token, in ascending order of
the index, at which the running sum exceeds the uniform.
"""
import math
import random

import torch

own = False

DEV = "cuda:0"
SPANS = {"long": (0.25, 1.0), "full": (1.0, 1.0), "any": (0.0, 1.0)}
# what requests ask for: (T, top-k, top-p, min-p), 0 and 1.0 where a filter is off
ASKS = {
    "chat": [(0.7, 20, 0.8, 0.0), (0.8, 40, 0.95, 0.0), (1.0, 50, 0.9, 0.05), (0.6, 20, 0.95, 0.0)],
    "nucleus": [(1.0, 0, 0.9, 0.0), (0.8, 0, 0.95, 0.0), (0.6, 0, 0.95, 0.0), (1.2, 0, 0.98, 0.0)],
    "min_p": [(1.0, 0, 1.0, 0.05), (1.5, 0, 1.0, 0.1), (0.9, 0, 1.0, 0.02)],
    "mix": [(0.0, 0, 1.0, 0.0), (0.7, 20, 0.8, 0.0), (1.0, 0, 0.9, 0.0), (1.0, 0, 1.0, 0.05), (0.8, 1000, 0.95, 0.0),
            (1.0, 0, 1.0, 0.0), (1.3, 100, 1.0, 0.02), (0.3, 0, 0.99, 0.0)],
}


# ------------------------------------------------------------------ cases
def _rows(name, op, B, K, V, wide, ask):
    return {"name": name, "op": op, "B": B, "K": K, "V": V, "wide": wide, "ask": ask}


def _window(name, B, T, Hq, Hkv, D, L, W, sinks, span, quant, tree, staged=True):
    return {"name": name, "op": "window", "B": B, "T": T, "Hq": Hq, "Hkv": Hkv, "D": D, "L": L, "W": W,
            "sinks": sinks, "span": span, "quant": quant, "tree": tree, "staged": staged}


def listed():
    return [
        # the next token of one sequence: the smallest call, latency counts
        _rows("sample_one", "sample", 1, 1, 32000, True, "chat"),
        # the drafting step of the throughput batch, requests that ask for different things
        _rows("sample_batch", "sample", 256, 1, 128256, False, "mix"),
        # top-p alone over a large vocabulary: every weight counts in the total
        _rows("sample_nucleus", "sample", 128, 1, 262144, False, "nucleus"),
        # all positions of a block drafter, a vocabulary that no vector length divides, float32
        _rows("sample_odd", "sample", 7, 5, 32003, True, "mix"),
        # one sequence, K = 4 drafts
        _rows("verify_one", "verify", 1, 4, 32000, True, "chat"),
        # the throughput batch
        _rows("verify_batch", "verify", 256, 4, 128256, False, "chat"),
        # a smaller batch with long drafts, requests that ask for different things
        _rows("verify_mix", "verify", 32, 7, 152064, False, "mix"),
        # one sequence decoding one token, its entry already in the cache
        _window("window_one_token", 1, 1, 32, 8, 128, 4096, 1024, 4, "full", False, False, staged=False),
        # a serving batch of long conversations, K = 4 drafts
        _window("window_long", 64, 5, 32, 8, 128, 16384, 4096, 4, "long", False, False),
        # the throughput batch, a short window, the cache in 8 bits
        _window("window_short_q8", 256, 5, 32, 8, 128, 4096, 512, 4, "long", True, False),
        # draft trees of 61 nodes under their mask, eight query heads to a key head
        _window("window_tree", 32, 61, 64, 8, 128, 2048, 1021, 16, "any", False, True),
        # five query heads to a key head, heads of 64, many sinks, nothing a multiple of a tile
        _window("window_odd_q8", 7, 9, 20, 4, 64, 1021, 333, 130, "any", True, False),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["sample", "verify", "window"])
    while True:
        if op == "window":
            tree = rng.random() < 0.25
            Hkv, G = rng.choice([1, 2, 4, 8, 8]), rng.choice([1, 2, 3, 4, 4, 5, 8])
            T = rng.randint(2, 61) if tree else rng.choice([1, 2, 3, 5, 5, 9, 17, 32])
            c = _window("", _log(rng, 1, 256), T, G * Hkv, Hkv, rng.choice([64, 128, 128]), _log(rng, 1, 16384),
                        _log(rng, 1, 8192), rng.choice([0, 1, 4, 4, 16, _log(rng, 1, 300)]),
                        rng.choice(sorted(SPANS)), rng.random() < 0.5, tree, staged=tree or rng.random() < 0.9)
            w = work(c)
            fits = (w["bytes"] <= 1e9 and w["flops"] <= 2e11 and c["B"] * T * c["Hq"] * c["L"] <= 5e8
                    and c["B"] * c["L"] * Hkv * c["D"] <= 1.1e9)
        else:
            K = rng.choice([1, 1, 2, 5]) if op == "sample" else rng.randint(1, 9)
            c = _rows("", op, _log(rng, 1, 256), K, _log(rng, 1000, 262144), rng.random() < 0.4,
                      rng.choice(sorted(ASKS)))
            fits = work(c)["bytes"] <= (1.2e8 if op == "sample" else 5.8e8)
        if fits:
            del c["name"]
            return c


def _lengths(c):
    """The cache length of each sequence: part of the case, so that its work is known."""
    r = random.Random(c["B"] * 7919 + c["L"])
    lo, hi = SPANS[c["span"]]
    n = [int(round(c["L"] * r.uniform(lo, hi))) for _ in range(c["B"])]
    if c["span"] == "any" and c["B"] > 2:
        n[0], n[1] = 0, c["L"]
    return n


def _tree(T):
    """For each node of a tree of T nodes (branching 4, 2, 2, 1, 1, longer trees a chain), its path from the root."""
    paths, level = [[0]], [0]
    for k in (4, 2, 2, 1, 1):
        nxt = []
        for p in level:
            for _ in range(k):
                if len(paths) < T:
                    nxt.append(len(paths))
                    paths.append(paths[p] + [len(paths)])
        level = nxt or level
    while len(paths) < T:
        paths.append(paths[-1] + [len(paths)])
    return paths


def _seen(c):
    """How many entries of the pass each token sees, itself included."""
    if not c["staged"]:
        return [0] * c["T"]
    return [len(p) for p in _tree(c["T"])] if c["tree"] else list(range(1, c["T"] + 1))


# ------------------------------------------------------------------ inputs
def _logits(g, rows, V):
    """Rows shaped like a language model's: -a ln(rank) with ranks at random and a of each row in [1.1, 2.2], and
    noise.  Returns float32."""
    rank = torch.rand((rows, V), generator=g, device=DEV) * V + 1
    a = 1.1 + 1.1 * torch.rand((rows, 1), generator=g, device=DEV)
    return 12.0 - a * rank.log_() + 0.3 * torch.randn((rows, V), generator=g, device=DEV)


def _filters(c, seed):
    """T, top-k, top-p and min-p of each sequence."""
    r = random.Random(seed * 31 + c["B"])
    asks = [r.choice(ASKS[c["ask"]]) for _ in range(c["B"])]
    kinds = (torch.float32, torch.int32, torch.float32, torch.float32)
    return [torch.tensor([a[i] for a in asks], dtype=kinds[i], device=DEV) for i in range(4)]


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
    if c["op"] == "window":
        B, T, Hq, Hkv, D, L = (c[k] for k in ("B", "T", "Hq", "Hkv", "D", "L"))
        bf = torch.bfloat16
        s["q"] = torch.randn((B, T, Hq, D), generator=g, device=DEV, dtype=bf)
        s["seq_len"] = torch.tensor(_lengths(c), dtype=torch.int32, device=DEV)
        if c["quant"]:
            s["cache"], s["cache_scale"] = _codes(g, (B, L, 2, Hkv, D))
        else:
            s["cache"] = torch.randn((B, L, 2, Hkv, D), generator=g, device=DEV, dtype=bf)
        if c["staged"]:
            s["staged"] = torch.randn((B, T, 2, Hkv, D), generator=g, device=DEV, dtype=bf)
        if c["tree"]:
            m = torch.zeros((T, T), dtype=torch.uint8)
            for n, path in enumerate(_tree(T)):
                m[n, path] = 1
            s["mask"] = m.to(DEV).expand(B, T, T).contiguous()
        return s
    B, K, V = c["B"], c["K"], c["V"]
    dtype = torch.float32 if c["wide"] else torch.bfloat16
    s["temperature"], s["top_k"], s["top_p"], s["min_p"] = _filters(c, seed)
    if c["op"] == "sample":
        s["logits"] = _logits(g, B * K, V).to(dtype).view(B, K, V)
        s["uniforms"] = torch.rand((B, K), generator=g, device=DEV)
        return s
    s["target"] = torch.empty((B, K + 1, V), dtype=dtype, device=DEV)
    s["draft"] = torch.empty((B, K, V), dtype=dtype, device=DEV)
    for b in range(0, B, 32):
        n = min(32, B - b)
        z = _logits(g, n * (K + 1), V).view(n, K + 1, V)
        s["target"][b : b + n] = z
        s["draft"][b : b + n] = z[:, :K] + 0.4 * torch.randn((n, K, V), generator=g, device=DEV)
    # the drafts come from the filtered draft rows
    s["draft_tokens"] = _plain_sample(s["draft"], torch.rand((B, K), generator=g, device=DEV), s)[0]
    s["uniforms"] = torch.rand((B, K + 1, 2), generator=g, device=DEV)
    return s


# ------------------------------------------------------------------ one pass
def _filtered(z, s, b, n):
    """The filtered distributions of the rows z [n][R][V] of the sequences b .. b + n - 1, in 64 bits: the borders of
    top-p and of the draw lie anywhere between two sums."""
    V = z.shape[-1]
    T, k, p, least = (s[x][b : b + n, None, None].double() for x in ("temperature", "top_k", "top_p", "min_p"))
    z, index = torch.sort(z.double() + 0.0, dim=-1, descending=True, stable=True)
    w = torch.exp((z - z[..., :1]) / torch.where(T > 0, T, 1.0))
    rank = torch.arange(V, device=DEV)
    k = torch.where(T > 0, torch.where(k > 0, k, float(V)), 1.0)
    w = torch.where(rank < k, w, 0.0)
    total = torch.cumsum(w, -1)
    before = torch.cat([torch.zeros_like(total[..., :1]), total[..., :-1]], -1)
    keep = ((before < p * total[..., -1:]) | (p >= 1)) & (w >= least) | (rank == 0)
    w = torch.where(keep, w, 0.0)
    w /= w.sum(-1, keepdim=True)
    return torch.zeros_like(w).scatter_(-1, index, w)


def _drawn(w, v):
    """The first index at which the running sum of w [..., V] exceeds v [...] times their total."""
    c = torch.cumsum(w, -1)
    return torch.searchsorted(c, v.double()[..., None] * c[..., -1:], right=True)[..., 0]


def _plain_sample(logits, uniforms, s):
    B, K, V = logits.shape
    tokens = torch.empty((B, K), dtype=torch.int32, device=DEV)
    prob = torch.empty((B, K), dtype=torch.float32, device=DEV)
    step = max(1, 2 ** 26 // (K * V))
    for b in range(0, B, step):
        n = min(step, B - b)
        w = _filtered(logits[b : b + n], s, b, n)
        x = _drawn(w, uniforms[b : b + n])
        tokens[b : b + n] = x
        prob[b : b + n] = w.gather(-1, x[..., None])[..., 0]
    return tokens, prob


def _plain_verify(s):
    target, draft, d, u = s["target"], s["draft"], s["draft_tokens"], s["uniforms"]
    B, K1, V = target.shape
    K = K1 - 1
    tokens = torch.empty((B, K1), dtype=torch.int32, device=DEV)
    accepted = torch.empty(B, dtype=torch.int32, device=DEV)
    step = max(1, 2 ** 26 // (K1 * V))
    for b in range(0, B, step):
        n = min(step, B - b)
        q = _filtered(target[b : b + n], s, b, n)
        p = _filtered(draft[b : b + n], s, b, n)
        at = d[b : b + n, :, None].long()
        fine = u[b : b + n, :K, 0].double() * p.gather(-1, at)[..., 0] < q[:, :K].gather(-1, at)[..., 0]
        a = torch.cumprod(fine.long(), -1).sum(-1)
        row = torch.arange(n, device=DEV)
        p = torch.cat([p, torch.zeros_like(p[:, :1])], 1)       # a bonus token comes from the target's own row
        r = (q[row, a] - p[row, a]).clamp(min=0)
        r = torch.where(r.sum(-1, keepdim=True) > 0, r, q[row, a])
        x = _drawn(r, u[b : b + n][row, a, 1])
        i = torch.arange(K1, device=DEV)[None, :]
        dd = torch.cat([d[b : b + n], torch.full((n, 1), -1, dtype=torch.int32, device=DEV)], 1)
        out = torch.where(i < a[:, None], dd, -1)
        tokens[b : b + n] = torch.where(i == a[:, None], x[:, None].to(torch.int32), out)
        accepted[b : b + n] = a
    return tokens, accepted


def _pow2(e):
    """2^e in float32 from its bits (exact), e in [-126, 127]."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _plain_window(s):
    c = s["case"]
    B, T, Hq, Hkv, D, L = (c[k] for k in ("B", "T", "Hq", "Hkv", "D", "L"))
    G = Hq // Hkv
    n = s["seq_len"].long()
    if c["tree"]:
        shown = s["mask"] != 0
    else:
        shown = torch.ones((T, T), dtype=torch.bool, device=DEV).tril().expand(B, T, T)
    # a token's entries in order: the cache's, then those of the pass that it is shown
    if c["staged"]:
        count = n[:, None] + shown.sum(-1)
    else:
        count = n[:, None].expand(B, T)
    kv = s["cache"].float()
    if c["quant"]:
        kv = kv * _pow2(s["cache_scale"].int() - 127)[..., None]
    at = torch.arange(L, device=DEV)
    seen = (at < n[:, None])[:, None] & ((at < c["sinks"]) | (at >= (count - c["W"])[:, :, None]))
    if c["staged"]:
        kv = torch.cat([kv, s["staged"].float()], 1)
        at = n[:, None, None] + torch.cumsum(shown.long(), -1) - 1
        seen = torch.cat([seen, shown & ((at < c["sinks"]) | (at >= (count - c["W"])[:, :, None]))], -1)
    q = s["q"].float().view(B, T, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, T * G, D)
    hide = ~seen[:, None, :, None, :].expand(B, Hkv, T, G, seen.shape[-1]).reshape(B, Hkv, T * G, -1)
    x = (torch.matmul(q, kv[:, :, 0].permute(0, 2, 3, 1)) / math.sqrt(D)).masked_fill(hide, -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(torch.isinf(m), 0.0, m)
    w = torch.exp(x - m)
    total = w.sum(-1, keepdim=True)
    o = torch.matmul(w, kv[:, :, 1].transpose(1, 2))
    o = torch.where(total > 0, o / total, 0.0)
    lse = (m + torch.log(total))[..., 0]
    out = o.view(B, Hkv, T, G, D).permute(0, 2, 1, 3, 4).reshape(B, T, Hq, D).to(torch.bfloat16)
    return out, lse.view(B, Hkv, T, G).permute(0, 2, 1, 3).reshape(B, T, Hq)


def run(state):
    s, c = state, state["case"]
    if own:
        import speculative_decoding_verification_sampling_gb300 as sv
    if c["op"] == "window":
        if own:
            out, lse = sv.spec_verify_window_attention(
                s["q"], s["cache"], s["seq_len"], c["W"], sinks=c["sinks"], staged=s.get("staged"),
                mask=s.get("mask"), cache_scale=s.get("cache_scale"))
        else:
            out, lse = _plain_window(s)
        return {"out": out, "lse": lse}
    if own:
        filters = sv.Filters(temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"], min_p=s["min_p"])
    if c["op"] == "sample":
        if own:
            tokens, prob = sv.spec_filter_sample(s["logits"], s["uniforms"], filters)
        else:
            tokens, prob = _plain_sample(s["logits"], s["uniforms"], s)
        return {"tokens": tokens, "prob": prob}
    if own:
        tokens, accepted = sv.spec_verify_filtered(s["target"], s["draft"], s["draft_tokens"], s["uniforms"], filters)
    else:
        tokens, accepted = _plain_verify(s)
    return {"tokens": tokens, "accept_len": accepted}


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    c = case
    B = c["B"]
    if c["op"] == "window":
        T, Hq, Hkv, D, W, sinks = (c[k] for k in ("T", "Hq", "Hkv", "D", "W", "sinks"))
        count = _seen(c)
        entries = pairs = 0
        for n in _lengths(c):
            first = min(max(n + min(count) - W, 0), n)               # of the window, as the least token sees it
            entries += min(sinks, first) + n - first
            for m in count:
                pairs += min(n + m, min(sinks, max(n + m - W, 0)) + W)
        b = 2 * B * T * Hq * D * 2 + B * T * Hq * 4 + 4 * B + 2 * Hkv * (D + 1 if c["quant"] else 2 * D) * entries
        if c["staged"]:
            b += B * T * 2 * Hkv * D * 2 + (B * T * T if c["tree"] else 0)
        return {"bytes": b, "flops": 4 * Hq * D * pairs}
    K, es = c["K"], 4 if c["wide"] else 2
    if c["op"] == "sample":
        return {"bytes": B * K * (c["V"] * es + 12) + 16 * B, "flops": 0}
    return {"bytes": B * ((2 * K + 1) * c["V"] * es + 4 * K + 8 * (K + 1) + 4 * (K + 1) + 4) + 16 * B, "flops": 0}


# ------------------------------------------------------------------ the definition, in 64 bits
def _kept(z, T, k, p, least):
    """One row: the tokens that the filters keep, ascending, and their probabilities."""
    z = z.double()
    order = torch.argsort(-z, stable=True)
    if T == 0:
        return order[:1], torch.ones(1, dtype=torch.float64, device=DEV)
    if 0 < k < len(order):
        order = order[:k]
    w = torch.exp((z[order] - z[order[0]]) / T)
    n = len(order)
    if p < 1:
        # the shortest head whose sum reaches p of the whole
        n = min(n, int((torch.cumsum(w, 0) < p * w.sum()).sum()) + 1)
    if least > 0:
        n = min(n, max(1, int((w >= least).sum())))
    order, at = torch.sort(order[:n])
    w = w[:n][at]
    return order, w / w.sum()


def _pick(tokens, w, v):
    c = torch.cumsum(w, 0)
    return int(tokens[min(int((c <= v * c[-1]).sum()), len(tokens) - 1)])


def _exact_verify(s):
    target, draft = s["target"], s["draft"]
    B, K1, V = target.shape
    ask = list(zip(*(s[x].tolist() for x in ("temperature", "top_k", "top_p", "min_p"))))
    d, u = s["draft_tokens"].tolist(), s["uniforms"].tolist()
    tokens, accepted = [], []
    for b in range(B):
        for i in range(K1):
            xq, wq = _kept(target[b, i], *ask[b])
            q = torch.zeros(V, dtype=torch.float64, device=DEV).index_put_((xq,), wq)
            if i < K1 - 1:
                xp, wp = _kept(draft[b, i], *ask[b])
                p = torch.zeros(V, dtype=torch.float64, device=DEV).index_put_((xp,), wp)
                if u[b][i][0] * float(p[d[b][i]]) < float(q[d[b][i]]):
                    continue
                r = (q[xq] - p[xq]).clamp(min=0)
                wq = r if float(r.sum()) > 0 else wq
            tokens.append(d[b][:i] + [_pick(xq, wq, u[b][i][1])] + [-1] * (K1 - 1 - i))
            accepted.append(i)
            break
    kind = dict(dtype=torch.int32, device=DEV)
    return {"tokens": torch.tensor(tokens, **kind), "accept_len": torch.tensor(accepted, **kind)}


def _exact_sample(s):
    B, K, _ = s["logits"].shape
    ask = list(zip(*(s[x].tolist() for x in ("temperature", "top_k", "top_p", "min_p"))))
    u = s["uniforms"].tolist()
    tokens = torch.empty((B, K), dtype=torch.int32, device=DEV)
    prob = torch.empty((B, K), dtype=torch.float64, device=DEV)
    for b in range(B):
        for i in range(K):
            x, w = _kept(s["logits"][b, i], *ask[b])
            tokens[b, i] = t = _pick(x, w, u[b][i])
            prob[b, i] = w[x == t][0]
    return {"tokens": tokens, "prob": prob}


def _exact_window(c, s):
    B, T, Hq, Hkv, D, W, sinks = (c[k] for k in ("B", "T", "Hq", "Hkv", "D", "W", "sinks"))
    G = Hq // Hkv
    out = torch.zeros((B, T, Hq, D), dtype=torch.float64, device=DEV)
    lse = torch.full((B, T, Hq), -math.inf, dtype=torch.float64, device=DEV)
    paths = _tree(T) if c["tree"] else [list(range(t + 1)) for t in range(T)]
    for b, n in enumerate(s["seq_len"].tolist()):
        kv = s["cache"][b, :n].double()
        if c["quant"]:
            kv *= torch.exp2(s["cache_scale"][b, :n].double() - 127)[..., None]
        if c["staged"]:
            kv = torch.cat([kv, s["staged"][b].double()])
        hide = torch.ones((T, len(kv)), dtype=torch.bool)
        for t in range(T):
            line = list(range(n)) + ([n + j for j in paths[t]] if c["staged"] else [])
            hide[t, torch.tensor(line[:sinks] + line[-W:], dtype=torch.long)] = False
        if not len(kv):
            continue
        hide = hide.to(DEV)
        for h in range(Hkv):
            at = (b, slice(None), slice(h * G, (h + 1) * G))
            x = torch.einsum("tgd,jd->tgj", s["q"][at].double(), kv[:, 0, h]) / D ** 0.5
            x = x.masked_fill(hide[:, None], -math.inf)
            z = torch.logsumexp(x, -1)
            lse[at] = z
            out[at] = torch.nan_to_num(torch.einsum("tgj,jd->tgd", torch.exp(x - z[..., None]), kv[:, 1, h]))
    return {"out": out, "lse": lse}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "window":
        return _exact_window(case, s) if case["B"] * case["Hkv"] <= 4096 else None
    return _exact_sample(s) if case["op"] == "sample" else _exact_verify(s)
