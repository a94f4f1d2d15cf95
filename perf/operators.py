"""Attention over KV caches that stay in device memory: cases, plain forms and exact values.

Four operators over a paged pool of cache blocks, K and V [slots][kv heads][block][head dim]:

  window   causal attention of ragged query rows with a sliding window and first tokens that stay visible
  prefix   attention of a batch whose requests share a long prefix, then each its own tokens
  weights  causal attention that also accumulates, per key, the softmax weight its kv head's queries gave it
  evict    the tokens a cache keeps (first, recent, most accumulated weight), gathered into new blocks

`own` False: elementary torch operations in 32 bits.  `own` True: the framework's calls.
"""
import math
import random

import torch

own = False

_BF16, _FP8 = "bf16", "fp8"


# ------------------------------------------------------------------------------------------ cases
def _attn(name, op, batch, ctx, q_len, heads, kv_heads, dim, block, kv, window=0, sink=0):
    return {"name": name, "op": op, "batch": batch, "ctx": ctx, "q_len": q_len, "heads": heads, "kv_heads": kv_heads,
            "dim": dim, "block": block, "kv": kv, "window": window, "sink": sink}


def listed():
    return [
        # one user's next token in a layer with a local window: the call's latency is what counts
        _attn("window one token", "window", 1, 4096, 1, 32, 8, 128, 16, _BF16, 1024, 4),
        # a serving batch's next tokens, contexts of every length up to 64K, 8-bit cache
        _attn("window batch fp8", "window", 32, 65536, 1, 32, 8, 128, 64, _FP8, 4096, 4),
        # a prompt of 16K tokens prefilled in one call
        _attn("window prompt", "window", 1, 16384, 16384, 32, 8, 128, 64, _BF16, 4096, 4),
        # chunks of prompts and single tokens in one batch, small heads in groups of three, odd lengths
        _attn("window mixed", "window", 9, 5001, 700, 24, 8, 64, 32, _BF16, 1000, 1),
        # a few users behind one short system prompt
        _attn("prefix few", "prefix", 4, 200, 1, 32, 8, 128, 16, _BF16) | {"prefix": 1000, "prefixes": 1},
        # a batch behind one 32K document
        _attn("prefix batch", "prefix", 32, 2048, 1, 32, 8, 128, 64, _BF16) | {"prefix": 32768, "prefixes": 1},
        # two documents, a token and its four drafts verified per request
        _attn("prefix drafts", "prefix", 64, 1024, 5, 32, 8, 128, 64, _BF16) | {"prefix": 65536, "prefixes": 2},
        # the same kind of batch with an 8-bit cache and odd lengths
        _attn("prefix batch fp8", "prefix", 24, 777, 1, 32, 8, 128, 16, _FP8) | {"prefix": 20001, "prefixes": 3},
        # a batch's next tokens, weights accumulated for a later eviction
        _attn("weights batch", "weights", 16, 8192, 1, 32, 8, 128, 64, _BF16),
        # a prompt whose tokens are all weighed before the cache is cut down
        _attn("weights prompt", "weights", 1, 8192, 8192, 32, 8, 128, 64, _BF16),
        # caches cut back to 2048 tokens each time one block more has filled
        {"name": "evict step", "op": "evict", "batch": 8, "ctx": 2112, "keep": 2048, "heads": 32, "kv_heads": 8, "dim": 128,
         "block": 64, "kv": _BF16, "sink": 4, "recent": 256},
        # 32K prompts cut down to 2048 tokens
        {"name": "evict prompt", "op": "evict", "batch": 8, "ctx": 32768, "keep": 2048, "heads": 32, "kv_heads": 8, "dim": 128,
         "block": 16, "kv": _BF16, "sink": 4, "recent": 256},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    most = {op: max((w["bytes"] / 5e12 + w["flops"] / 5e14) for c in listed() if c["op"] == op for w in [work(c)])
            for op in ("window", "prefix", "weights", "evict")}
    while True:
        op = rng.choice(("window", "window", "prefix", "prefix", "weights", "evict"))
        heads, kv_heads = rng.choice(((32, 8), (8, 2), (24, 8), (16, 16), (32, 4), (28, 4)))
        dim, block, kv = rng.choice((64, 128)), rng.choice((16, 32, 64, 128)), rng.choice((_BF16, _BF16, _FP8))
        if op == "evict":
            ctx = _log(rng, 64, 65536)
            c = {"op": op, "batch": _log(rng, 1, 32), "ctx": ctx, "keep": max(20, min(4096, int(ctx * rng.uniform(0.02, 0.99)))),
                 "heads": heads, "kv_heads": kv_heads, "dim": dim, "block": block, "kv": kv, "sink": rng.randint(0, 8),
                 "recent": rng.randint(0, 12)}
        elif op == "prefix":
            b = _log(rng, 1, 64)
            c = _attn("", op, b, _log(rng, 8, 4096), rng.randint(1, 6), heads, kv_heads, dim, block, kv)
            c |= {"prefix": _log(rng, 100, 65536), "prefixes": rng.choice([p for p in (1, 2, 3, 4) if b % p == 0])}
        else:
            ctx = _log(rng, 4, 65536 if op == "window" else 16384)
            one = rng.random() < 0.5
            q = 1 if one else min(ctx, _log(rng, 2, 8192))
            c = _attn("", op, _log(rng, 1, 64 if one else 8), ctx, q, heads, kv_heads, dim, block, kv)
            if op == "window":
                c |= {"window": _log(rng, 16, 8192), "sink": rng.randint(0, 64)}
        c.pop("name", None)
        w = work(c)
        n = sum(_lens(c)[1]) if op in ("window", "weights") else 1
        wide = n * c["heads"] * (min(c["ctx"], c["window"] + 512) if c.get("window") else c["ctx"]) if op in ("window", "weights") else 0
        if w["bytes"] / 5e12 + w["flops"] / 5e14 <= most[op] and wide <= 4.5e9:
            return c


def _lens(c):
    """Each request's context (with the call's own tokens) and number of query tokens; part of the case, not of the seed."""
    r = random.Random(repr(sorted((k, v) for k, v in c.items() if k != "name")))
    ctx, q = [], []
    for i in range(c["batch"]):
        n = c["ctx"] if i == 0 else 1 + int((c["ctx"] - 1) * (1 - 0.75 * r.random()))
        if c["op"] == "prefix":
            n, m = max(n, c["q_len"]), c["q_len"]
        elif c["op"] == "evict":
            n, m = n if i == 0 else int(0.95 * c["keep"] + (c["ctx"] - 0.95 * c["keep"]) * r.random()), 0
        elif i == 0:
            m = c["q_len"]
        else:
            m = 1 if c["q_len"] == 1 or r.random() < 0.4 else 1 + int(c["q_len"] * r.random())
            if i == 3:
                n = 1           # a request's first token
            if i == 7:
                n, m = 0, 1     # a free place of the batch
            m = max(1, min(m, n))
        ctx.append(n)
        q.append(m)
    return ctx, q


def _prefixes(c):
    """Lengths of the shared prefixes, the first of them the longest."""
    return [c["prefix"] - 17 * i * (c["prefix"] // 200) for i in range(c["prefixes"])]


# ------------------------------------------------------------------------------------------ floors
def _seen(ctx, q, window, sink):
    """(pairs of query token and visible key, keys visible to some query) of one request."""
    window = window or ctx
    pairs = sum(min(p + 1, window) + min(sink, max(0, p + 1 - window)) for p in range(ctx - q, ctx))
    low = max(0, ctx - q + 1 - window)
    return pairs, ctx - low + min(sink, low)


def work(c):
    e = 2 if c["kv"] == _BF16 else 1
    row = c["kv_heads"] * c["dim"] * 2 * e                       # K and V of one token
    ctx, q = _lens(c)
    if c["op"] == "evict":
        keep = [min(n, c["keep"]) for n in ctx]
        return {"bytes": sum(4 * n * c["kv_heads"] for n in ctx) + sum(k * (2 * row + 8 * c["kv_heads"]) for k in keep), "flops": 0}
    io = sum(q) * c["heads"] * c["dim"] * 4                      # queries in, outputs out, 2 bytes each
    per = 4 * c["heads"] * c["dim"]
    if c["op"] == "prefix":
        pre, each = _prefixes(c), c["batch"] // c["prefixes"]
        return {"bytes": io + (sum(ctx) + sum(pre)) * row,
                "flops": per * sum(m * (pre[i // each] + n - m) + m * (m + 1) // 2 for i, (n, m) in enumerate(zip(ctx, q)))}
    both = [_seen(n, m, c["window"], c["sink"]) for n, m in zip(ctx, q) if n]
    w = sum(8 * n * c["kv_heads"] for n in ctx) if c["op"] == "weights" else 0
    return {"bytes": io + sum(k for _, k in both) * row + w, "flops": per * sum(p for p, _ in both)}


# ------------------------------------------------------------------------------------------ inputs
def _blocks(n, block):
    return (n + block - 1) // block


def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    ctx, q_len = _lens(c)
    bs, hk, d, b = c["block"], c["kv_heads"], c["dim"], c["batch"]
    own_blocks = [_blocks(n, bs) for n in ctx]
    most = max(ctx)
    pre = _prefixes(c) if c["op"] == "prefix" else []
    nb = _blocks(max([most] + pre), bs)
    keep_blocks = [_blocks(min(n, c["keep"]), bs) for n in ctx] if c["op"] == "evict" else []
    n_src = sum(own_blocks) + sum(_blocks(n, bs) for n in pre)
    n_slots = n_src + sum(keep_blocks) + 1                       # the last slot belongs to nobody
    shape = (1, n_slots, hk, bs, d)

    def rows(heavy):
        x = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)
        if heavy:   # one key in a hundred stands out
            x *= 1 + 3 * (torch.rand(shape[:-1], generator=g, device="cuda") < 0.01).unsqueeze(-1)
        x = x.to(torch.bfloat16)
        return x if c["kv"] == _BF16 else (x.float() / 0.05).clamp_(-448, 448).to(torch.float8_e4m3fn)

    k, v = rows(True), rows(False)
    order = torch.randperm(n_src, generator=g, device="cuda").to(torch.int32)

    def tables(counts, at, ids):
        t = torch.full((len(counts), nb), -1, dtype=torch.int32, device="cuda")
        for i, n in enumerate(counts):
            t[i, :n] = ids[at:at + n]
            at += n
        return t, at

    s = {"case": dict(c), "k": k, "v": v, "scale": 1.0 if c["kv"] == _BF16 else 0.05,
         "ctx_len": torch.tensor(ctx, dtype=torch.int32, device="cuda")}
    s["block2slot"], at = tables(own_blocks, 0, order)
    if pre:
        s["prefix2slot"], at = tables([_blocks(n, bs) for n in pre], at, order)
        s["prefix_len"] = torch.tensor(pre, dtype=torch.int32, device="cuda")
        s["prefix_req"] = torch.arange(0, b + 1, b // len(pre), dtype=torch.int32, device="cuda")
    n_tok = sum(q_len)
    if c["op"] == "evict":
        ids = torch.arange(n_slots, dtype=torch.int32, device="cuda")
        s["dst2slot"], _ = tables(keep_blocks, n_src, ids)
        for x in (k, v):
            x.view(torch.uint8)[:, n_src:] = 0
        s["n_src"] = n_src
        # accumulated softmax weights: most keys little, some much
        w = torch.rand((b, hk, nb * bs), generator=g, device="cuda").log_().neg_().pow_(3)
        s["weight"] = w
        s["weight_out"] = torch.zeros_like(w)
        s["kept"] = torch.full((b, hk, c["keep"]), -1, dtype=torch.int32, device="cuda")
        s["n_kept"] = torch.zeros(b, dtype=torch.int32, device="cuda")
    else:
        s["q"] = torch.randn((n_tok, c["heads"], d), generator=g, device="cuda").to(torch.bfloat16)
        s["out"] = torch.empty_like(s["q"])
        cu = [0]
        for m in q_len:
            cu.append(cu[-1] + m)
        s["cu_q"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
        s["step"] = min(256, max(q_len))
        s["n_blocks"] = sum(_blocks(m, s["step"]) for m in q_len)
        if c["op"] == "weights":
            w = torch.rand((b, hk, nb * bs), generator=g, device="cuda")
            s["weight"] = w * (torch.arange(nb * bs, device="cuda") < s["ctx_len"].view(-1, 1, 1))
    s["n_tok"], s["most"] = n_tok, most
    if own:
        import sparse_kv_cache_decode_gb300 as K
        s["pool"] = K.Pool(K.make_pool_config(
            n_layer=1, n_slots=n_slots, n_q_head=c["heads"], n_kv_head=hk, head_dim=d, block_size=bs, max_ctx=nb * bs, max_req=b,
            max_tokens=max(1, n_tok), max_prefix_tokens=n_tok if pre else 0, kv_dtype=c["kv"], k_scale=s["scale"], v_scale=s["scale"]), k, v)
    return s


# ------------------------------------------------------------------------------------------ plain forms
def _rows(side, table, idx, scale):
    """Cache rows of token indices idx [R][T] (clamped by the caller) through table [R][blocks], fp32 [R][kv heads][T][dim]."""
    bs = side.shape[3]
    slot = torch.gather(table.long(), 1, idx // bs).clamp_(min=0)
    x = side[0].view(torch.uint8)[slot, :, idx % bs].view(side.dtype).float()
    return (x * scale).transpose(1, 2)


def _softmax(logits, seen):
    """exp(logits - max) over the seen columns, and its sum (1 where a row sees nothing)."""
    logits = torch.where(seen, logits, -math.inf)
    m = logits.amax(-1, keepdim=True)
    p = torch.exp(logits - torch.where(m == -math.inf, 0.0, m))
    s = p.sum(-1, keepdim=True)
    return p, torch.where(s == 0, 1.0, s)


def _plain_attention(s):
    """Blocks of `step` query tokens, each against the span of keys its window reaches and the first `sink` keys."""
    c, cu, ctx = s["case"], s["cu_q"].long(), s["ctx_len"].long()
    step, n, hq, hk, d, window, sink = s["step"], s["n_tok"], c["heads"], c["kv_heads"], c["dim"], c["window"], c["sink"]
    g = hq // hk
    dev = cu.device
    ends = torch.cumsum((cu[1:] - cu[:-1] + step - 1) // step, 0)
    b = torch.arange(s["n_blocks"], device=dev)
    r = torch.searchsorted(ends, b, right=True)
    before = torch.where(r > 0, ends[(r - 1).clamp(min=0)], 0)
    row = (cu[r] + (b - before) * step).unsqueeze(1) + torch.arange(step, device=dev)
    real = row < cu[r + 1].unsqueeze(1)
    pos = ctx[r].unsqueeze(1) - cu[r + 1].unsqueeze(1) + row                            # the query tokens' positions
    q = s["q"][row.clamp(max=n - 1)].float()
    q = q.view(-1, step, hk, g, d).permute(0, 2, 3, 1, 4).reshape(-1, hk, g * step, d)
    most = s["most"]
    low = (pos[:, :1] - window + 1).clamp(min=0) if window else torch.zeros_like(pos[:, :1])
    key = low + torch.arange(min(most, window + step - 1) if window else most, device=dev)
    if sink and window:
        first = torch.arange(min(sink, most), device=dev).expand(len(b), -1)
        key = torch.cat((key, torch.where(first < low, first, 1 << 30)), 1)
    k, p = key.unsqueeze(1), pos.unsqueeze(2)
    seen = (k <= p) & real.unsqueeze(2)
    if window:
        seen &= (p - k < window) | (k < sink)
    at = key.clamp(max=most - 1)
    table = s["block2slot"][r]
    logits = q @ _rows(s["k"], table, at, s["scale"]).transpose(2, 3) / math.sqrt(d)
    seen = seen.unsqueeze(1).expand(-1, g, -1, -1).reshape(len(b), 1, g * step, -1)
    prob, total = _softmax(logits, seen)
    del logits
    o = (prob @ _rows(s["v"], table, at, s["scale"])) / total
    o = o.view(-1, hk, g, step, d).permute(0, 3, 1, 2, 4).reshape(-1, hq, d).to(torch.bfloat16)
    out = torch.empty((n + 1, hq, d), dtype=torch.bfloat16, device=dev)
    out[torch.where(real, row, n).reshape(-1)] = o
    if c["op"] == "window":
        return out[:n]
    w = torch.zeros((c["batch"], hk, s["weight"].shape[2]), device=dev)
    w[:, :, :most].index_add_(0, r, (prob / total).sum(2))
    t = torch.arange(w.shape[2], device=dev)
    new = t >= (ctx - cu[1:] + cu[:-1]).view(-1, 1, 1)              # the call's own tokens start here
    there = t < ctx.view(-1, 1, 1)
    s["weight"].copy_(torch.where(there, torch.where(new, w, s["weight"] + w), s["weight"]))
    return out[:n], s["weight"]


def _plain_prefix(s):
    c = s["case"]
    b, m, hq, hk, d, n_pre = c["batch"], c["q_len"], c["heads"], c["kv_heads"], c["dim"], c["prefixes"]
    g, dev = hq // hk, s["q"].device
    q = s["q"].float().view(b, m, hk, g, d).permute(0, 2, 3, 1, 4)                      # [b][hk][g][m][d]
    t = torch.arange(c["prefix"], device=dev)
    at = t.expand(n_pre, -1)
    kp, vp = (_rows(s[x], s["prefix2slot"], at, s["scale"]) for x in ("k", "v"))
    shared = q.reshape(n_pre, b // n_pre, hk, g * m, d).transpose(1, 2).reshape(n_pre, hk, -1, d)
    first = shared @ kp.transpose(2, 3) / math.sqrt(d)
    first = torch.where(t < s["prefix_len"].view(-1, 1, 1, 1), first, -math.inf)
    first = first.view(n_pre, hk, b // n_pre, g * m, -1).transpose(1, 2).reshape(b, hk, g * m, -1)
    key = torch.arange(max(_lens(c)[0]), device=dev)
    ctx = s["ctx_len"].long()
    at = key.expand(b, -1)
    rest = q.reshape(b, hk, g * m, d) @ _rows(s["k"], s["block2slot"], at, s["scale"]).transpose(2, 3) / math.sqrt(d)
    pos = ctx.view(-1, 1) - m + torch.arange(m, device=dev)
    seen = (key <= pos.unsqueeze(2)).unsqueeze(1).expand(-1, g, -1, -1).reshape(b, 1, g * m, -1)
    rest = torch.where(seen, rest, -math.inf)
    top = torch.maximum(first.amax(-1, keepdim=True), rest.amax(-1, keepdim=True))
    first, rest = torch.exp(first - top), torch.exp(rest - top)
    total = first.sum(-1, keepdim=True) + rest.sum(-1, keepdim=True)
    o = rest @ _rows(s["v"], s["block2slot"], at, s["scale"])
    first = first.view(n_pre, b // n_pre, hk, g * m, -1).transpose(1, 2).reshape(n_pre, hk, -1, c["prefix"])
    o += (first @ vp).view(n_pre, hk, b // n_pre, g * m, d).transpose(1, 2).reshape(b, hk, g * m, d)
    o = (o / total).view(b, hk, g, m, d).permute(0, 3, 1, 2, 4)
    return o.reshape(-1, hq, d).to(torch.bfloat16)


def _plain_evict(s):
    c = s["case"]
    keep, w, ctx = c["keep"], s["weight"], s["ctx_len"].long().view(-1, 1, 1)
    t = torch.arange(w.shape[2], device=w.device)
    there = t < ctx
    forced = (t < c["sink"]) | (t >= ctx - c["recent"])
    key = torch.where(there, torch.where(forced, math.inf, w), -math.inf)
    best = torch.sort(key, dim=2, descending=True, stable=True).indices[:, :, :min(keep, w.shape[2])]
    held = torch.zeros(w.shape, dtype=torch.bool, device=w.device).scatter_(2, best, True) & there
    kept = torch.sort(torch.where(held, t, 1 << 30), dim=2).values[:, :, :min(keep, w.shape[2])]
    there = kept < (1 << 30)
    at = torch.where(there, kept, 0)
    n = kept.shape[2]
    s["kept"][:, :, :n] = torch.where(there, kept, -1).int()
    s["n_kept"].copy_(ctx.view(-1).clamp(max=keep))
    s["weight_out"][:, :, :n] = torch.where(there, torch.gather(w, 2, at), s["weight_out"][:, :, :n])
    bs, hk = c["block"], kept.shape[1]
    i = torch.arange(n, device=w.device)
    head = torch.arange(hk, device=w.device).view(1, -1, 1)
    src = torch.gather(s["block2slot"].long().unsqueeze(1).expand(-1, hk, -1), 2, at // bs).clamp_(min=0)
    dst = torch.where(there, s["dst2slot"].long()[:, i // bs].unsqueeze(1), s["k"].shape[1] - 1)
    for x in (s["k"], s["v"]):
        x = x[0].view(torch.uint8)
        x[dst, head, i % bs] = x[src, head, at % bs]
    return _evicted(s)


def _evicted(s):
    return s["kept"], s["n_kept"], s["weight_out"], s["k"][:, s["n_src"]:-1], s["v"][:, s["n_src"]:-1]


def run(s):
    c = s["case"]
    if not own:
        return (_plain_evict if c["op"] == "evict" else _plain_prefix if c["op"] == "prefix" else _plain_attention)(s)
    if c["op"] == "evict":
        s["pool"].evict(0, s["weight"], s["ctx_len"], s["block2slot"], c["keep"], c["sink"], c["recent"], s["dst2slot"], s["kept"],
                        s["n_kept"], s["weight_out"])
        return _evicted(s)
    if c["op"] == "prefix":
        s["pool"].prefix_attn(0, s["q"], s["cu_q"], s["ctx_len"], s["block2slot"], s["prefix_req"], s["prefix_len"], s["prefix2slot"],
                              s["out"])
        return s["out"]
    if c["op"] == "weights":
        s["pool"].attn(0, s["q"], s["cu_q"], s["ctx_len"], s["block2slot"], s["out"], weight=s["weight"])
        return s["out"], s["weight"]
    s["pool"].attn(0, s["q"], s["cu_q"], s["ctx_len"], s["block2slot"], s["out"], window=c["window"], n_sink=c["sink"])
    return s["out"]


# ------------------------------------------------------------------------------------------ exact values
def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "evict":
        return None
    hq, hk, d, bs = c["heads"], c["kv_heads"], c["dim"], c["block"]
    g = hq // hk
    ctx, q_len = _lens(c)
    out = torch.zeros((s["n_tok"], hq, d), dtype=torch.float64, device="cuda")
    weight = s["weight"].double() if c["op"] == "weights" else None

    def cached(side, table, lo, hi):
        x = side[0][table[lo // bs:_blocks(hi, bs)].long()].double() * s["scale"]         # [blocks][hk][bs][d]
        x = x.permute(1, 0, 2, 3).reshape(hk, -1, d)
        return x[:, lo - lo // bs * bs:][:, :hi - lo]

    at = 0
    for r, (n, m) in enumerate(zip(ctx, q_len)):
        added = torch.zeros((hk, n), dtype=torch.float64, device="cuda")
        for i0 in range(0, m if n else 0, 512):
            i1 = min(m, i0 + 512)
            p0, p1 = n - m + i0, n - m + i1
            if p1 <= 0:
                continue
            lo = max(0, p0 - c["window"] + 1) if c["window"] else 0
            first = min(c["sink"], lo)
            parts = [(s["block2slot"][r], 0, first)] if first else []
            parts.append((s["block2slot"][r], lo, p1))
            where = list(range(first)) + list(range(lo, p1))
            t = torch.tensor(where, device="cuda")
            shared = 0
            if c["op"] == "prefix":
                i = r // (c["batch"] // c["prefixes"])
                shared = int(s["prefix_len"][i])
                parts.insert(0, (s["prefix2slot"][i], 0, shared))
            k, v = (torch.cat([cached(s[x], *a) for a in parts], 1) for x in ("k", "v"))
            x = s["q"][at + i0:at + i1].double().view(i1 - i0, hk, g, d).permute(1, 2, 0, 3)
            a = torch.einsum("hgid,htd->hgit", x, k) / math.sqrt(d)
            p = torch.arange(p0, p1, device="cuda").unsqueeze(1)
            hide = t > p
            if c["window"]:
                hide = hide | ((p - t >= c["window"]) & (t >= c["sink"]))
            a[..., shared:].masked_fill_(hide, -math.inf)
            a = torch.softmax(a, -1).nan_to_num_(0.0)
            out[at + i0:at + i1] = torch.einsum("hgit,htd->ihgd", a, v).reshape(i1 - i0, hq, d)
            if weight is not None:
                added[:, :p1] += a.sum((1, 2))
        if weight is not None and n:
            weight[r, :, :n - m] += added[:, :n - m]
            weight[r, :, n - m:n] = added[:, n - m:]
        at += m
    return out if weight is None else (out, weight)
