"""What stands between a projection and the attention over a paged pool: cases, plain forms and exact values.

Four operators around cache blocks, K and V [slots][kv heads][block][head dim]:

  tables      block tables, slot maps and positions of a batch, built from the requests' lengths and a ring of free slots
  rotate      norms of queries and keys for each head and the rotation by their positions, along one or several axes
  append      the same rotation, with K and V written to their places in the pool in the same pass
  reposition  keys that stay after an eviction, rotated from their old positions to their new ones

`own` False: elementary torch operations in 32 bits (angles in 64).  `own` True: the framework's calls.
"""
import math
import random

import torch

own = False

_BF16, _FP8 = "bf16", "fp8"
_EPS = 1e-6


# ------------------------------------------------------------------------------------------ cases
def _tables(name, batch, ctx, q_len, block):
    return {"name": name, "op": "tables", "batch": batch, "ctx": ctx, "q_len": q_len, "block": block}


def _rows(name, op, batch, ctx, q_len, heads, kv_heads, dim, rot=0, theta=10000.0, axes=1, cycle=False, adjacent=False, norm=True):
    """rot: dims that turn (0: all); axes: of the positions; cycle: the axes alternate over the pairs, else a run of pairs each;
    adjacent: dims 2i and 2i + 1 are a pair, else i and i + rot / 2."""
    return {"name": name, "op": op, "batch": batch, "ctx": ctx, "q_len": q_len, "heads": heads, "kv_heads": kv_heads, "dim": dim,
            "rot": rot or dim, "theta": theta, "axes": axes, "cycle": cycle, "adjacent": adjacent, "norm": norm}


def _reposition(name, batch, ctx, keep, kv_heads, dim, block, kv, theta):
    return {"name": name, "op": "reposition", "batch": batch, "ctx": ctx, "keep": keep, "heads": kv_heads, "kv_heads": kv_heads, "dim": dim,
            "block": block, "kv": kv, "rot": dim, "theta": theta, "axes": 1, "cycle": False, "adjacent": False}


def listed():
    return [
        # a serving batch's next tokens: one request in sixteen starts a block
        _tables("tables step", 64, 32768, 1, 16),
        # a token and its five drafts for many requests, the drafts' blocks taken back after they were refused
        _tables("tables drafts", 500, 8000, 6, 16),
        # a wave of prompts that all start at once
        _tables("tables prompts", 24, 32768, 32768, 64),
        # one user's next token, normed and rotated for a step that scores and attends by itself
        _rows("rotate one token", "rotate", 1, 32768, 1, 32, 8, 128, theta=500000.0),
        # the 64 rotated dims of 128 query heads and one shared key, inside rows of 576
        _rows("rotate latent batch", "rotate", 64, 131072, 1, 128, 1, 64, adjacent=True, norm=False) | {"row": 576},
        # prompts with images and video: positions in time, height and width
        _rows("rotate images", "rotate", 3, 4099, 4099, 28, 4, 128, theta=1e6, axes=3, norm=False),
        # one user's next token into the pool: the call's latency is what counts
        _rows("append one token", "append", 1, 4096, 1, 32, 8, 128, theta=500000.0) | {"block": 16, "kv": _BF16},
        # a serving batch's next tokens into an 8-bit pool, contexts up to 128K
        _rows("append batch fp8", "append", 128, 131072, 1, 32, 8, 128, theta=500000.0) | {"block": 64, "kv": _FP8},
        # a prompt of 16K tokens
        _rows("append prompt", "append", 1, 16384, 16384, 32, 8, 128, theta=1e6) | {"block": 64, "kv": _BF16},
        # chunks of prompts with images and single tokens in one batch, small heads, part of their dims turning, odd lengths
        _rows("append mixed", "append", 9, 5001, 701, 24, 8, 64, rot=48, theta=1e6, axes=3, cycle=True) | {"block": 32, "kv": _BF16},
        # caches that were cut back to 2048 tokens when one more block had filled
        _reposition("reposition step", 8, 2112, 2048, 8, 128, 64, _BF16, 500000.0),
        # long prompts cut down to 4096 tokens each, 8-bit pool
        _reposition("reposition prompts fp8", 32, 65536, 4096, 8, 128, 16, _FP8, 500000.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    most = {op: max(w["bytes"] for c in listed() if c["op"] == op for w in [work(c)]) for op in ("tables", "rotate", "append", "reposition")}
    while True:
        op = rng.choice(("tables", "rotate", "rotate", "append", "append", "append", "reposition"))
        heads, kv_heads = rng.choice(((32, 8), (8, 2), (24, 8), (16, 16), (40, 8), (28, 4), (7, 1)))
        dim, block, kv = rng.choice((64, 128)), rng.choice((16, 32, 64, 128)), rng.choice((_BF16, _BF16, _FP8))
        theta = rng.choice((10000.0, 500000.0, 1e6))
        batch, ctx = _log(rng, 1, 1024), _log(rng, 4, 65536)
        if op == "tables":
            c = _tables("", batch, ctx, min(ctx, rng.choice((1, rng.randint(2, 8), _log(rng, 9, 32768)))), block)
            if batch * _blocks(ctx, block) > 1 << 20:
                continue
        elif op == "reposition":
            c = _reposition("", _log(rng, 1, 64), max(ctx, 20), max(16, min(4096, int(ctx * rng.uniform(0.02, 0.99)))), kv_heads, dim, block,
                            kv, theta)
        else:
            one = rng.random() < 0.4
            batch = batch if one else _log(rng, 1, 16)
            axes = rng.choice((1, 1, 2, 3, 4))
            if op == "rotate":
                dim = rng.choice((64, 128, 256))
            c = _rows("", op, batch, ctx, 1 if one else min(ctx, _log(rng, 2, 16384)), heads, kv_heads, dim,
                      rng.choice((dim, dim, dim // 2, 48)), theta, axes, axes > 1 and rng.random() < 0.5, rng.random() < 0.4, rng.random() < 0.7)
            if op == "append":
                c |= {"block": block, "kv": kv}
            elif rng.random() < 0.3:
                c |= {"row": dim + rng.choice((16, 128, 512))}
        c.pop("name")
        if work(c)["bytes"] <= most[op]:
            return c


def _lens(c):
    """Each request's context (with the call's own tokens) and number of new tokens; part of the case, not of the seed."""
    r = random.Random(repr(sorted((k, v) for k, v in c.items() if k != "name")))
    ctx, q = [], []
    for i in range(c["batch"]):
        n = c["ctx"] if i == 0 else 1 + int((c["ctx"] - 1) * (1 - 0.75 * r.random()))
        m = c.get("q_len", 0)
        if c["op"] == "reposition":
            n = n if i == 0 else int(0.95 * c["keep"] + (c["ctx"] - 0.95 * c["keep"]) * r.random())
        elif i and m > 8:
            m = n if m == c["ctx"] else 1 if r.random() < 0.4 else 1 + int(m * r.random())   # whole prompts, or chunks and tokens
        if i == 3 and c["op"] != "reposition":
            n = 1           # a request's first token
        if i == 7 and c["op"] != "reposition":
            n, m = 0, 1     # a free place of the batch
        ctx.append(n)
        q.append(m if n == 0 else min(m, n))
    return ctx, q


def _axes(c):
    """The axis of each pair of dims."""
    n, a = c["rot"] // 2, c["axes"]
    if c["cycle"]:
        return [i % a for i in range(n)]
    first = n // (2 * a) if a > 1 else 0                             # time turns fewer pairs than the others
    return [0 if i < first else (i - first) * (a - 1) // (n - first) + 1 if a > 1 else 0 for i in range(n)]


def _blocks(n, block):
    return (n + block - 1) // block


# ------------------------------------------------------------------------------------------ floors
def work(c):
    ctx, q = _lens(c)
    if c["op"] == "tables":
        # there: lengths, blocks held (read and written) and offsets, new slots out of the ring into the table, a place and a position
        # a token; back: lengths and blocks held, the slots out of the table into the ring
        new = sum(_blocks(n, c["block"]) - _blocks(max(0, n - m), c["block"]) for n, m in zip(ctx, q))
        return {"bytes": c["batch"] * 28 + new * 16 + sum(q) * 12, "flops": 0}
    hk, d = c["kv_heads"], c["dim"]
    if c["op"] == "reposition":
        rows = sum(min(n, c["keep"]) for n in ctx) * hk
        return {"bytes": rows * (4 + 2 * d * (2 if c["kv"] == _BF16 else 1)), "flops": rows * d * 3}
    n, turned = sum(q), c["heads"] + hk
    per = turned * d * 4 + 4 * c["axes"]                             # q and k in and out, positions
    if c["op"] == "append":
        e = 2 if c["kv"] == _BF16 else 1
        per = c["heads"] * d * 4 + 2 * hk * d * (2 + e) + 4 * c["axes"] + 8
    return {"bytes": n * per + (8 * d if c["norm"] else 0), "flops": n * turned * (3 * c["rot"] + (4 * d if c["norm"] else 0))}


# ------------------------------------------------------------------------------------------ inputs
def _positions(c, ctx, q):
    """[axes][tokens]: text counts on along all axes; every other run is an image, whose patches share a time and spread over the
    other axes."""
    r = random.Random(c["ctx"] * 7 + c["batch"])
    out = []
    for n, m in zip(ctx, q):
        if c["axes"] == 1:
            out.append(torch.arange(n - m, n).view(1, -1))
            continue
        at, left, parts, image = n - m, m, [], False
        while left:
            size = min(left, r.randint(20, 400))
            i = torch.arange(size)
            wide = r.randint(8, 24)
            parts.append(at + torch.stack([torch.zeros_like(i) if a == 0 else i // wide if a == 1 else i % wide + a - 2
                                           for a in range(c["axes"])]) if image else at + i.expand(c["axes"], -1))
            at, left, image = int(parts[-1].max()) + 1, left - size, not image
        out.append(torch.cat(parts, 1))
    return torch.cat(out, 1).to(torch.int32).cuda().contiguous()


def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    ctx, q = _lens(c)
    n_tok, b = sum(q), c["batch"]
    s = {"case": dict(c), "n_tok": n_tok}
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    if own:
        import sparse_kv_cache_decode_gb300 as K
    if "block" in c:
        bs = c["block"]
        need = [_blocks(min(n, c.get("keep", n)), bs) for n in ctx]
        nb = max(need)
        n_slots = sum(need) + 5
        ids = torch.randperm(n_slots - 1, generator=g, device="cuda").to(torch.int32)
        ids = torch.cat((ids, torch.full((1,), n_slots - 1, dtype=torch.int32, device="cuda")))     # the last slot belongs to nobody
        cfg = dict(n_layer=1, n_slots=n_slots, n_q_head=c.get("heads", 8), n_kv_head=c.get("kv_heads", 2), head_dim=c.get("dim", 64), block_size=bs,
                   max_ctx=nb * bs, max_req=b, max_tokens=max(1, n_tok), kv_dtype=c.get("kv", _BF16))
    if c["op"] == "tables":
        before = [max(0, n - m) for n, m in zip(ctx, q)]             # lengths ahead of the call
        held = [_blocks(n, bs) for n in before]
        table, at = torch.full((b, nb), -1, dtype=torch.int32, device="cuda"), 0
        for i, h in enumerate(held):
            table[i, :h] = ids[at:at + h]
            at += h
        head = seed % n_slots
        s |= {"table": table, "held": dev(held), "state": dev([head, n_slots - at, 0]),
              "ring": torch.cat((ids[at:], torch.full((at,), -1, dtype=torch.int32, device="cuda"))).roll(head),
              "ctx": dev(ctx), "before": dev(before), "cu": dev([sum(q[:i]) for i in range(b + 1)]),
              "delta": torch.randint(0, 3, (b,), generator=g, device="cuda", dtype=torch.int32) * -50,
              "place": torch.empty(n_tok, dtype=torch.int64, device="cuda"), "pos": torch.empty(n_tok, dtype=torch.int32, device="cuda")}
        if own:
            shape = (1, n_slots, cfg["n_kv_head"], bs, cfg["head_dim"])
            pool = K.Pool(K.make_pool_config(**cfg), *(torch.zeros(shape, dtype=torch.bfloat16, device="cuda") for _ in range(2)))
            s["tables"] = K.BlockTables(pool, s["table"], s["held"], s["ring"], s["state"])
        return s
    hq, hk, d = c["heads"], c["kv_heads"], c["dim"]
    s["freq"] = c["theta"] ** (-torch.arange(0, c["rot"], 2, dtype=torch.float64, device="cuda") / c["rot"])
    s["axis"] = torch.tensor(_axes(c), device="cuda")
    if own:
        s["rope"] = K.Rope(K.make_rope_config(d, c["rot"], theta=c["theta"], adjacent=c["adjacent"], axes=_axes(c) if c["axes"] > 1 else None,
                                              norm_eps=_EPS))

    def values(*shape):     # a few channels of a projection stand out
        return torch.randn(shape, generator=g, device="cuda") * (1 + 6 * (torch.rand(shape[-1], generator=g, device="cuda") < 0.03))

    if c["op"] != "rotate":
        shape = (1, n_slots, hk, bs, d)
        kv = {_BF16: torch.bfloat16, _FP8: torch.float8_e4m3fn}[c["kv"]]
        s["scale"] = 1.0 if c["kv"] == _BF16 else 0.05
        if c["op"] == "reposition":
            s["k"] = (values(*shape) / s["scale"]).clamp_(-448, 448).to(kv)
            s["v"] = torch.zeros((), device="cuda").to(kv).expand(shape).contiguous()
        else:
            s["k"], s["v"] = (torch.zeros(shape, device="cuda").to(kv) for _ in range(2))
        if own:
            s["pool"] = K.Pool(K.make_pool_config(**cfg, k_scale=s["scale"], v_scale=s["scale"]), s["k"], s["v"])
    if c["op"] == "reposition":
        keep = c["keep"]
        s["table"], at = torch.full((b, nb), -1, dtype=torch.int32, device="cuda"), 0
        s["kept"] = torch.full((b, hk, keep), -1, dtype=torch.int32, device="cuda")
        for i, n in enumerate(ctx):
            s["table"][i, :need[i]] = ids[at:at + need[i]]
            at += need[i]
            k = min(n, keep)
            w = torch.rand((hk, n), generator=g, device="cuda")
            w[:, :4] = w[:, n - min(n, 8):] = 2.0                     # the first and the newest tokens always stay
            s["kept"][i, :, :k] = w.topk(k, dim=1).indices.sort(dim=1).values.to(torch.int32)
        s["n_kept"] = dev([min(n, keep) for n in ctx])
        return s
    s["pos"] = _positions(c, ctx, q)
    row = c.get("row", 0)
    if row:                                                          # the rotated dims are the last of longer rows
        s["q"], s["k_new"] = (values(n_tok, h, row).to(torch.bfloat16)[:, :, row - d:] for h in (hq, hk))
        s["q_out"], s["k_out"] = (torch.zeros((n_tok, h, row), dtype=torch.bfloat16, device="cuda")[:, :, row - d:] for h in (hq, hk))
    else:                                                            # parts of a fused projection
        x = values(n_tok, hq + 2 * hk, d).to(torch.bfloat16)
        s["q"], s["k_new"], s["v_new"] = x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:]
        s["q_out"], s["k_out"] = (torch.zeros((n_tok, h, d), dtype=torch.bfloat16, device="cuda") for h in (hq, hk))
    if c["norm"]:
        s["q_norm"], s["k_norm"] = (1 + 0.2 * torch.randn(d, generator=g, device="cuda") for _ in range(2))
    if c["op"] == "append":
        pos = torch.cat([torch.arange(n - m, n) for n, m in zip(ctx, q)]).cuda()      # places go by the token's number, not its axes
        first = torch.tensor([sum(need[:i]) for i in range(b)], device="cuda")
        block = first.repeat_interleave(torch.tensor(q, device="cuda"), output_size=n_tok) + pos.clamp(min=0) // bs
        s["place"] = torch.where(pos < 0, -1, ids[block].long() * bs + pos % bs)
    return s


# ------------------------------------------------------------------------------------------ plain forms
def _plain_tables(s, ctx, tokens):
    """Blocks past a request's length go to the end of the ring, request by request, then missing ones come from its front."""
    bs, table, ring, held = s["case"]["block"], s["table"], s["ring"], s["held"].long()
    size = ring.numel()
    head, n_free = s["state"][0].long(), s["state"][1].long()
    ctx = ctx.long()
    need = (ctx + bs - 1) // bs
    take, give = (need - held).clamp(min=0), (held - need).clamp(min=0)
    end = head + n_free
    b = torch.arange(table.shape[1], device=ring.device)
    j = (torch.cumsum(give, 0) - give).unsqueeze(1) + b - need.unsqueeze(1)
    there = (b >= need.unsqueeze(1)) & (b < held.unsqueeze(1))
    more = torch.cat((ring, ring[:1]))                               # the last entry takes what goes nowhere
    more[torch.where(there, (end + j) % size, size).reshape(-1)] = table.reshape(-1)
    ring.copy_(more[:size])
    i = (torch.cumsum(take, 0) - take).unsqueeze(1) + b - held.unsqueeze(1)
    there = (b >= held.unsqueeze(1)) & (b < need.unsqueeze(1))
    table.copy_(torch.where(there, ring[(head + i) % size], table))
    s["held"].copy_(need)
    s["state"][0] = (head + take.sum()) % size
    s["state"][1] = n_free + give.sum() - take.sum()
    if tokens:
        cu = s["cu"].long()
        t = torch.arange(s["n_tok"], device=cu.device)
        r = torch.searchsorted(cu, t, right=True) - 1
        p = ctx[r] - cu[r + 1] + t
        s["pos"].copy_(p + s["delta"].long()[r])
        s["place"].copy_(torch.where(p < 0, -1, table.long()[r, p.clamp(min=0) // bs] * bs + p % bs))


def _plain_turn(x, angle, adjacent):
    """x [..., dim] fp32, its first 2 * pairs dims turned by angle [..., pairs] (64 bits)."""
    n = angle.shape[-1]
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    a, b = (x[..., 0:2 * n:2], x[..., 1:2 * n:2]) if adjacent else (x[..., :n], x[..., n:2 * n])
    y = (a * cos - b * sin, b * cos + a * sin)
    y = torch.stack(y, -1).flatten(-2) if adjacent else torch.cat(y, -1)
    return torch.cat((y, x[..., 2 * n:]), -1)


def _plain_rows(s, x, weight):
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + _EPS) * weight
    angle = s["pos"][s["axis"]].T.double() * s["freq"]
    return _plain_turn(x, angle.unsqueeze(1), s["case"]["adjacent"])


def _plain_store(pool, place, x, scale):
    """Rows x [tokens][heads][dim] to their places; those without one end in a row that is cut off."""
    _, n_slots, hk, bs, d = pool.shape
    if pool.dtype != torch.bfloat16:
        x = (x / scale).clamp(-448, 448)
    x = x.to(pool.dtype).view(torch.int16 if pool.dtype == torch.bfloat16 else torch.uint8)
    flat = pool[0].view(x.dtype)
    held = flat[-1, :, -1].clone()                                   # (nobody's row)
    at = torch.where(place < 0, n_slots * bs - 1, place)
    flat[at // bs, :, at % bs] = x
    flat[-1, :, -1] = held


def _plain_reposition(s):
    c = s["case"]
    bs, n, hk = c["block"], c["keep"], c["kv_heads"]
    i = torch.arange(n, device="cuda")
    there = (i < s["n_kept"].view(-1, 1)).unsqueeze(1).expand(-1, hk, -1)
    slot = torch.where(there, s["table"][:, i // bs].unsqueeze(1), s["k"].shape[1] - 1).long()
    h = torch.arange(hk, device="cuda").view(1, -1, 1)
    kind = torch.int16 if c["kv"] == _BF16 else torch.uint8
    flat = s["k"][0].view(kind)
    x = flat[slot, h, i % bs]
    by = (i - s["kept"]).unsqueeze(-1).double() * s["freq"]
    y = _plain_turn(x.view(s["k"].dtype).float(), by, c["adjacent"])
    if c["kv"] == _FP8:
        y = y.clamp(-448, 448)
    held = flat[-1].clone()
    flat[slot, h, i % bs] = y.to(s["k"].dtype).view(kind)
    flat[-1] = held


def _tables_out(s):
    return s["table"], s["ring"], s["held"], s["state"], s["place"], s["pos"]


def run(s):
    c = s["case"]
    if c["op"] == "tables":
        if own:
            s["tables"].reserve(s["ctx"], s["cu"], s["place"], s["pos"], pos_delta=s["delta"])
            s["tables"].reserve(s["before"])
        else:
            _plain_tables(s, s["ctx"], True)
            _plain_tables(s, s["before"], False)
        return _tables_out(s)
    if c["op"] == "reposition":
        if own:
            s["pool"].reposition(0, s["rope"], s["kept"], s["n_kept"], s["table"])
        else:
            _plain_reposition(s)
        return s["k"]
    q_norm, k_norm = s.get("q_norm"), s.get("k_norm")
    if c["op"] == "rotate":
        if own:
            s["rope"].rotate(s["q"], s["pos"], s["q_out"], s["k_new"], s["k_out"], q_norm=q_norm, k_norm=k_norm)
        else:
            s["q_out"].copy_(_plain_rows(s, s["q"], q_norm))
            s["k_out"].copy_(_plain_rows(s, s["k_new"], k_norm))
        return s["q_out"], s["k_out"]
    if own:
        s["pool"].rotate_append(0, s["rope"], s["q"], s["k_new"], s["v_new"], s["pos"], s["place"], s["q_out"], q_norm=q_norm, k_norm=k_norm)
    else:
        s["q_out"].copy_(_plain_rows(s, s["q"], q_norm))
        _plain_store(s["k"], s["place"], _plain_rows(s, s["k_new"], k_norm), s["scale"])
        _plain_store(s["v"], s["place"], s["v_new"].float(), s["scale"])
    return s["q_out"], s["k"], s["v"]


# ------------------------------------------------------------------------------------------ exact values
def exact(c, seed):
    """Pairs as complex numbers, turned by a product with exp(i angle)."""
    if c["op"] == "tables":
        return None
    s = prepare(c, seed)
    rot, n = c["rot"], c["rot"] // 2
    freq = torch.exp(torch.arange(n, dtype=torch.float64, device="cuda") * (-math.log(c["theta"]) / n))

    def turned(x, pos):     # x [..., dim], pos [..., pairs]
        x = x.double().clone()
        z = x[..., :rot]
        z = torch.view_as_complex(z.unflatten(-1, (n, 2)).contiguous() if c["adjacent"] else z.unflatten(-1, (2, n)).transpose(-1, -2).contiguous())
        z = torch.view_as_real(z * torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), pos * freq))
        x[..., :rot] = (z if c["adjacent"] else z.transpose(-1, -2)).flatten(-2)
        return x

    if c["op"] == "reposition":
        k = s["k"].double()
        for i, m in enumerate(s["n_kept"].tolist()):
            for h in range(c["kv_heads"]):
                new = torch.arange(m, device="cuda")
                slots = s["table"][i].long()[new // c["block"]]
                by = (new - s["kept"][i, h, :m].long()).double().view(-1, 1)
                k[0, slots, h, new % c["block"]] = turned(k[0, slots, h, new % c["block"]], by)
        return k
    pos = torch.stack([s["pos"][a] for a in _axes(c)], 1).double().unsqueeze(1)

    def rows(x, weight):
        x = x.double()
        if weight is not None:
            x = x / torch.sqrt(x.square().sum(-1, keepdim=True) / c["dim"] + _EPS) * weight.double()
        return turned(x, pos)

    q, k = rows(s["q"], s.get("q_norm")), rows(s["k_new"], s.get("k_norm"))
    if c["op"] == "rotate":
        return q, k
    out = []
    for x in (k, s["v_new"].double()):
        pool = torch.zeros(s["k"].shape, dtype=torch.float64, device="cuda")
        ok = s["place"] >= 0
        at = s["place"][ok]
        pool[0, at // c["block"], :, at % c["block"]] = x[ok] / s["scale"]
        out.append(pool)
    return (q, *out)
