"""Cases and plain forms of the paged serving operators: block tables, the
query/key/value append, attention over the paged pool with a window and sinks,
and attention of a batch that shares a prefix.

The pool is the one cg_decode_into_paged fills: [L][2][num_pages][page_tokens][H][D].
``run`` computes each operator with elementary torch operations in 32 bits where
``own`` is false, and calls the library where it is true; ``exact`` gives the
same results from the definition in 64 bits.
"""
import math
import random

import torch

own = False

F16, BF16 = "float16", "bfloat16"


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # One decode step of a busy server: every request adds one token.
        dict(name="tables_step", op="tables", requests=256, held=8192, added=1, spread=0, page=16,
             base=0, mix=1),
        # Admission of a ragged batch of prompts, about 64K tokens at once.
        dict(name="tables_admit", op="tables", requests=61, held=0, added=2048, spread=1, page=16,
             base=1536, mix=2),
        # The decode step of a 64-request batch (grouped heads, normed queries and keys).
        dict(name="append_step", op="append", tokens=64, q_heads=32, kv_heads=8, dim=128, rot=128,
             norm=1, inter=0, page=16, far=32768, dtype=F16),
        # A prompt's chunk with as many key heads as query heads, no norm.
        dict(name="append_prompt", op="append", tokens=10752, q_heads=32, kv_heads=32, dim=128,
             rot=128, norm=0, inter=0, page=16, far=10752, dtype=F16),
        # bf16, small heads, half of each head rotated, pairs next to each other, odd count.
        dict(name="append_partial", op="append", tokens=4099, q_heads=16, kv_heads=2, dim=64,
             rot=32, norm=1, inter=1, page=48, far=131072, dtype=BF16),
        # A few requests, one token each: the latency of a step.
        dict(name="window_step_few", op="window", requests=4, held=2000, added=1, spread=1,
             q_heads=32, kv_heads=8, dim=128, page=16, window=1024, sinks=4, dtype=F16, mix=3),
        # A full batch of single tokens behind long contexts.
        dict(name="window_step_batch", op="window", requests=128, held=32768, added=1, spread=1,
             q_heads=32, kv_heads=8, dim=128, page=16, window=4096, sinks=4, dtype=F16, mix=4),
        # Ragged prompts in one call.
        dict(name="window_prompt", op="window", requests=3, held=0, added=8192, spread=1,
             q_heads=32, kv_heads=8, dim=128, page=16, window=4096, sinks=4, dtype=F16, mix=5),
        # Chunks behind what the requests hold already, small heads, odd pages, bf16, no window.
        dict(name="window_chunk", op="window", requests=7, held=1500, added=500, spread=1,
             q_heads=16, kv_heads=2, dim=64, page=48, window=0, sinks=0, dtype=BF16, mix=6),
        # A batch answering about one 1,536-token chunk, as many key heads as query heads.
        dict(name="shared_step", op="shared", prefix=1536, requests=32, held=200, added=1, spread=1,
             q_heads=32, kv_heads=32, dim=128, page=16, dtype=F16, mix=7),
        # A large batch behind a long shared document.
        dict(name="shared_step_long", op="shared", prefix=79872, requests=96, held=700, added=1,
             spread=1, q_heads=64, kv_heads=8, dim=128, page=16, dtype=F16, mix=8),
        # The questions of a batch, a few dozen tokens each, behind one document, bf16.
        dict(name="shared_ask", op="shared", prefix=10752, requests=24, held=0, added=61, spread=1,
             q_heads=32, kv_heads=8, dim=128, page=64, dtype=BF16, mix=9),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tables", "append", "window", "window", "shared", "shared"])
    page = rng.choice([1, 7, 16, 16, 32, 48, 64, 256]) if op != "tables" else rng.choice([8, 16, 32, 50])
    dtype = rng.choice([F16, BF16])
    mix = rng.randrange(1 << 30)
    heads = rng.choice([(32, 8), (32, 32), (64, 8), (16, 2), (8, 1), (6, 2), (7, 7), (20, 4)])
    dim = rng.choice([16, 64, 80, 96, 128, 128, 128, 256])
    if op == "tables":
        step = rng.random() < 0.5
        b = _log(rng, 1, 500)
        return dict(op=op, requests=b, held=_log(rng, 1, 8192) if step else rng.choice([0, 77]),
                    added=rng.randint(1, 4) if step else min(2048, _log(rng, 1, 65536 // b + 1)),
                    spread=rng.randint(0, 1), page=page, base=rng.choice([0, 1536]), mix=mix)
    if op == "append":
        width = (heads[0] + 2 * heads[1]) * dim
        return dict(op=op, tokens=min(_log(rng, 1, 11000), max(1, 100_000_000 // width)),
                    q_heads=heads[0], kv_heads=heads[1], dim=dim,
                    rot=rng.choice([dim, dim // 2]), norm=rng.randint(0, 1), inter=rng.randint(0, 1),
                    page=page, far=_log(rng, 16, 131072), dtype=dtype)
    if op == "window":
        window, sinks = rng.choice([(0, 0), (128, 4), (1000, 1), (1024, 0), (4096, 4), (4096, 130)])
        if rng.random() < 0.5:  # single tokens, or a few
            b, added = _log(rng, 1, 128), rng.choice([1, 1, 1, 2, 5])
            held = min(_log(rng, 1, 32768), max(1, 160_000_000 // (b * heads[1] * dim)))
        else:                   # prompts and chunks
            b, added = rng.randint(1, 6), _log(rng, 2, 4096)
            added = max(2, min(added, 12000 // b))
            held = rng.choice([0, 0, _log(rng, 1, 8000)])
            while b * added * (held + added) * heads[0] > 5e9 or \
                    b * added * (held + added) * heads[0] * dim > 4e11:
                held, added = held // 2, max(2, added // 2)
        return dict(op=op, requests=b, held=held, added=added, spread=rng.randint(0, 1),
                    q_heads=heads[0], kv_heads=heads[1], dim=dim, page=page, window=window,
                    sinks=sinks, dtype=dtype, mix=mix)
    b, added = _log(rng, 2, 96), rng.choice([1, 1, 1, 3, 61])
    added = max(1, min(added, 3000 // b))
    prefix = _log(rng, 64, 79872)
    rows = b * added * heads[0]
    prefix = max(64, min(prefix, 1_000_000_000 // rows, 80_000_000 // (heads[1] * dim)))
    return dict(op=op, prefix=prefix, requests=b, held=rng.choice([0, _log(rng, 1, 900)]),
                added=added, spread=rng.randint(0, 1), q_heads=heads[0], kv_heads=heads[1],
                dim=dim, page=page, dtype=dtype, mix=mix)


def _lengths(case):
    """(held, added) of every request: fixed by the case, ragged where it says so."""
    r = random.Random(case["mix"])
    held, added = [], []
    for _ in range(case["requests"]):
        f = r.uniform(0.25, 1.0) if case["spread"] else 1.0
        g = r.uniform(0.25, 1.0) if case["spread"] else 1.0
        held.append(int(case["held"] * f))
        added.append(max(1, int(case["added"] * g)))
    return held, added


def _pairs(case, held, added):
    """Visible (row, key) pairs and keys read, over all requests, of one key head."""
    window, sinks = case.get("window", 0), case.get("sinks", 0)
    pairs = keys = 0
    for h, n in zip(held, added):
        kv = h + n
        if not window:
            pairs += n * h + n * (n + 1) // 2
            keys += kv
            continue
        first = max(0, h - window + 1)
        keys += kv - first + min(sinks, first)
        for p in range(h, kv):
            lo = max(0, p - window + 1)
            pairs += p + 1 - lo + min(sinks, lo)
    return pairs, keys


def work(case):
    if case["op"] == "tables":
        _, added = _lengths(case)
        n, b = sum(added), case["requests"]
        pages = -(-n // case["page"])
        return {"bytes": 16 * b + 12 * n + 8 * pages, "flops": 4 * n}
    width = case["q_heads"] * case["dim"]
    kv_width = case["kv_heads"] * case["dim"]
    if case["op"] == "append":
        n = case["tokens"]
        rows = min(n, case["far"])
        return {"bytes": 4 * n * (width + 2 * kv_width) + 12 * n + 4 * case["rot"] * rows,
                "flops": 8 * n * (width + kv_width)}
    held, added = _lengths(case)
    pairs, keys = _pairs(case, held, added)
    n = sum(added)
    if case["op"] == "shared":
        pairs += n * case["prefix"]
        keys += case["prefix"]
    return {"bytes": 4 * n * width + 4 * keys * kv_width, "flops": 4 * pairs * width}


# ------------------------------------------------------------------ the inputs

def _heads(gen, shape, dtype, spread=0.5):
    """Values with a scale for each channel and a few large channels, as keys and values have."""
    dev = gen.device
    x = torch.randn(shape, generator=gen, device=dev, dtype=torch.float32)
    scale = torch.exp(spread * torch.randn(shape[-2:], generator=gen, device=dev))
    large = torch.rand(shape[-2:], generator=gen, device=dev) < 0.01
    return (x * torch.where(large, 4 * scale, scale)).to(dtype)


def _tables(gen, counts, columns, num_pages):
    """One table row for each request, pages in shuffled order; unused entries are -1."""
    dev = gen.device
    c = torch.tensor(counts, device=dev)
    perm = torch.randperm(num_pages, generator=gen, device=dev).to(torch.int32)
    col = torch.arange(columns, device=dev)
    start = torch.cumsum(c, 0) - c
    at = (start[:, None] + col[None, :]).clamp(max=num_pages - 1)
    rows = torch.where(col[None, :] < c[:, None], perm[at], torch.full_like(at, -1).to(torch.int32))
    return rows.contiguous(), perm[int(sum(counts)):].contiguous()


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed * 1000003 + 17)
    s = {"case": case}
    page = case["page"]
    if case["op"] == "tables":
        r = random.Random(seed * 7919 + case["mix"])
        held, added = _lengths(case)
        held = [max(0, h - r.randint(0, page)) for h in held]
        have = [-(-h // page) for h in held]
        columns = -(-(max(held) + max(added) + 2 * page) // page)
        grow = sum(-(-(h + a) // page) - p for h, a, p in zip(held, added, have))
        num_pages = sum(have) + grow + 64
        s["tables"], free = _tables(gen, have, columns, num_pages)
        skip = torch.full((3,), -7, dtype=torch.int32, device=dev)  # entries taken earlier
        s["free"] = torch.cat([skip, free])
        s["taken"] = torch.full((1,), 3, dtype=torch.int32, device=dev)
        s["held"] = torch.tensor(held, dtype=torch.int32, device=dev)
        s["added"] = torch.tensor(added, dtype=torch.int32, device=dev)
        s["num_pages"] = num_pages
        s["rows"] = sum(added) + 8  # a padded batch: rows behind the last token
        if own:
            from kv_cache_compression_cachegen_b200 import torch_api as ta
            s["handle"] = ta.PagedTables(case["requests"], s["rows"], page, num_pages, dev)
        return s

    dtype = getattr(torch, case["dtype"])
    hq, h, d = case["q_heads"], case["kv_heads"], case["dim"]
    if case["op"] == "append":
        n, rot = case["tokens"], case["rot"]
        num_pages = -(-n // page) + 3
        s["qkv"] = _heads(gen, (n, hq + 2 * h, d), dtype)
        s["q_out"] = torch.empty((n, hq, d), dtype=dtype, device=dev)
        s["pool"] = torch.zeros((1, 2, num_pages, page, h, d), dtype=dtype, device=dev)
        s["positions"] = torch.randint(0, case["far"], (n,), generator=gen, device=dev,
                                       dtype=torch.int32)
        s["slots"] = torch.randperm(num_pages * page, generator=gen, device=dev)[:n].contiguous()
        s["weights"] = [None, None]
        if case["norm"]:
            s["weights"] = [(1 + 0.2 * torch.randn(d, generator=gen, device=dev)).to(dtype)
                            for _ in range(2)]
        inv = 10000.0 ** (-torch.arange(0, rot, 2, device=dev, dtype=torch.float64) / rot)
        angle = torch.arange(case["far"], device=dev, dtype=torch.float64)[:, None] * inv
        s["rope"] = torch.cat([angle.cos(), angle.sin()], 1).to(torch.float32).contiguous()
        if own:
            from kv_cache_compression_cachegen_b200 import torch_api as ta
            s["handle"] = ta.PagedAppend((1, h, d), hq, dtype, dev)
        return s

    held, added = _lengths(case)
    kv = [a + b for a, b in zip(held, added)]
    counts = [-(-x // page) for x in kv]
    prefix = case.get("prefix", 0)
    prefix_pages = -(-prefix // page)
    num_pages = sum(counts) + prefix_pages + 2
    columns = max(counts) + 1
    s["tables"], rest = _tables(gen, counts, columns, num_pages)
    s["prefix_table"] = rest[:prefix_pages].contiguous()
    s["pool"] = _heads(gen, (1, 2, num_pages, page, h, d), dtype)
    n = sum(added)
    s["q"] = _heads(gen, (n, hq, d), dtype, 0.2)
    s["out"] = torch.empty((n, hq, d), dtype=dtype, device=dev)
    starts = [0]
    for a in added:
        starts.append(starts[-1] + a)
    s["starts"] = torch.tensor(starts, dtype=torch.int32, device=dev)
    s["lens"] = torch.tensor(kv, dtype=torch.int32, device=dev)
    s["max_q"], s["max_kv"] = max(added), max(kv)
    if own:
        from kv_cache_compression_cachegen_b200 import torch_api as ta
        s["handle"] = ta.PagedAttention((1, h, d), hq, dtype, n, case["requests"], dev)
    return s


# ------------------------------------------------------------- the plain forms

def _plain_tables(s):
    page = s["case"]["page"]
    held, added = s["held"].long(), s["added"].long()
    b, rows = held.numel(), s["rows"]
    dev = held.device
    have = (held + page - 1) // page
    need = (held + added + page - 1) // page - have
    starts = torch.cumsum(added, 0) - added
    ends = starts + added
    first = torch.cumsum(need, 0) - need
    taken = s["taken"].long()
    columns = s["tables"].shape[1]
    # deal the pages: entry i of the free list belongs to the request whose range holds i
    i = torch.arange(s["free"].numel(), device=dev) - taken
    r = torch.searchsorted(first + need, i.clamp(min=0), right=True)
    good = (i >= 0) & (r < b)
    r = r.clamp(max=b - 1)
    col = have[r] + i - first[r]
    table = torch.cat([s["tables"], torch.zeros_like(s["tables"][:, :1])], 1)
    table[r, torch.where(good, col, columns)] = s["free"]
    table = table[:, :columns].contiguous()
    # one slot and position for each new token
    t = torch.arange(rows, device=dev)
    r = torch.searchsorted(ends, t, right=True)
    good = r < b
    r = r.clamp(max=b - 1)
    at = held[r] + t - starts[r]
    slot = table[r, torch.where(good, at // page, 0)].long() * page + at % page
    slots = torch.where(good, slot, torch.full_like(slot, -1))
    positions = torch.where(good, at + s["case"]["base"], torch.full_like(at, -1)).int()
    return {"tables": table, "slots": slots, "positions": positions,
            "lens": (held + added).int(), "starts": torch.cat([starts, ends[-1:]]).int(),
            "taken": (taken + need.sum()).int()}


def _plain_append(s):
    c = s["case"]
    hq, h, rot = c["q_heads"], c["kv_heads"], c["rot"]
    qk = s["qkv"][:, :hq + h].float()
    if c["norm"]:
        qk = qk * torch.rsqrt((qk * qk).mean(-1, keepdim=True) + 1e-6)
        w = torch.cat([s["weights"][0].float().expand(hq, -1), s["weights"][1].float().expand(h, -1)])
        qk = qk * w
    cs = s["rope"][s["positions"].long()][:, None, :]
    cos, sin = cs[..., :rot // 2], cs[..., rot // 2:]
    if c["inter"]:
        a, b = qk[..., 0:rot:2], qk[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = qk[..., :rot // 2], qk[..., rot // 2:rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    qk = torch.cat([turned, qk[..., rot:]], -1).to(s["qkv"].dtype)
    pool = s["pool"].clone()
    rows = pool.view(2, -1, h, c["dim"])
    rows[0, s["slots"]] = qk[:, hq:]
    rows[1, s["slots"]] = s["qkv"][:, hq + h:]
    return {"q": qk[:, :hq].contiguous(), "pool": pool}


def _plain_rows(s):
    """Where each query row stands in a padded batch, and the queries laid out so."""
    starts, n = s["starts"].long(), s["q"].shape[0]
    t = torch.arange(n, device=starts.device)
    r = torch.searchsorted(starts[1:], t, right=True)
    i = t - starts[r]
    q = torch.zeros((starts.numel() - 1, s["max_q"], *s["q"].shape[1:]), device=t.device)
    q[r, i] = s["q"].float()
    return q, r, i


def _plain_scores(q, k):
    """[B, n, Hq, D] x [B, m, H, D] -> [B, H, n * G, m] scaled by 1 / sqrt(D)."""
    b, n, hq, d = q.shape
    h = k.shape[2]
    rows = q.view(b, n, h, hq // h, d).permute(0, 2, 1, 3, 4).reshape(b, h, n * (hq // h), d)
    return (rows / math.sqrt(d)) @ k.permute(0, 2, 3, 1)


def _plain_back(o, r, i, n):
    """[B, H, n * G, D] -> the packed rows [N, Hq, D]."""
    b, h, ng, d = o.shape
    o = o.view(b, h, n, ng // n, d).permute(0, 2, 1, 3, 4).reshape(b, n, -1, d)
    return o[r, i]


def _plain_keys(s):
    """The positions that any row of a request may see, its keys and values, and the mask."""
    c, page = s["case"], s["case"]["page"]
    lens, n = s["lens"].long(), s["starts"].long().diff()
    window, sinks = c.get("window", 0), c.get("sinks", 0)
    dev = lens.device
    if window and window + s["max_q"] + sinks < s["max_kv"]:
        first = (lens - n - window + 1).clamp(min=sinks)
        j = torch.arange(sinks + window + s["max_q"], device=dev)[None, :]
        j = torch.where(j < sinks, j, j - sinks + first[:, None])
    else:
        j = torch.arange(s["max_kv"], device=dev)[None, :].expand(lens.numel(), -1)
    inside = j < lens[:, None]
    at = torch.where(inside, j, torch.zeros_like(j))
    slot = torch.gather(s["tables"].long(), 1, at // page) * page + at % page
    pool = s["pool"].view(2, -1, c["kv_heads"], c["dim"])
    p = (lens - n)[:, None] + torch.arange(s["max_q"], device=dev)[None, :]
    see = inside[:, None, :] & (j[:, None, :] <= p[:, :, None])
    if window:
        see &= (j[:, None, :] > p[:, :, None] - window) | (j[:, None, :] < sinks)
    groups = c["q_heads"] // c["kv_heads"]
    see = see.repeat_interleave(groups, 1)[:, None]  # [B, 1, n * G, m]
    return pool[0, slot].float(), pool[1, slot].float(), see


def _plain_window(s):
    q, r, i = _plain_rows(s)
    k, v, see = _plain_keys(s)
    x = _plain_scores(q, k).masked_fill_(~see, -math.inf)
    m = x.amax(-1, keepdim=True)
    x = torch.exp(x.sub_(torch.where(m > -math.inf, m, torch.zeros_like(m))))
    o = (x @ v.permute(0, 2, 1, 3)) / x.sum(-1, keepdim=True).clamp(min=1e-30)
    return _plain_back(o, r, i, s["max_q"]).to(s["q"].dtype)


def _plain_shared(s):
    c, page = s["case"], s["case"]["page"]
    n, hq = s["q"].shape[:2]
    h, d = c["kv_heads"], c["dim"]
    # the prefix, read once for every row of the batch
    j = torch.arange(c["prefix"], device=s["q"].device)
    slot = s["prefix_table"].long()[j // page] * page + j % page
    pool = s["pool"].view(2, -1, h, d)
    x = _plain_scores(s["q"].float()[None], pool[0, slot].float()[None])
    m1 = x.amax(-1, keepdim=True)
    x = torch.exp(x.sub_(m1))
    l1 = x.sum(-1, keepdim=True)
    o1 = x @ pool[1, slot].float().permute(1, 0, 2)[None]
    o1, m1, l1 = (y.view(h, n, hq // h, -1).permute(1, 0, 2, 3).reshape(n, hq, -1)
                  for y in (o1, m1, l1))
    # each request's own tokens
    q, r, i = _plain_rows(s)
    k, v, see = _plain_keys(s)
    x = _plain_scores(q, k).masked_fill_(~see, -math.inf)
    m2 = x.amax(-1, keepdim=True)
    x = torch.exp(x.sub_(torch.where(m2 > -math.inf, m2, torch.zeros_like(m2))))
    l2 = x.sum(-1, keepdim=True)
    o2, m2, l2 = (_plain_back(y, r, i, s["max_q"]) for y in (x @ v.permute(0, 2, 1, 3), m2, l2))
    # joined by their maxima and sums
    m = torch.maximum(m1, m2)
    a1, a2 = torch.exp(m1 - m), torch.exp(m2 - m)
    return ((o1 * a1 + o2 * a2) / (l1 * a1 + l2 * a2)).to(s["q"].dtype)


# ------------------------------------------------------------- the calls

def _own_tables(s):
    t = s["handle"]
    t.extend(s["held"], s["added"], s["tables"], s["free"], s["taken"],
             position_base=s["case"]["base"])
    return {"tables": s["tables"], "slots": t.slots, "positions": t.positions,
            "lens": t.kv_lens, "starts": t.q_starts, "taken": t.taken}


def _own_append(s):
    c = s["case"]
    hq, h = c["q_heads"], c["kv_heads"]
    qkv = s["qkv"]
    s["handle"].append(qkv[:, :hq], qkv[:, hq:hq + h], qkv[:, hq + h:], s["q_out"], s["pool"], 0,
                       s["positions"], s["slots"], s["rope"], q_weight=s["weights"][0],
                       k_weight=s["weights"][1], eps=1e-6, interleaved=bool(c["inter"]))
    return {"q": s["q_out"], "pool": s["pool"]}


def _own_window(s):
    c = s["case"]
    s["handle"].run(s["q"], s["pool"], 0, s["starts"], s["lens"], s["tables"], s["max_q"],
                    s["out"], window=c["window"], sinks=c["sinks"])
    return s["out"]


def _own_shared(s):
    s["handle"].run_shared(s["q"], s["pool"], 0, s["prefix_table"], s["case"]["prefix"],
                           s["starts"], s["lens"], s["tables"], s["max_q"], s["out"])
    return s["out"]


def run(state):
    op = state["case"]["op"]
    if own:
        call = {"tables": _own_tables, "append": _own_append, "window": _own_window,
                "shared": _own_shared}[op]
    else:
        call = {"tables": _plain_tables, "append": _plain_append, "window": _plain_window,
                "shared": _plain_shared}[op]
    return call(state)


# ------------------------------------------------------------- the definition in 64 bits

def _exact_attend(q, keys, values, see):
    """q [n, Hq, D], keys/values [m, H, D], see [n, m]: softmax attention in 64 bits."""
    n, hq, d = q.shape
    h = keys.shape[1]
    g = hq // h
    out = torch.zeros((n, hq, d), dtype=torch.float64, device=q.device)
    block = max(1, 50_000_000 // keys.shape[0])
    for head in range(hq):
        kk, vv = keys[:, head // g].double(), values[:, head // g].double()
        for a in range(0, n, block):
            x = q[a:a + block, head].double() @ kk.T * (d ** -0.5)
            x = torch.where(see[a:a + block], x, torch.full_like(x, -math.inf))
            out[a:a + block, head] = torch.softmax(x, -1) @ vv
    return out


def exact(case, seed):
    s = prepare(case, seed)
    page = case["page"]
    if case["op"] == "tables":
        return None
    h, d = case["kv_heads"], case["dim"]
    if case["op"] == "append":
        hq, rot, half = case["q_heads"], case["rot"], case["rot"] // 2
        x = s["qkv"].double()
        table = s["rope"].double()[s["positions"].long()]
        out = x.clone()
        for head in range(hq + h):
            y = x[:, head]
            if case["norm"]:
                y = y / (y.square().sum(-1, keepdim=True) / d + 1e-6).sqrt()
                y = y * s["weights"][0 if head < hq else 1].double()
            y = y.clone()
            z = y.clone()
            for i in range(half):
                a, b = (2 * i, 2 * i + 1) if case["inter"] else (i, i + half)
                co, si = table[:, i], table[:, half + i]
                z[:, a] = y[:, a] * co - y[:, b] * si
                z[:, b] = y[:, b] * co + y[:, a] * si
            out[:, head] = z
        pool = s["pool"].double()
        flat = pool.view(2, -1, h, d)
        flat[0].index_copy_(0, s["slots"], out[:, hq:hq + h])
        flat[1].index_copy_(0, s["slots"], out[:, hq + h:])
        return {"q": out[:, :hq], "pool": pool}
    if work(case)["flops"] > 4e12:
        return None
    held, added = _lengths(case)
    pool = s["pool"].view(2, -1, h, d)
    prefix = case.get("prefix", 0)
    dev = s["q"].device
    j = torch.arange(prefix, device=dev)
    head_rows = s["prefix_table"][j // page].long() * page + j % page
    outs, at = [], 0
    for r, (a, n) in enumerate(zip(held, added)):
        j = torch.arange(a + n, device=dev)
        p = torch.arange(a, a + n, device=dev)[:, None]
        see = j[None] <= p
        if case.get("window", 0):
            see = see & ((p - j[None] < case["window"]) | (j[None] < case["sinks"]))
        rows = s["tables"][r][j // page].long() * page + j % page
        keep = see.any(0)
        see, rows = see[:, keep], rows[keep]
        if prefix:
            see = torch.cat([torch.ones((n, prefix), dtype=torch.bool, device=dev), see], 1)
            rows = torch.cat([head_rows, rows])
        outs.append(_exact_attend(s["q"][at:at + n], pool[0, rows], pool[1, rows], see))
        at += n
    return torch.cat(outs)
