"""The operators on several branches of one context as they are measured: the
next batch's pages from the present ones (fork), used pages moved to the pool's
front (compact), attention of sequences that share a prefix, and log
probabilities of given tokens.

`run` takes what `prepare` made and does one pass: in its plain form with
elementary torch operations in 32 bits, or (`own`) with the framework's calls.

The cache: pages of `page` tokens, codes [pages][kv heads][page][d] uint8 (code
+ 128) whose bytes inside a (page, head) stand in fragment order (_k_natural,
_v_natural), and one fp32 scale per (page, head) for keys and values each.
Fork and compact copy these bytes and change none, so the pool itself is what
they return beside the tables: equal bytes and scales are equal values.
"""
import math
import random

import torch

own = False


def listed():
    pages = {"seqs": 8, "rows": 32, "context": 1500, "slots": 9, "hkv": 8, "d": 128, "page": 64, "pool": 1024, "lens": 1}
    heads = {"groups": 1, "members": 4, "new": 1, "prefix": 1000, "tail": 30, "aligned": True, "ragged": True, "loose": 0, "hq": 40,
             "hkv": 8, "d": 128, "page": 64, "window": 0, "sinks": 0, "lens": 1}
    logits = {"rows": 1, "vocab": 124160, "gap": 0, "type": "bf16", "top": 8, "tokens": 1, "scale": 1.0, "kept": 0}
    return [
        # eight requests open four branches each after a verification: nothing but latency
        {**pages, "name": "fork_few", "op": "fork"},
        # beams of many requests, two kv heads a rank: a third of them ends, others branch, new prompts come
        {**pages, "name": "fork_many", "op": "fork", "seqs": 512, "rows": 1024, "context": 4000, "hkv": 2, "page": 32,
         "pool": 60000, "lens": 2},
        # a small pool drawn together
        {**pages, "name": "compact_few", "op": "compact", "seqs": 16, "context": 2000, "pool": 700, "lens": 3},
        # a pool of 1.07 GB, two fifths of it in use at random places, drawn together to give the rest back
        {**pages, "name": "compact_pool", "op": "compact", "seqs": 64, "context": 6000, "pool": 8192, "lens": 4},
        # one request's four drafts, a slot each, short context: latency
        {**heads, "name": "attend_few", "op": "attend"},
        # 64 samples of one long prompt
        {**heads, "name": "attend_samples", "op": "attend", "members": 64, "prefix": 8192, "tail": 500, "lens": 5},
        # four requests, four branches each, nine slots to verify at once; prefixes that end inside a page
        {**heads, "name": "attend_slots", "op": "attend", "groups": 4, "members": 4, "new": 9, "prefix": 20000, "tail": 60,
         "aligned": False, "lens": 6},
        # users' prompts arriving over one system prompt
        {**heads, "name": "attend_prompts", "op": "attend", "members": 16, "new": 200, "prefix": 6000, "tail": 0, "lens": 7},
        # large heads, few of keys, a window and four first tokens; two sequences of their own beside the groups
        {**heads, "name": "attend_window", "op": "attend", "groups": 2, "members": 12, "new": 4, "prefix": 9000, "tail": 300, "hq": 16,
         "hkv": 2, "d": 256, "page": 128, "window": 2048, "sinks": 4, "loose": 2, "lens": 8},
        # the drafted token's log probability: latency
        {**logits, "name": "logprobs_one", "op": "logprobs"},
        # the draft slots of eight requests, from rows that hold the reranked tokens alone
        {**logits, "name": "logprobs_slots", "op": "logprobs", "rows": 72, "scale": 1.25, "kept": 32},
        # a prompt's tokens scored
        {**logits, "name": "logprobs_score", "op": "logprobs", "rows": 2048, "top": 20},
    ]


def draw(rng):
    most = {}
    for c in listed():
        w, m = work(c), most.setdefault(c["op"], [0, 0])
        m[0], m[1] = max(m[0], w["bytes"]), max(m[1], w["flops"])

    def log(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    while True:
        op = rng.choice(["fork", "compact", "attend", "attend", "attend", "logprobs", "logprobs"])
        c = {"op": op, "lens": rng.randrange(1 << 20)}
        if op == "logprobs":
            c.update(rows=log(1, 4096), vocab=log(500, 250000), gap=rng.choice([0, 0, 1, 40]), type=rng.choice(["bf16", "bf16", "fp32"]),
                     top=rng.choice([1, 5, 8, 20, 64]), tokens=rng.choice([1, 1, 3, 8]), scale=rng.choice([1.0, 0.7, 1.6]),
                     kept=rng.choice([0, 0, 40]))
        elif op == "attend":
            hkv, group = rng.choice([(8, 5), (8, 4), (16, 1), (2, 8), (1, 8), (4, 7), (3, 3)])
            c.update(groups=log(1, 12), members=log(1, 64), new=rng.choice([1, 1, rng.randint(2, 12), log(13, 300)]), prefix=log(1, 40000),
                     tail=log(1, 1500), aligned=rng.random() < 0.5, ragged=True, loose=rng.choice([0, 0, 3]), hq=hkv * group, hkv=hkv,
                     d=rng.choice([64, 128, 128, 256]), page=rng.choice([32, 64, 64, 128, 256]), window=0, sinks=0)
            if rng.random() < 0.3:
                c["window"], c["sinks"] = log(64, 8192), rng.choice([0, 1, 4, 64])
        else:
            c.update(seqs=log(1, 600), rows=log(1, 1200), context=log(1, 8000), slots=rng.randint(1, 16), hkv=rng.choice([1, 2, 3, 8]),
                     d=rng.choice([64, 128, 256]), page=rng.choice([32, 64, 128, 256]), pool=0)
            c["pool"] = int(_pages_asked(c) * rng.uniform(1.02, 2.5)) + 1
            if c["pool"] * c["hkv"] * c["page"] * c["d"] * 2 > 1.1e9:
                continue
        w, m = work(c), most[op]
        if w["bytes"] > m[0] or w["flops"] > max(m[1], 1):
            continue
        if op == "attend":
            p = _spans(c)
            rows = max(p["group_rows"]) * len(p["group_rows"]) * c["hq"]
            if rows * p["near_a"] * c["page"] > 7e8 or len(p["lens"]) * p["near_b"] * c["page"] * c["hkv"] * c["d"] > 9e8:
                continue
            if len(p["lens"]) * c["hq"] * c["new"] * p["near_b"] * c["page"] > 7e8 or len(p["group_rows"]) * p["near_a"] * c["page"] * c["hkv"] * c["d"] > 9e8:
                continue
        return c


# ------------------------------------------------------------------ sizes
def _lens(c):
    """attend: per sequence (group or -1, new tokens, prefix, tokens in the cache)."""
    r, got = random.Random(c["lens"]), []
    for g in range(c["groups"]):
        prefix = int(c["prefix"] * r.uniform(0.5, 1.0)) if c["ragged"] and c["groups"] > 1 else c["prefix"]
        if c["aligned"]:
            prefix = max(c["page"], prefix // c["page"] * c["page"])
        members = max(1, int(c["members"] * r.uniform(0.5, 1.0))) if c["ragged"] and c["groups"] > 1 else c["members"]
        for i in range(members):
            n = max(1, int(c["new"] * r.uniform(0.3, 1.0))) if c["ragged"] and c["new"] > 1 else c["new"]
            if i == 5:          # a branch without new tokens
                n = 0
            got.append((g, n, prefix, prefix + int(c["tail"] * (r.uniform(0.2, 1.0) if c["ragged"] else 1.0)) + n))
    for _ in range(c["loose"]):
        got.append((-1, c["new"], 0, c["new"] + int(c["prefix"] * r.uniform(0.2, 0.6))))
    return got


def _spans(c):
    """attend: what the plain form's padded arrays take: first page and pages of each group's prefix and of each sequence's own tokens."""
    lens, w, page = _lens(c), c["window"], c["page"]
    p = {"lens": lens, "group_rows": [], "low_a": [], "low_b": [], "near_a": 1, "near_b": 1}
    for g in range(c["groups"]):
        own_ = [x for x in lens if x[0] == g]
        p["group_rows"].append(max(1, sum(x[1] for x in own_)))
        begin = min(x[3] - x[1] for x in own_)
        low = max(0, begin - w + 1) // page if w else 0
        p["low_a"].append(low)
        p["near_a"] = max(p["near_a"], -(-own_[0][2] // page) - low)
    for _, n, prefix, length in lens:
        low = max(prefix, length - n - w + 1 if w else 0) // page
        p["low_b"].append(low)
        p["near_b"] = max(p["near_b"], -(-length // page) - low)
    return p


def _seen(c):
    """attend: (row, visible token) pairs of one query head; tokens that some row sees, a shared one once."""
    pairs, tokens, w, k = 0, 0, c["window"], c["sinks"]
    low_of = {}
    for g, n, prefix, length in _lens(c):
        for p in range(length - n, length):
            low = max(0, p - w + 1) if w else 0
            pairs += p + 1 - low + min(k, low)
        if not n:
            continue
        low = max(0, length - n - w + 1) if w else 0
        tokens += length - max(low, prefix) + max(0, min(k, low) - prefix)
        if g >= 0:
            low_of[g] = (prefix, min(low, low_of.get(g, (0, low))[1]))
    for prefix, low in low_of.values():
        tokens += max(0, prefix - low) + min(k, low, prefix)
    return pairs, tokens


def _present(c):
    """fork: per present sequence (tokens, pages held); parents and positions needed of the next rows.  compact: the first of these."""
    r = random.Random(c["lens"])
    page = c["page"]
    seqs = [int(c["context"] * r.uniform(0.3, 1.0)) for _ in range(c["seqs"])]
    held = [(n, -(-(n + c["slots"]) // page)) for n in seqs]
    parents = sorted(r.randrange(c["seqs"]) for _ in range(c["rows"]))
    need = []
    for i, p in enumerate(parents):
        if c["rows"] >= 20 and i >= c["rows"] - c["rows"] // 20:      # new prompts
            parents[i] = -1
            need.append(max(1, c["context"] // 2))
        else:
            need.append(seqs[p] + c["slots"])
    return held, parents, need


def _shared(held, i, page):
    """Pages that sequence i has from the one before it: half the full ones of every second sequence's neighbour."""
    return min(held[i][0], held[i - 1][0]) // page // 2 if i % 2 else 0


def _asked(c):
    """fork: (pages in use, pages taken, pages copied)."""
    held, parents, need = _present(c)
    page, seen, taken, copied = c["page"], set(), 0, 0
    for p, n in zip(parents, need):
        length, has = held[p] if p >= 0 else (0, 0)
        full, last = length // page, -(-max(n, length) // page)
        kept = max(0, min(has, last) - full) if p >= 0 and p not in seen else 0
        taken += last - full - kept
        copied += p >= 0 and p in seen and length % page > 0
        seen.add(p)
    return sum(h[1] - _shared(held, i, page) for i, h in enumerate(held)), taken, copied


def _pages_asked(c):
    used, taken, _ = _asked(c)
    return used + taken


def work(c):
    if c["op"] == "logprobs":
        n = c["rows"] * c["vocab"]
        return {"bytes": n * (2.0 if c["type"] == "bf16" else 4.0) + c["rows"] * (8.0 * c["tokens"] + 8.0 * c["top"] + 8.0), "flops": 6.0 * n}
    if c["op"] == "attend":
        pairs, tokens = _seen(c)
        rows = sum(x[1] for x in _lens(c))
        return {"bytes": rows * c["hq"] * (4.0 * c["d"] + 4) + tokens * c["hkv"] * (2.0 * c["d"] + 8.0 / c["page"]),
                "flops": 4.0 * c["d"] * c["hq"] * pairs}
    page_bytes = c["hkv"] * (2 * c["page"] * c["d"] + 8)
    held, _, need = _present(c)
    used, _, copied = _asked(c)
    if c["op"] == "compact":
        moved = used * (1 - used / c["pool"])
        return {"bytes": 2.0 * moved * page_bytes + 8.0 * c["pool"] + 8.0 * sum(h[1] for h in held), "flops": 1.0 * c["pool"]}
    return {"bytes": 2.0 * copied * page_bytes + 8.0 * c["pool"] + 4.0 * (sum(h[1] for h in held) + sum(-(-n // c["page"]) for n in need)),
            "flops": 1.0 * c["pool"]}


# ------------------------------------------------------------------ inputs
def prepare(c, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))
    if c["op"] == "logprobs":
        return _prepare_logits(c, gen, dev)
    return _prepare_attend(c, gen, dev) if c["op"] == "attend" else _prepare_pages(c, gen, dev)


def _prepare_logits(c, gen, dev):
    m, n = c["rows"], c["vocab"]
    x = torch.empty((m, n + c["gap"]), dtype=torch.bfloat16 if c["type"] == "bf16" else torch.float32, device=dev)
    for i in range(0, m, 256):
        part = torch.randn((min(256, m - i), n + c["gap"]), generator=gen, device=dev) * 2.0
        few = torch.randint(0, n, (part.shape[0], 12), generator=gen, device=dev)      # a few likely tokens
        part.scatter_add_(1, few, torch.rand(few.shape, generator=gen, device=dev) * 14.0)
        if c["kept"]:      # a row for a top-k caller: the reranked tokens, -inf elsewhere
            kept = torch.zeros_like(part, dtype=torch.bool).scatter_(1, part[:, :n].topk(min(c["kept"], n), dim=1).indices, True)
            part.masked_fill_(~kept, -math.inf)
        x[i:i + 256] = part.to(x.dtype)
    tokens = torch.randint(0, n, (m, c["tokens"]), generator=gen, device=dev)
    tokens[:, 0] = torch.where(torch.rand(m, generator=gen, device=dev) < 0.7, x[:, :n].argmax(1), tokens[:, 0])    # mostly the likeliest
    if c["tokens"] > 2:
        tokens[:, 2] = n + 17      # another shard's
    return {"case": dict(c), "logits": x[:, :n], "tokens": tokens.to(torch.int32)}


def _codes(shape, gen, dev):
    codes = torch.empty(shape, dtype=torch.uint8, device=dev)
    step = max(1, (1 << 26) // (shape[1] * shape[2] * shape[3]))
    for i in range(0, shape[0], step):   # as a block's largest value of about 3.8 deviations leaves them
        codes[i:i + step] = (torch.randn(codes[i:i + step].shape, generator=gen, device=dev) * 33.0).round_().clamp_(-127, 127).add_(128)
    return codes


def _pool(c, n_pages, gen, dev):
    shape = (n_pages, c["hkv"], c["page"], c["d"])
    return {"k_codes": _codes(shape, gen, dev), "v_codes": _codes(shape, gen, dev),
            "k_scale": torch.rand(shape[:2], generator=gen, device=dev) * 0.02 + 0.02,
            "v_scale": torch.rand(shape[:2], generator=gen, device=dev) * 0.02 + 0.02}


def _prepare_attend(c, gen, dev):
    spans = _spans(c)
    lens, page = spans["lens"], c["page"]
    most = max(-(-x[3] // page) for x in lens)
    leads = [x[0] < 0 or x[0] != y[0] for x, y in zip(lens, [(-1,)] + lens)]      # its prefix's pages are its own
    total = sum(-(-x[3] // page) - (0 if lead else x[2] // page) for x, lead in zip(lens, leads))
    order = torch.randperm(total, generator=gen, device=dev).to(torch.int32).cpu()
    table, at, starts, groups, prefixes = torch.full((len(lens), max(1, most)), -1, dtype=torch.int32), 0, [0], [0], []
    for s, (g, n, prefix, length) in enumerate(lens):
        shared = 0
        if leads[s]:
            first = s
            if g >= 0:
                groups.append(s)
                prefixes.append(prefix)
        else:
            shared = prefix // page
            table[s, :shared] = table[first, :shared]
        if g >= 0:
            groups[g + 1] = s + 1
        own_ = -(-length // page) - shared
        table[s, shared:shared + own_] = order[at:at + own_]
        at += own_
        starts.append(starts[-1] + n)
    rows = starts[-1]
    q = torch.randn((rows, c["hq"], c["d"]), generator=gen, device=dev)
    q[:, :, torch.randperm(c["d"], generator=gen, device=dev)[:max(1, c["d"] // 100)]] *= 4.0      # a few channels with large values
    ints = {"q_start": starts, "kv_len": [x[3] for x in lens], "group_start": groups, "prefix_len": prefixes, "low_a": spans["low_a"],
            "low_b": spans["low_b"]}
    return {"case": dict(c), "rows": rows, "workspace": None, "table": table.to(dev), "q": q.to(torch.bfloat16),
            "near_a": spans["near_a"], "near_b": spans["near_b"], "group_rows": max(spans["group_rows"]), "new": max(x[1] for x in lens),
            **{k: torch.tensor(v, dtype=torch.int32, device=dev) for k, v in ints.items()}, **_pool(c, total, gen, dev)}


def _prepare_pages(c, gen, dev):
    held, parents, need = _present(c)
    page, n_pages = c["page"], c["pool"]
    order = torch.randperm(n_pages, generator=gen, device=dev).to(torch.int32).cpu()
    wide = max(max(h[1] for h in held), max(-(-n // page) for n in need))
    table, at = torch.full((len(held), wide), -1, dtype=torch.int32), 0
    for i, (_, has) in enumerate(held):
        shared = _shared(held, i, page)
        table[i, :shared] = table[i - 1, :shared]
        table[i, shared:has] = order[at:at + has - shared]
        at += has - shared
    uses = torch.bincount(table[table >= 0].long(), minlength=n_pages).to(torch.int32)
    return {"case": dict(c), "workspace": None, "table": table.to(dev), "uses": uses.to(dev), "kv_len": torch.tensor([h[0] for h in held], dtype=torch.int32, device=dev),
            "parents": torch.tensor(parents, dtype=torch.int32, device=dev), "need": torch.tensor(need, dtype=torch.int32, device=dev),
            **_pool(c, n_pages, gen, dev)}


# ------------------------------------------------------------------ one pass
def run(s):
    c = s["case"]
    if not own:
        return {"fork": _fork, "compact": _compact, "attend": _attend, "logprobs": _logprobs}[c["op"]](s, c)
    import bit_quantized_lm_amd as lib
    if c["op"] == "logprobs":
        return lib.draft_branch_logprobs(s["logits"], s["tokens"], top=c["top"], scale=c["scale"])
    cache = (s["k_codes"], s["v_codes"], s["k_scale"], s["v_scale"])
    if c["op"] == "attend":
        if s["workspace"] is None:
            s["workspace"] = lib.draft_branch_attend_workspace(s["rows"], s["kv_len"].shape[0], c["hq"], c["hkv"], c["d"], s["q"].device)
        return lib.draft_branch_attend(s["q"], *cache, s["q_start"], s["kv_len"], s["table"], s["group_start"], s["prefix_len"],
                                       window=c["window"], sinks=c["sinks"], workspace=s["workspace"])
    if s["workspace"] is None:
        s["workspace"] = lib.draft_branch_pages_workspace(c["pool"], c["rows"], s["table"].device)
    if c["op"] == "fork":
        got = lib.draft_branch_fork(*cache, s["uses"], s["table"], s["kv_len"], s["parents"], s["need"], workspace=s["workspace"])
    else:
        got = lib.draft_branch_compact(*cache, s["uses"], s["table"], workspace=s["workspace"])
    return (*got, *cache)


# ------------------------------------------------------------------ the plain forms
def _count(table, n_pages):
    """Table entries that name each page."""
    held = (table >= 0) & (table < n_pages)
    at = torch.where(held, table, n_pages).reshape(-1)
    return torch.zeros(n_pages + 1, dtype=torch.int64, device=table.device).index_add_(0, at, torch.ones_like(at))[:n_pages]


def _fork(s, c):
    table, uses, page = s["table"].long(), s["uses"].long(), c["page"]
    n_seq, wide = table.shape
    n_pages, parents, dev = uses.shape[0], s["parents"].long(), table.device
    row, j = torch.arange(parents.shape[0], device=dev), torch.arange(wide, device=dev)[None, :]
    child = (parents >= 0) & (parents < n_seq)
    p = parents.clamp(0, n_seq - 1)
    length = torch.where(child, s["kv_len"].long()[p].clamp(0, wide * page), 0)
    old = torch.where(child[:, None], table[p], -1)
    held = (old >= 0) & (old < n_pages)
    full = (length // page)[:, None]
    last = (torch.maximum(s["need"].long(), length).clamp(max=wide * page) + page - 1).div(page, rounding_mode="floor")[:, None]
    first = torch.full((n_seq,), len(row), device=dev).scatter_reduce_(0, p, torch.where(child, row, len(row)), "amin")
    eldest = child & (first[p] == row)
    kept = (j >= full) & (j < last) & held & eldest[:, None] & (uses[old.clamp(0, n_pages - 1)] == 1)
    fresh = (j >= full) & (j < last) & ~kept
    free = uses <= 0
    ids = torch.full((n_pages + 1,), -1, device=dev)
    ids[torch.where(free, torch.cumsum(free, 0) - 1, n_pages)] = torch.arange(n_pages, device=dev)
    taken = ids[(torch.cumsum(fresh.reshape(-1), 0) - 1).clamp(0, n_pages - 1)].reshape(fresh.shape)
    short = fresh.sum() - free.sum()
    new = torch.where((j < full) & held | kept, old, torch.where(fresh, taken, -1))
    new = torch.where(short > 0, torch.full_like(new, -1), new)
    after = torch.where(short > 0, uses, uses - _count(table, n_pages) + _count(new, n_pages))
    part = full[:, 0].clamp(max=wide - 1)[:, None]
    copied = ((length % page > 0) & (short <= 0))[:, None] & fresh.gather(1, part) & held.gather(1, part)
    src, dst = old.gather(1, part)[copied], new.gather(1, part)[copied]
    for x in (s["k_codes"], s["v_codes"], s["k_scale"], s["v_scale"]):
        x[dst] = x[src]
    status = torch.stack([(after <= 0).sum(), short.clamp(min=0)])
    return (new.to(torch.int32), after.to(torch.int32), status.to(torch.int32), s["k_codes"], s["v_codes"], s["k_scale"], s["v_scale"])


def _compact(s, c):
    table, uses = s["table"].long(), s["uses"]
    n_pages = uses.shape[0]
    at = torch.arange(n_pages, device=uses.device)
    taken = uses > 0
    used = taken.sum()
    src, dst = torch.nonzero(taken & (at >= used))[:, 0], torch.nonzero(~taken & (at < used))[:, 0]
    for x in (s["k_codes"], s["v_codes"], s["k_scale"], s["v_scale"]):
        x[dst] = x[src]
    to = at.clone()
    to[src] = dst
    held = (table >= 0) & (table < n_pages)
    after = uses.clone()
    after[dst], after[src] = uses[src], 0
    status = torch.stack([used, torch.tensor(src.shape[0], device=used.device)])
    return (torch.where(held, to[table.clamp(0, n_pages - 1)], table).to(torch.int32), after, status.to(torch.int32), s["k_codes"], s["v_codes"],
            s["k_scale"], s["v_scale"])


def _logprobs(s, c):
    x, tokens, k = s["logits"], s["tokens"].long(), c["top"]
    n = x.shape[1]
    z = x.float() * c["scale"]
    top = z.amax(1, keepdim=True)
    base = torch.where(top == -math.inf, torch.zeros_like(top), top)
    e = torch.exp(z - base)
    total = e.sum(1, keepdim=True)
    lse = base + torch.log(total)
    entropy = (torch.log(total) + torch.where(e > 0, e * (base - z), torch.zeros_like(e)).sum(1, keepdim=True) / total)[:, 0]
    here = (tokens >= 0) & (tokens < n)
    logprob = torch.where(here, z.gather(1, tokens.clamp(0, n - 1)) - base - torch.log(total), torch.full_like(lse, -math.inf))
    # the best by (value, lowest index): one whole number each
    bits = x.float().view(torch.int32).long()
    order = torch.where(bits < 0, (-(1 << 31)) - 1 - bits, bits)
    key = order * (1 << 32) + ((1 << 32) - 1 - torch.arange(n, device=x.device))
    best = key.topk(min(k, n), dim=1).indices
    value = z.gather(1, best) - base - torch.log(total)
    some = x.gather(1, best) > -math.inf
    return (logprob, torch.where(some, best, -1).to(torch.int32), torch.where(some, value, torch.full_like(value, -math.inf)), lse[:, 0], entropy)


def _k_natural(codes):
    """[..., page, d] key codes in fragment order -> [..., page, d]."""
    *lead, page, d = codes.shape
    n = len(lead)
    x = codes.reshape(*lead, page // 32, 2, d // 64, 4, 16, 16)        # group, half, 64 d, 16 d, token, d
    return x.permute(*range(n), n, n + 1, n + 4, n + 2, n + 3, n + 5).reshape(*lead, page, d)


def _v_natural(codes):
    """[..., page, d] value codes in fragment order -> [..., page, d]."""
    *lead, page, d = codes.shape
    n = len(lead)
    x = codes.reshape(*lead, page // 32, d // 32, 4, 16, 2, 2, 4)      # group, 32 d, four tokens, d, 16 d, half, token
    return x.permute(*range(n), n, n + 5, n + 2, n + 6, n + 1, n + 4, n + 3).reshape(*lead, page, d)


def _values(codes, scale, natural, ids):
    """fp32 [B][heads][tokens][d] of the pages `ids` [B][P]."""
    x = (natural(codes[ids]).float() - 128.0) * scale[ids][..., None, None]      # [B][P][heads][page][d]
    n_b, n_p, heads, page, d = x.shape
    return x.transpose(1, 2).reshape(n_b, heads, n_p * page, d)


def _part(s, c, table, row0, rows, most, lo, hi, low, near, at):
    """Attention of up to `most` rows from row0 [B] on over the tokens lo..hi-1 of the pages that `table` [B] names: `near` pages from low on,
    and the first tokens'.  Gives every row's (largest score, sum, value sums): fp32 [B][most][hq](...)."""
    dev, hkv, d, page, w, sinks = s["q"].device, c["hkv"], c["d"], c["page"], c["window"], c["sinks"]
    group, n_b, wide = c["hq"] // hkv, table.shape[0], table.shape[1]
    first = min(wide, -(-sinks // page)) if w else 0
    index = torch.cat([torch.arange(first, device=dev)[None, :].expand(n_b, first), low[:, None] + torch.arange(near, device=dev)[None, :]], 1)
    fresh = torch.cat([torch.arange(first, device=dev)[None, :] < low[:, None], index[:, first:] < wide], 1)
    ids = table.gather(1, index.clamp(max=wide - 1)).clamp(min=0)
    j = (index[:, :, None] * page + torch.arange(page, device=dev)).reshape(n_b, 1, -1)
    fresh = fresh[:, :, None].expand(-1, -1, page).reshape(n_b, 1, -1)
    k, v = _values(s["k_codes"], s["k_scale"], _k_natural, ids), _values(s["v_codes"], s["v_scale"], _v_natural, ids)
    i = torch.arange(most, device=dev)
    pad = (row0[:, None] + i).clamp(max=s["rows"] - 1)
    x = s["q"][pad].float().reshape(n_b, most, hkv, group, d).permute(0, 2, 1, 3, 4).reshape(n_b, hkv, most * group, d)
    scores = torch.matmul(x, k.transpose(2, 3)) * (1.0 / math.sqrt(d))
    p = at[pad][:, :, None]
    seen = (j <= p) & (j >= lo[:, None, None]) & (j < hi[:, None, None]) & fresh & (i[None, :, None] < rows[:, None, None])
    if w:
        seen &= (j > p - w) | (j < sinks)
    scores = scores.reshape(n_b, hkv, most, group, -1).masked_fill(~seen[:, None, :, None, :], -math.inf).reshape(scores.shape)
    top = scores.amax(-1, keepdim=True)
    e = torch.exp(scores - torch.where(top == -math.inf, torch.zeros_like(top), top))
    o = torch.matmul(e, v)

    def by_row(y):
        return y.reshape(n_b, hkv, most, group, -1).permute(0, 2, 1, 3, 4).reshape(n_b, most, c["hq"], -1)

    return by_row(top), by_row(e.sum(-1, keepdim=True)), by_row(o)


def _attend(s, c):
    """Each group's rows over the prefix's pages, each sequence's over its own, joined."""
    dev, table = s["q"].device, s["table"].long()
    start, kv_len, groups, prefix = (s[x].long() for x in ("q_start", "kv_len", "group_start", "prefix_len"))
    n_s = kv_len.shape[0]
    row = torch.arange(s["rows"], device=dev)
    seq = torch.searchsorted(start, row, right=True) - 1
    at = kv_len[seq] - start[seq + 1] + row
    group_of = torch.searchsorted(groups, torch.arange(n_s, device=dev), right=True) - 1
    grouped = group_of < prefix.shape[0]
    group_of = group_of.clamp(max=prefix.shape[0] - 1)
    own_from = torch.where(grouped, prefix[group_of], 0)
    row0 = start[groups]
    a = _part(s, c, table[groups[:-1]], row0[:-1], row0[1:] - row0[:-1], s["group_rows"], torch.zeros_like(prefix), prefix, s["low_a"].long(), s["near_a"], at)
    b = _part(s, c, table, start[:-1], start[1:] - start[:-1], s["new"], own_from, kv_len, s["low_b"].long(), s["near_b"], at)
    g = group_of[seq]
    inside = (row - row0[g]).clamp(max=s["group_rows"] - 1)
    (ta, la, oa), (tb, lb, ob) = (x[g, inside] for x in a), (x[seq, row - start[seq]] for x in b)
    ta = torch.where(grouped[seq][:, None, None], ta, torch.full_like(ta, -math.inf))
    top = torch.maximum(ta, tb)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    wa, wb = torch.exp(ta - top), torch.exp(tb - top)
    total = la * wa + lb * wb
    out = (oa * wa + ob * wb) / torch.where(total == 0, torch.ones_like(total), total)
    return out.to(torch.bfloat16), (top + torch.log(total))[:, :, 0]


# ------------------------------------------------------------------ the definition in 64 bits
def exact(c, seed):
    return {"fork": _exact_fork, "compact": _exact_compact, "attend": _exact_attend, "logprobs": _exact_logprobs}[c["op"]](prepare(c, seed), c)


def _exact_fork(s, c):
    page, dev = c["page"], s["table"].device
    table, uses = s["table"].tolist(), s["uses"].tolist()
    lens, parents, need = s["kv_len"].tolist(), s["parents"].tolist(), s["need"].tolist()
    free = [i for i, u in enumerate(uses) if u == 0]
    seen, new, copies, at = set(), [], [], 0
    for p, n in zip(parents, need):
        length, old = (lens[p], table[p]) if p >= 0 else (0, [])
        line = old[:length // page]
        for j in range(length // page, -(-max(n, length) // page)):
            has = old[j] if j < len(old) else -1
            if p not in seen and has >= 0 and uses[has] == 1:
                line.append(has)
                continue
            line.append(free[at])
            at += 1
            if j * page < length:
                copies.append((has, line[-1]))
        seen.add(p)
        new.append(line + [-1] * (len(table[0]) - len(line)))
    after = [0] * len(uses)
    for line in new:
        for i in line:
            if i >= 0:
                after[i] += 1
    for a, b in copies:
        for x in (s["k_codes"], s["v_codes"], s["k_scale"], s["v_scale"]):
            x[b].copy_(x[a])
    whole = [torch.tensor(x, dtype=torch.int32, device=dev) for x in (new, after, [after.count(0), 0])]
    return (*whole, s["k_codes"], s["v_codes"], s["k_scale"], s["v_scale"])


def _exact_compact(s, c):
    table, uses, dev = s["table"].tolist(), s["uses"].tolist(), s["table"].device
    used = sum(u > 0 for u in uses)
    holes = iter([i for i in range(used) if uses[i] == 0])
    to = {i: next(holes) for i in range(used, len(uses)) if uses[i] > 0}
    if to:
        src, dst = (torch.tensor(list(x), device=dev) for x in (to.keys(), to.values()))
        for x in (s["k_codes"], s["v_codes"], s["k_scale"], s["v_scale"]):
            x.index_copy_(0, dst, x.index_select(0, src))
    for a, b in to.items():
        uses[b], uses[a] = uses[a], 0
    whole = [torch.tensor(x, dtype=torch.int32, device=dev) for x in ([[to.get(i, i) for i in line] for line in table], uses, [used, len(to)])]
    return (*whole, s["k_codes"], s["v_codes"], s["k_scale"], s["v_scale"])


def _exact_logprobs(s, c):
    m, n, k = c["rows"], c["vocab"], c["top"]
    got = [[] for _ in range(5)]
    for i in range(0, m, 64):
        x, tokens = s["logits"][i:i + 64], s["tokens"][i:i + 64].long()
        lp = torch.log_softmax(x.double() * c["scale"], 1)
        here = (tokens >= 0) & (tokens < n)
        got[0].append(lp.gather(1, tokens.clamp(0, n - 1)).masked_fill(~here, -math.inf))
        value, at = torch.sort(x.float(), dim=1, descending=True, stable=True)
        some = value[:, :k] > -math.inf
        got[1].append(torch.where(some, at[:, :k], -1).to(torch.int32))
        got[2].append(torch.where(some, lp.gather(1, at[:, :k]), -math.inf))
        got[3].append(torch.logsumexp(x.double() * c["scale"], 1))
        got[4].append(-torch.where(lp > -math.inf, lp.exp() * lp, 0.0).sum(1))
    return [torch.cat(x) for x in got]


def _exact_attend(s, c):
    lens, page, hkv, hq, d, w = _lens(c), c["page"], c["hkv"], c["hq"], c["d"], c["window"]
    dev, table = s["q"].device, s["table"].tolist()
    t, e = torch.arange(page, device=dev)[:, None], torch.arange(d, device=dev)[None, :]
    u = t % 32
    place = {   # byte of token t, element e inside a (page, head), as the layout is documented
        "k": t // 32 * 32 * d + ((u // 16 * (d // 64) + e // 64) * 64 + e % 64 // 16 * 16 + u % 16) * 16 + e % 16,
        "v": t // 32 * 32 * d + ((e // 32 * 4 + u % 16 // 4) * 16 + e % 16) * 16 + e % 32 // 16 * 8 + u // 16 * 4 + u % 4,
    }

    def cached(which, ids, head):
        """Values of the pages' tokens."""
        raw = s[which + "_codes"][ids, head].reshape(len(ids), -1)[:, place[which].reshape(-1)].double().reshape(len(ids), page, d) - 128
        return (raw * s[which + "_scale"][ids, head].double()[:, None, None]).reshape(-1, d)

    out = torch.zeros((s["rows"], hq, d), dtype=torch.float64, device=dev)
    lse = torch.full((s["rows"], hq), -math.inf, dtype=torch.float64, device=dev)
    row, first, group = 0, {}, hq // hkv
    for i, (g, n, prefix, length) in enumerate(lens):
        leader = first.setdefault(g, i) if g >= 0 else i
        if not n:
            continue
        p = torch.arange(length - n, length, device=dev)[:, None]
        j = torch.arange(length, device=dev)
        hidden = j > p
        if w:
            hidden = hidden | ((j <= p - w) & (j >= c["sinks"]))
        some = (~hidden).any(0)
        r = slice(row, row + n)
        for h in range(hkv):
            mine = table[i][:-(-length // page)]
            a, b = table[leader][:-(-prefix // page)], mine[prefix // page:]
            k, v = (torch.cat([cached(x, a, h)[:prefix] if a else torch.zeros((0, d), dtype=torch.float64, device=dev),
                               cached(x, b, h)[prefix % page:length - prefix // page * page]])[some] for x in "kv")
            q = s["q"][r, h * group:(h + 1) * group].double()
            z = (q.transpose(0, 1) @ k.T) / math.sqrt(d)
            z = z.masked_fill(hidden[:, some][None], -math.inf)
            lse[r, h * group:(h + 1) * group] = torch.logsumexp(z, 2).T
            out[r, h * group:(h + 1) * group] = (torch.softmax(z, 2) @ v).transpose(0, 1)
        row += n
    return [out, lse]
