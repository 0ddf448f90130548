"""The draft layer's operators as they are measured: the rotary append to the
8-bit cache, its reading back, and the attention over it.

`run` takes what `prepare` made and does one pass: in its plain form with
elementary torch operations in 32 bits, or (`own`) with the framework's calls.

The cache: pages of `page` tokens, codes [pages][kv heads][page][d] uint8 (code
+ 128) whose bytes inside a (page, head) stand in fragment order (_k_natural,
_v_natural), and one fp32 scale per (page, head) for keys and values each.
A batch: q_start [S+1] and kv_len [S] (the new tokens included), page table.
"""
import math
import random

import torch

own = False

FLOOR = 2.0 ** -40          # smallest scale


def listed():
    base = {"seqs": 1, "new": 1, "context": 0, "ragged": False, "hq": 40, "hkv": 8, "d": 128, "page": 64, "rot": 128,
            "interleaved": False, "window": 0, "sinks": 0, "lens": 1}
    return [
        # one draft slot of one request: nothing but latency
        {**base, "name": "append_one", "op": "append", "context": 777},
        # the draft slots of eight requests (72 rows), part of the head rotated in pairs
        {**base, "name": "append_slots", "op": "append", "seqs": 8, "new": 9, "context": 4000, "ragged": True, "rot": 64,
         "interleaved": True, "lens": 2},
        # prompts of four requests arriving together
        {**base, "name": "append_prompt", "op": "append", "seqs": 4, "new": 6000, "context": 100, "ragged": True, "lens": 3},
        # a short prefix handed to code that wants bf16
        {**base, "name": "read_short", "op": "read", "new": 500},
        # eight long contexts read back whole
        {**base, "name": "read_long", "op": "read", "seqs": 8, "new": 16000, "ragged": True, "lens": 4},
        # one slot over a short context: latency
        {**base, "name": "attend_one", "op": "attend", "context": 1000},
        # one slot over a long context: one request alone has to fill the card
        {**base, "name": "attend_long", "op": "attend", "context": 131071},
        # the draft slots of eight requests
        {**base, "name": "attend_slots", "op": "attend", "seqs": 8, "new": 9, "context": 6000, "ragged": True, "lens": 5},
        # a full batch, one slot each, lengths mixed
        {**base, "name": "attend_batch", "op": "attend", "seqs": 64, "context": 12000, "ragged": True, "lens": 6},
        # long contexts seen through a window with four first tokens kept; small heads, none shared
        {**base, "name": "attend_window", "op": "attend", "seqs": 32, "context": 32000, "hq": 16, "hkv": 16, "d": 64, "rot": 64,
         "page": 32, "window": 4096, "sinks": 4, "ragged": True, "lens": 7},
        # a whole prompt
        {**base, "name": "attend_prompt", "op": "attend", "new": 4096},
        # pieces of two long prompts, windowed; large heads, few of keys
        {**base, "name": "attend_chunk", "op": "attend", "seqs": 2, "new": 1500, "context": 9000, "hq": 16, "hkv": 2, "d": 256,
         "rot": 256, "page": 128, "window": 2048, "sinks": 4, "ragged": True, "lens": 8},
    ]


def draw(rng):
    most = {}
    for c in listed():
        w = work(c)
        m = most.setdefault(c["op"], [0, 0])
        m[0], m[1] = max(m[0], w["bytes"]), max(m[1], w["flops"])

    def log(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    while True:
        op = rng.choice(["append", "append", "read", "attend", "attend", "attend"])
        d = rng.choice([64, 128, 128, 256])
        hkv, group = rng.choice([(8, 5), (8, 4), (16, 1), (2, 8), (1, 8), (4, 7), (3, 3)])
        c = {"op": op, "seqs": log(1, 64), "new": 1, "context": log(1, 60000), "ragged": rng.random() < 0.7, "hq": hkv * group,
             "hkv": hkv, "d": d, "page": rng.choice([32, 64, 64, 128, 256]), "rot": rng.choice([d, d // 2]),
             "interleaved": rng.random() < 0.5, "window": 0, "sinks": 0, "lens": rng.randrange(1 << 20)}
        kind = rng.choice(["one", "slots", "prompt"])
        if op == "read" or kind == "prompt":
            c["new"] = log(17, 12000)
            c["seqs"] = log(1, 8)
            c["context"] = log(1, 12000)
        elif kind == "slots":
            c["new"] = rng.randint(2, 16)
        if op == "attend" and rng.random() < 0.4:
            c["window"], c["sinks"] = log(16, 8192), rng.choice([0, 1, 4, 64])
        w, m = work(c), most[op]
        longest = max(l for _, l in _lens(c))
        dense = c["seqs"] * c["hkv"] * min(longest, c["window"] + c["new"] + c["sinks"] + 4 * c["page"] if c["window"] else longest)
        scores = dense * group * c["new"] if op == "attend" else 0
        if w["bytes"] <= m[0] and w["flops"] <= max(m[1], 1) and dense * d <= 9e8 and scores <= 7.5e8:
            return c


def _lens(c):
    """[(new tokens, tokens in the cache)] of the sequences."""
    r, got = random.Random(c["lens"]), []
    for s in range(c["seqs"]):
        n, ctx = c["new"], c["context"]
        if c["ragged"]:
            n = n if n == 1 else max(1, int(n * r.uniform(0.3, 1.0)))
            ctx = int(ctx * r.uniform(0.2, 1.0))
            if s == 3:          # a slot without new tokens
                n = 0
        got.append((n, ctx + n))
    return got


def _visible(c):
    """Over all rows: (row, visible token) pairs of one query head; tokens that some row of a sequence sees."""
    pairs = tokens = 0
    w, k = c["window"], c["sinks"]
    for n, length in _lens(c):
        if not n:
            continue
        if not w:
            first = length - n + 1
            pairs += n * (first + length) // 2
            tokens += length
            continue
        for p in range(length - n, length):
            low = max(0, p - w + 1)
            pairs += p + 1 - low + min(k, low)
        low = max(0, length - n - w + 1)
        tokens += length - low + min(k, low)
    return pairs, tokens


def work(c):
    d, hq, hkv = c["d"], c["hq"], c["hkv"]
    rows = sum(n for n, _ in _lens(c))
    if c["op"] == "attend":
        pairs, tokens = _visible(c)
        return {"bytes": rows * hq * (4 * d + 4) + tokens * hkv * 2 * d + tokens * hkv * 8 / c["page"], "flops": 4.0 * d * hq * pairs}
    if c["op"] == "read":
        return {"bytes": rows * hkv * 2 * d * 3 + rows * hkv * 8 / c["page"], "flops": 2.0 * rows * hkv * d}
    # the new tokens through the append, and the pages that it touched read back
    back = sum(_window_of(n, length, c["page"]) for n, length in _lens(c))
    return {"bytes": rows * (hq * 4 * d + hkv * 2 * d * 3 + 4 * c["rot"]) + back * hkv * 2 * d * 3,
            "flops": 3.0 * rows * (hq + hkv) * c["rot"] + 2.0 * rows * hkv * 2 * d}


def _window_of(n, length, page):
    """Tokens from the start of the first page that the new tokens touch."""
    return length - (length - n) // page * page if n else 0


def prepare(c, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))
    lens = _lens(c)
    hq, hkv, d, page = c["hq"], c["hkv"], c["d"], c["page"]
    pages = [max(1, -(-length // page)) for _, length in lens]
    total = sum(pages)
    order = torch.randperm(total, generator=gen, device=dev, dtype=torch.int64).to(torch.int32).cpu()
    table = torch.zeros((len(lens), max(pages)), dtype=torch.int32)
    at = 0
    for s, p in enumerate(pages):
        table[s, :p] = order[at:at + p]
        at += p
    starts = [0]
    for n, _ in lens:
        starts.append(starts[-1] + n)
    rows = starts[-1]
    state = {
        "case": dict(c), "rows": rows, "longest": max(length for _, length in lens), "new": max(n for n, _ in lens), "workspace": None,
        "q_start": torch.tensor(starts, dtype=torch.int32, device=dev),
        "kv_len": torch.tensor([length for _, length in lens], dtype=torch.int32, device=dev),
        "table": table.to(dev),
        # a page more than the tables name
        "k_codes": torch.empty((total + 1, hkv, page, d), dtype=torch.uint8, device=dev),
        "v_codes": torch.empty((total + 1, hkv, page, d), dtype=torch.uint8, device=dev),
        "k_scale": torch.rand((total + 1, hkv), generator=gen, device=dev) * 0.02 + 0.02,
        "v_scale": torch.rand((total + 1, hkv), generator=gen, device=dev) * 0.02 + 0.02,
    }
    step = max(1, (1 << 26) // (hkv * page * d))
    for codes in (state["k_codes"], state["v_codes"]):   # codes as a block's largest value of about 3.8 deviations leaves them
        for i in range(0, total + 1, step):
            x = torch.randn(codes[i:i + step].shape, generator=gen, device=dev)
            codes[i:i + step] = (x * 33.0).round_().clamp_(-127, 127).add_(128).to(torch.uint8)

    def activations(heads):
        x = torch.randn((rows, heads, d), generator=gen, device=dev)
        wide = torch.randperm(d, generator=gen, device=dev)[:max(1, d // 100)]   # a few channels with large values
        x[:, :, wide] *= 4.0
        return x.to(torch.bfloat16)

    if c["op"] == "attend":
        state["q"] = activations(hq)
    elif c["op"] == "append":
        # the three as the projection leaves them: side by side in one row
        qkv = torch.cat([activations(hq), activations(hkv), activations(hkv)], dim=1)
        state["q"], state["k"], state["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        pos = torch.arange(max(pages) * page, dtype=torch.float64, device=dev)
        inv = 10000.0 ** (-torch.arange(0, c["rot"], 2, dtype=torch.float64, device=dev) / c["rot"])
        angle = pos[:, None] * inv[None, :]
        state["rope"] = torch.stack([angle.cos(), angle.sin()], dim=-1).float()   # [positions][rot/2][2]
        back = [0]
        for n, length in lens:
            back.append(back[-1] + _window_of(n, length, page))
        state["back"], state["back_rows"] = torch.tensor(back, dtype=torch.int32, device=dev), back[-1]
        state["span"] = max(_window_of(n, length, page) for n, length in lens)
    return state


def run(s):
    c = s["case"]
    if own:
        import bit_quantized_lm_amd as lib
        cache = (s["k_codes"], s["v_codes"], s["k_scale"], s["v_scale"])
        if c["op"] == "attend":
            if s["workspace"] is None:
                s["workspace"] = lib.draft_layer_workspace(s["rows"], c["seqs"], c["hq"], c["hkv"], c["d"], s["q"].device)
            return lib.draft_layer_attend(s["q"], *cache, s["q_start"], s["kv_len"], s["table"], window=c["window"], sinks=c["sinks"],
                                          workspace=s["workspace"])
        if c["op"] == "read":
            return lib.draft_layer_read(*cache, s["q_start"], s["kv_len"], s["table"], s["rows"])
        q = lib.draft_layer_append(s["q"], s["k"], s["v"], s["rope"], *cache, s["q_start"], s["kv_len"], s["table"],
                                   interleaved=c["interleaved"])
        return (q, *lib.draft_layer_read(*cache, s["back"], s["kv_len"], s["table"], s["back_rows"]))
    if c["op"] == "attend":
        return _attend(s, c)
    if c["op"] == "read":
        return _read(s, s["q_start"], s["rows"])
    q = _append(s, c)
    return (q, *_read(s, s["back"], s["back_rows"]))


# ------------------------------------------------------------------ the plain forms
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


def _k_order(x):
    """The reverse of _k_natural."""
    *lead, page, d = x.shape
    n = len(lead)
    x = x.reshape(*lead, page // 32, 2, 16, d // 64, 4, 16)
    return x.permute(*range(n), n, n + 1, n + 3, n + 4, n + 2, n + 5).reshape(*lead, page, d)


def _v_order(x):
    """The reverse of _v_natural."""
    *lead, page, d = x.shape
    n = len(lead)
    x = x.reshape(*lead, page // 32, 2, 4, 4, d // 32, 2, 16)
    return x.permute(*range(n), n, n + 4, n + 2, n + 6, n + 5, n + 1, n + 3).reshape(*lead, page, d)


def _values(codes, scale, natural, ids):
    """fp32 [S][heads][tokens][d] of the pages `ids` [S][P]."""
    x = natural(codes[ids]).float() - 128.0                            # [S][P][heads][page][d]
    x = x * scale[ids][..., None, None]
    n_s, n_p, heads, page, d = x.shape
    return x.transpose(1, 2).reshape(n_s, heads, n_p * page, d)


def _rows_of(start, rows):
    """(sequence, index in it) of every row of a ragged batch."""
    at = torch.arange(rows, device=start.device, dtype=torch.int32)
    seq = torch.searchsorted(start, at, right=True) - 1
    return seq, at - start[seq]


def _attend(s, c):
    q, page, w, sinks = s["q"], c["page"], c["window"], c["sinks"]
    dev, hkv, d = q.device, c["hkv"], c["d"]
    group, n_s, most = c["hq"] // hkv, c["seqs"], s["new"]
    table, kv_len, start = s["table"].long(), s["kv_len"].long(), s["q_start"].long()
    n_pages = table.shape[1]
    if w:   # the pages of the first tokens, and those that the window can reach
        first = min(n_pages, -(-sinks // page))
        near = min(n_pages, -(-(w + most) // page) + 1)
        low = (torch.clamp(-(-kv_len // page), min=1) - near).clamp(min=0)
        index = torch.cat([torch.arange(first, device=dev)[None, :].expand(n_s, first), low[:, None] + torch.arange(near, device=dev)[None, :]], 1)
        fresh = torch.cat([torch.arange(first, device=dev)[None, :] < low[:, None], torch.ones((n_s, near), dtype=torch.bool, device=dev)], 1)
    else:
        index = torch.arange(n_pages, device=dev)[None, :].expand(n_s, n_pages)
        fresh = torch.ones_like(index, dtype=torch.bool)
    ids = table.gather(1, index)
    j = (index[:, :, None] * page + torch.arange(page, device=dev)).reshape(n_s, -1)
    fresh = fresh[:, :, None].expand(-1, -1, page).reshape(n_s, -1)
    k = _values(s["k_codes"], s["k_scale"], _k_natural, ids)
    v = _values(s["v_codes"], s["v_scale"], _v_natural, ids)
    i = torch.arange(most, device=dev)
    pad = (start[:-1, None] + i[None, :]).clamp(max=s["rows"] - 1)
    x = q[pad].float().reshape(n_s, most, hkv, group, d).permute(0, 2, 1, 3, 4).reshape(n_s, hkv, most * group, d)
    scores = torch.matmul(x, k.transpose(2, 3)) * (1.0 / math.sqrt(d))
    p = (kv_len - (start[1:] - start[:-1]))[:, None] + i[None, :]
    seen = (j[:, None, :] <= p[:, :, None]) & fresh[:, None, :]
    if w:
        seen &= (j[:, None, :] > p[:, :, None] - w) | (j[:, None, :] < sinks)
    scores = scores.reshape(n_s, hkv, most, group, -1).masked_fill(~seen[:, None, :, None, :], -math.inf).reshape(scores.shape)
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    e = torch.exp(scores - top)
    total = e.sum(-1, keepdim=True)
    o = torch.matmul(e, v) / torch.where(total == 0, torch.ones_like(total), total)
    lse = top + torch.log(total)
    seq, at = _rows_of(s["q_start"], s["rows"])
    o = o.reshape(n_s, hkv, most, group, d).permute(0, 2, 1, 3, 4).reshape(n_s, most, c["hq"], d)[seq, at]
    lse = lse.reshape(n_s, hkv, most, group).permute(0, 2, 1, 3).reshape(n_s, most, c["hq"])[seq, at]
    return o.to(torch.bfloat16), lse


def _read(s, start, rows):
    c = s["case"]
    page, table = c["page"], s["table"].long()
    seq, at = _rows_of(start, rows)
    begin = s["kv_len"] - (start[1:] - start[:-1])
    first = (begin // page).long()
    index = first[:, None] + torch.arange(-(-(s["span"] if c["op"] == "append" else s["new"] + page) // page), device=table.device)
    ids = table.gather(1, index.clamp(max=table.shape[1] - 1))
    inside = (begin[seq] + at).long() - first[seq] * page
    return [_values(codes, scale, natural, ids)[seq, :, inside].to(torch.bfloat16)
            for codes, scale, natural in ((s["k_codes"], s["k_scale"], _k_natural), (s["v_codes"], s["v_scale"], _v_natural))]


def _rotate(x, cos, sin, interleaved):
    """x fp32 [..., heads, d]; cos, sin [..., 1, rot/2]."""
    half = cos.shape[-1]
    r, rest = x[..., :2 * half], x[..., 2 * half:]
    a, b = (r[..., 0::2], r[..., 1::2]) if interleaved else (r[..., :half], r[..., half:])
    u, v = a * cos - b * sin, b * cos + a * sin
    r = torch.stack([u, v], -1).flatten(-2) if interleaved else torch.cat([u, v], -1)
    return torch.cat([r, rest], -1)


def _append(s, c):
    dev, page, hkv, d = s["q"].device, c["page"], c["hkv"], c["d"]
    rope, n_s = s["rope"], c["seqs"]
    kv_len, start = s["kv_len"].long(), s["q_start"].long()
    begin = kv_len - (start[1:] - start[:-1])
    seq, at = _rows_of(s["q_start"], s["rows"])
    angle = rope[begin[seq] + at]
    q = _rotate(s["q"].float(), angle[:, None, :, 0], angle[:, None, :, 1], c["interleaved"]).to(torch.bfloat16)
    # the pages that new tokens touch, as many for each sequence; the spare page stands for those that one lacks
    n_p = -(-s["span"] // page)
    index = (begin // page)[:, None] + torch.arange(n_p, device=dev)[None, :]
    used = (index * page < kv_len[:, None]) & (begin < kv_len)[:, None]
    spare = s["k_codes"].shape[0] - 1
    ids = torch.where(used, s["table"].long().gather(1, index.clamp(max=s["table"].shape[1] - 1)), spare)
    pos = index[:, :, None] * page + torch.arange(page, device=dev)                       # [S][P][page]
    new = (pos >= begin[:, None, None]) & (pos < kv_len[:, None, None])
    old = pos < begin[:, None, None]
    row = (start[:-1, None, None] + pos - begin[:, None, None]).clamp(0, s["rows"] - 1)
    angle = rope[pos.clamp(max=rope.shape[0] - 1)]
    for x, codes, scale, natural, order in ((s["k"], s["k_codes"], s["k_scale"], _k_natural, _k_order),
                                            (s["v"], s["v_codes"], s["v_scale"], _v_natural, _v_order)):
        x = x[row].float()                                                                # [S][P][page][heads][d]
        if scale is s["k_scale"]:
            x = _rotate(x, angle[..., None, :, 0], angle[..., None, :, 1], c["interleaved"])
        x = x.transpose(2, 3)                                                             # [S][P][heads][page][d]
        fresh, kept = new[:, :, None, :, None], old[:, :, None, :, None]
        amax = torch.where(fresh, x.abs(), torch.zeros_like(x)).amax((-1, -2))
        before = scale[ids]
        step = torch.clamp(amax / 127.0, min=FLOOR)
        step = torch.where(old.any(-1)[:, :, None], torch.maximum(step, before), step)
        was = natural(codes[ids]).float() - 128.0
        again = torch.round(was * (before / step)[..., None, None])
        written = torch.round(x * (1.0 / step)[..., None, None]).clamp(-127, 127)
        value = torch.where(fresh, written, torch.where(kept, again, was))
        codes[ids] = order(value + 128.0).to(torch.uint8)
        scale[ids] = step
    return q


# ------------------------------------------------------------------ the definition in 64 bits
def exact(c, seed):
    s = prepare(c, seed)
    lens, page, hkv, hq, d = _lens(c), c["page"], c["hkv"], c["hq"], c["d"]
    dev = s["k_codes"].device
    table = s["table"].cpu().tolist()
    t, e = torch.arange(page, device=dev)[:, None], torch.arange(d, device=dev)[None, :]
    u = t % 32
    place = {   # byte of token t, element e inside a (page, head), as the layout is documented
        "k": t // 32 * 32 * d + ((u // 16 * (d // 64) + e // 64) * 64 + e % 64 // 16 * 16 + u % 16) * 16 + e % 16,
        "v": t // 32 * 32 * d + ((e // 32 * 4 + u % 16 // 4) * 16 + e % 16) * 16 + e % 32 // 16 * 8 + u // 16 * 4 + u % 4,
    }

    def codes_of(which, ids, head):
        raw = s[which + "_codes"][ids, head].reshape(len(ids), -1)
        return raw[:, place[which].reshape(-1)].double().reshape(len(ids), page, d) - 128

    def cached(which, seq, head, lo, hi):
        """Values of positions lo..hi-1."""
        if hi <= lo:
            return torch.zeros((0, d), dtype=torch.float64, device=dev)
        p0, p1 = lo // page, -(-hi // page)
        ids = table[seq][p0:p1]
        x = codes_of(which, ids, head) * s[which + "_scale"][ids, head].double()[:, None, None]
        return x.reshape(-1, d)[lo - p0 * page:hi - p0 * page]

    at = [0]
    for n, _ in lens:
        at.append(at[-1] + n)
    if c["op"] == "read":
        k, v = (torch.empty((s["rows"], hkv, d), dtype=torch.float64, device=dev) for _ in range(2))
        for i, (n, length) in enumerate(lens):
            for h in range(hkv):
                k[at[i]:at[i + 1], h] = cached("k", i, h, length - n, length)
                v[at[i]:at[i + 1], h] = cached("v", i, h, length - n, length)
        return [k, v]
    if c["op"] == "attend":
        out = torch.zeros((s["rows"], hq, d), dtype=torch.float64, device=dev)
        lse = torch.full((s["rows"], hq), -math.inf, dtype=torch.float64, device=dev)
        g, w = hq // hkv, c["window"]
        for i, (n, length) in enumerate(lens):
            if not n:
                continue
            q = s["q"][at[i]:at[i + 1]].double()
            p = torch.arange(length - n, length, device=dev)[:, None]
            low = max(0, length - n - w + 1) if w else 0
            j = torch.arange(low, length, device=dev)
            if low:
                j = torch.cat([torch.arange(min(low, c["sinks"]), device=dev), j])
            hidden = j > p
            if w:
                hidden |= (j <= p - w) & (j >= c["sinks"])
            for h in range(hkv):
                k, v = (torch.cat([cached(x, i, h, 0, min(low, c["sinks"])), cached(x, i, h, low, length)]) for x in "kv")
                for m in range(h * g, h * g + g):
                    z = (q[:, m] @ k.T) / math.sqrt(d)
                    z.masked_fill_(hidden, -math.inf)
                    lse[at[i]:at[i + 1], m] = torch.logsumexp(z, 1)
                    out[at[i]:at[i + 1], m] = torch.softmax(z, 1) @ v
        return [out, lse]
    rot, back = c["rot"] // 2, s["back"].cpu().tolist()
    turn = torch.view_as_complex(s["rope"].double())

    def rotated(x, pos):
        x = x.double()
        r = x[..., :2 * rot]
        z = torch.complex(r[..., 0::2], r[..., 1::2]) if c["interleaved"] else torch.complex(r[..., :rot], r[..., rot:])
        z = z * turn[pos][:, None, :]
        r = torch.view_as_real(z).flatten(-2) if c["interleaved"] else torch.cat([z.real, z.imag], -1)
        return torch.cat([r, x[..., 2 * rot:]], -1)

    q = torch.empty((s["rows"], hq, d), dtype=torch.float64, device=dev)
    both = {x: torch.empty((s["back_rows"], hkv, d), dtype=torch.float64, device=dev) for x in "kv"}
    for i, (n, length) in enumerate(lens):
        if not n:
            continue
        begin = length - n
        pos = torch.arange(begin, length, device=dev)
        q[at[i]:at[i + 1]] = rotated(s["q"][at[i]:at[i + 1]], pos)
        fresh = {"k": rotated(s["k"][at[i]:at[i + 1]], pos), "v": s["v"][at[i]:at[i + 1]].double()}
        for page_no in range(begin // page, -(-length // page)):
            lo, hi = page_no * page, min(length, page_no * page + page)
            old = max(0, begin - lo)
            for x in "kv":
                new = fresh[x][max(lo, begin) - begin:hi - begin]                     # [tokens][heads][d]
                step = (new.abs().amax((0, 2)) / 127).clamp(min=FLOOR)
                to = both[x][back[i] + lo - begin // page * page:back[i] + hi - begin // page * page]
                if old:
                    before = s[x + "_scale"][table[i][page_no]].double()
                    step = torch.maximum(step, before)
                    was = torch.stack([codes_of(x, [table[i][page_no]], h)[0, :old] for h in range(hkv)], 1)
                    to[:old] = torch.round(was * (before / step)[:, None]) * step[:, None]
                to[old:] = torch.round(new / step[:, None]).clamp(-127, 127) * step[:, None]
    return [q, both["k"], both["v"]]
