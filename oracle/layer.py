"""Float64 oracle of the draft layer's attention: rotary table, the 8-bit append,
reading back and attention, written from the formulas with plain loops over
sequences, pages and heads.  Shares no code with the library.
"""
import math

import numpy as np

FLOOR = 2.0 ** -40


def rope_table(positions, rot, base=10000.0, factor=1.0, original=0, beta_fast=32.0, beta_slow=1.0, mscale=1.0):
    """float64 [positions][rot/2][2]."""
    i = np.arange(rot // 2, dtype=np.float64)
    f = base ** (-2.0 * i / rot)
    if original > 0:
        def c(n):
            return rot * math.log(original / (2 * math.pi * n)) / (2 * math.log(base))
        lo = max(math.floor(c(beta_fast)), 0)
        hi = min(math.ceil(c(beta_slow)), rot - 1)
        ramp = np.clip((i - lo) / max(hi - lo, 0.001), 0.0, 1.0)
    else:
        ramp = np.ones_like(i)
    f = f * (1 - ramp) + f / factor * ramp
    angle = np.arange(positions, dtype=np.float64)[:, None] * f[None, :]
    return np.stack([mscale * np.cos(angle), mscale * np.sin(angle)], axis=-1)


def key_byte(t, e, d):
    u = t % 32
    return (t // 32) * 32 * d + (((u // 16) * (d // 64) + e // 64) * 64 + ((e % 64) // 16) * 16 + u % 16) * 16 + e % 16


def value_byte(t, e, d):
    u = t % 32
    return (t // 32) * 32 * d + (((e // 32) * 4 + (u % 16) // 4) * 16 + e % 16) * 16 + ((e % 32) // 16) * 8 + (u // 16) * 4 + u % 4


def natural(codes, byte_of):
    """codes uint8 [pages][heads][page][d] in stored order -> signed codes float64, token by element."""
    n, h, page, d = codes.shape
    t, e = np.meshgrid(np.arange(page), np.arange(d), indexing="ij")
    return codes.reshape(n, h, page * d)[:, :, byte_of(t, e, d)].astype(np.float64) - 128.0


def rotate(x, turn, interleaved):
    """x [heads][d] of one token, turn [rot/2][2] -> float64."""
    x = np.array(x, dtype=np.float64)
    half = turn.shape[0]
    c, s = turn[:, 0].astype(np.float64), turn[:, 1].astype(np.float64)
    a, b = (x[:, 0:2 * half:2].copy(), x[:, 1:2 * half:2].copy()) if interleaved else (x[:, :half].copy(), x[:, half:2 * half].copy())
    u, v = a * c - b * s, b * c + a * s
    if interleaved:
        x[:, 0:2 * half:2], x[:, 1:2 * half:2] = u, v
    else:
        x[:, :half], x[:, half:2 * half] = u, v
    return x


def positions_of(q_start, kv_len):
    """[(sequence, row, position)] of every row."""
    out = []
    for s in range(len(kv_len)):
        n = q_start[s + 1] - q_start[s]
        out += [(s, q_start[s] + i, kv_len[s] - n + i) for i in range(n)]
    return out


def append(q, k, v, rope, kc, vc, ks, vs, q_start, kv_len, table, interleaved):
    """What the append leaves, before its last roundings: q_out float64, and per
    (page id, head, which) {"step", "want": {token: float codes}, "old": tokens
    re-rounded}; pages that no new token touches are absent.  kc, vc: signed
    codes from `natural`, ks, vs: the scales before."""
    rows = positions_of(q_start, kv_len)
    page, d = kc.shape[2], kc.shape[3]
    hkv = kc.shape[1]
    cap = table.shape[1] * page
    q_out = None if q is None else np.array(q, dtype=np.float64)
    fresh = {}
    for s, r, p in rows:
        at = rope[min(max(p, 0), cap - 1)] if rope is not None else np.zeros((0, 2))
        if q is not None:
            q_out[r] = rotate(q[r], at, interleaved)
        if 0 <= p < cap and 0 <= table[s, p // page] < kc.shape[0]:
            fresh.setdefault((s, p // page), {})[p % page] = (rotate(k[r], at, interleaved), np.array(v[r], dtype=np.float64))
    pages = {}
    for (s, j), tokens in fresh.items():
        pid, first = int(table[s, j]), min(tokens)
        for w, (codes, scale) in enumerate(((kc, ks), (vc, vs))):
            for h in range(hkv):
                step = max(max(np.abs(x[w][h]).max() for x in tokens.values()) / 127.0, FLOOR)
                before = float(scale[pid, h])
                if first > 0:
                    step = max(step, before)
                want = {t: np.clip(x[w][h] / step, -127, 127) for t, x in tokens.items()}
                for t in range(first):
                    want[t] = codes[pid, h, t] * (before / step)
                pages[(pid, h, w)] = {"step": step, "want": want, "kept": first > 0 and step == before, "old": set(range(first))}
    return q_out, pages


def attend(q, kc, vc, ks, vs, q_start, kv_len, table, scale, window, sinks):
    """(out, lse, spread, absqk): float64; spread = sum p |v| and absqk = the
    largest scale * sum |q||k| of a row, which the tolerances are made of."""
    rows, hq, d = q.shape
    page, hkv = kc.shape[2], kc.shape[1]
    group = hq // hkv
    out, spread = np.zeros((rows, hq, d)), np.zeros((rows, hq, d))
    lse, absqk = np.full((rows, hq), -np.inf), np.zeros((rows, hq))
    cap = table.shape[1] * page
    for s in range(len(kv_len)):
        n = int(q_start[s + 1] - q_start[s])
        length = int(min(max(kv_len[s], 0), cap))
        if n == 0 or length == 0:
            continue
        ids = table[s, : -(-length // page)]
        good = (ids >= 0) & (ids < kc.shape[0])
        ids = np.where(good, ids, 0)
        j = np.arange(length)
        there = np.repeat(good, page)[:length]
        p = (int(kv_len[s]) - n + np.arange(n))[:, None]
        seen = (j[None, :] <= p) & there[None, :]
        if window:
            seen &= (j[None, :] > p - window) | (j[None, :] < sinks)
        r = slice(int(q_start[s]), int(q_start[s + 1]))
        for h in range(hkv):
            k = (kc[ids, h] * ks[ids, h].astype(np.float64)[:, None, None]).reshape(-1, d)[:length]
            v = (vc[ids, h] * vs[ids, h].astype(np.float64)[:, None, None]).reshape(-1, d)[:length]
            k, v = np.where(there[:, None], k, 0.0), np.where(there[:, None], v, 0.0)
            for m in range(h * group, (h + 1) * group):
                x = q[r, m].astype(np.float64)
                z = np.where(seen, scale * (x @ k.T), -np.inf)
                top = z.max(axis=1, keepdims=True)
                some = np.isfinite(top[:, 0])
                e = np.exp(z - np.where(some[:, None], top, 0.0))
                total = e.sum(axis=1, keepdims=True)
                w = e / np.where(total == 0, 1.0, total)
                out[r, m], spread[r, m] = w @ v, w @ np.abs(v)
                lse[r, m] = np.where(some, top[:, 0] + np.log(np.where(some, total[:, 0], 1.0)), -np.inf)
                absqk[r, m] = np.where(seen, scale * (np.abs(x) @ np.abs(k).T), 0.0).max(axis=1)
    return out, lse, spread, absqk
