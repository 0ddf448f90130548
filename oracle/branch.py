"""Oracle of the operators on several branches of one context: the next batch's
pages, the pool drawn together, log probabilities (float64).  Written from the
definitions with plain loops; shares no code with the library.
"""
import numpy as np


def fork(uses, table, kv_len, parents, need, page):
    """(table_out, uses_out, status, copies [(from, to)])."""
    uses, table = np.maximum(uses, 0), np.asarray(table)
    n_pages, wide = len(uses), table.shape[1]

    def held(i):
        return 0 <= i < n_pages

    free = [i for i in range(n_pages) if uses[i] <= 0]
    asked, seen, new, copies = 0, set(), [], []
    for p, n in zip(parents, need):
        there = 0 <= p < len(table)
        old = [int(i) for i in table[p]] if there else [-1] * wide
        length = min(max(int(kv_len[p]), 0), wide * page) if there else 0
        full, last = length // page, -(-min(max(int(n), length), wide * page) // page)
        line = [i if held(i) else -1 for i in old[:full]]
        for j in range(full, last):
            if there and p not in seen and held(old[j]) and uses[old[j]] == 1:
                line.append(old[j])
                continue
            got = free[asked] if asked < len(free) else -1
            asked += 1
            if j * page < length and held(old[j]):
                copies.append((old[j], got))
            line.append(got)
        if there:
            seen.add(p)
        new.append(line + [-1] * (wide - len(line)))
    if asked > len(free):
        return np.full((len(new), wide), -1, np.int32), uses.copy(), np.array([len(free), asked - len(free)], np.int32), []
    out = uses.copy()
    for i in table.ravel():
        if held(i):
            out[i] -= 1
    for line in new:
        for i in line:
            if i >= 0:
                out[i] += 1
    return np.array(new, np.int32), out, np.array([int((out <= 0).sum()), 0], np.int32), copies


def compact(uses, table):
    """(table_out, uses_out, status, moves [(from, to)])."""
    uses = np.maximum(uses, 0)
    used = int((uses > 0).sum())
    moves = list(zip([i for i in range(used, len(uses)) if uses[i] > 0], [i for i in range(used) if uses[i] <= 0]))
    out, to = uses.copy(), {}
    for a, b in moves:
        out[b], out[a], to[a] = uses[a], 0, b
    return np.array([[to.get(int(i), int(i)) for i in line] for line in table], np.int32), out, np.array([used, len(moves)], np.int32), moves


def attend(q, kc, vc, ks, vs, q_start, kv_len, table, group_start, prefix_len, scale, window, sinks):
    """(out, lse, spread, absqk) as oracle.layer.attend gives them; kc, vc: signed
    codes token by element."""
    rows, hq, d = q.shape
    n_pages, hkv, page = kc.shape[0], kc.shape[1], kc.shape[2]
    group, cap = hq // hkv, table.shape[1] * page
    out, spread = np.zeros((rows, hq, d)), np.zeros((rows, hq, d))
    lse, absqk = np.full((rows, hq), -np.inf), np.zeros((rows, hq))
    leader, shared = np.arange(len(kv_len)), np.zeros(len(kv_len), np.int64)
    for g, p in enumerate(prefix_len):
        for s in range(group_start[g], group_start[g + 1]):
            leader[s], shared[s] = group_start[g], max(int(p), 0)
    for s in range(len(kv_len)):
        n = int(q_start[s + 1] - q_start[s])
        length = int(min(max(kv_len[s], 0), cap))
        if n == 0 or length == 0:
            continue
        j = np.arange(length)
        ids = np.where(j < shared[s], table[leader[s], j // page], table[s, j // page])     # every token's page
        there = (ids >= 0) & (ids < n_pages)
        ids = np.where(there, ids, 0)
        p = (int(kv_len[s]) - n + np.arange(n))[:, None]
        seen = (j[None, :] <= p) & there[None, :]
        if window:
            seen &= (j[None, :] > p - window) | (j[None, :] < sinks)
        r = slice(int(q_start[s]), int(q_start[s + 1]))
        for h in range(hkv):
            k = np.where(there[:, None], kc[ids, h, j % page] * ks[ids, h].astype(np.float64)[:, None], 0.0)
            v = np.where(there[:, None], vc[ids, h, j % page] * vs[ids, h].astype(np.float64)[:, None], 0.0)
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


def logprobs(x, tokens, top, factor):
    """x [M][N], factor [M]: dict of float64 results, and what tolerances are made
    of: far = mean of |z - max z|, far2 = mean of its square."""
    x = np.asarray(x, np.float64)
    m, n = x.shape
    r = {"logprob": np.empty(tokens.shape), "lse": np.empty(m), "entropy": np.empty(m), "top_id": np.full((m, top), -1), "top_logprob": np.full((m, top), -np.inf),
         "far": np.zeros(m), "far2": np.zeros(m), "max": np.zeros(m)}
    for i in range(m):
        f = float(factor[i])
        here = (tokens[i] >= 0) & (tokens[i] < n)
        if not (f > 0 and np.isfinite(f)) or np.isnan(x[i]).any() or np.isposinf(x[i]).any():
            for k in ("logprob", "lse", "entropy", "top_logprob"):
                r[k][i] = np.nan
            continue
        if np.isneginf(x[i]).all():
            r["logprob"][i] = r["lse"][i] = -np.inf
            r["entropy"][i] = 0.0
            continue
        d = (x[i] - x[i].max()) * f
        e = np.exp(d)
        lnl = np.log(e.sum())
        p = e / e.sum()
        some = e > 0
        r["max"][i] = f * x[i].max()
        r["lse"][i] = r["max"][i] + lnl
        r["far"][i], r["far2"][i] = (p[some] * -d[some]).sum(), (p[some] * d[some] ** 2).sum()
        r["entropy"][i] = lnl + r["far"][i]
        r["logprob"][i] = np.where(here, d[np.where(here, tokens[i], 0)] - lnl, -np.inf)
        best = np.lexsort((np.arange(n), -x[i]))[:top]
        best = best[x[i][best] > -np.inf]
        r["top_id"][i, :len(best)] = best
        r["top_logprob"][i, :len(best)] = d[best] - lnl
    return r
