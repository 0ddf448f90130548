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
