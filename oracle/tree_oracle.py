"""A verify round over trees of drafted tokens in numpy fp64, from the definitions.

A tree is a list `end`: row j's subtree is rows j .. end[j] - 1, in depth-first
order. The functions walk parents, where the kernels compare intervals."""

import numpy as np

from oracle import paged_oracle as P


def parents(end):
    """The parent of each row (-1: none): the nearest row before it whose subtree holds it."""
    n, up = len(end), []
    for i in range(n):
        j = i - 1
        while j >= 0 and not i < min(int(end[j]), n):
            j -= 1
        up.append(j)
    return up


def ancestors(end):
    """[n, n]: row i is row j or descends from it, along the chain of parents."""
    up = parents(end)
    out = np.zeros((len(end), len(end)), dtype=bool)
    for i in range(len(end)):
        j = i
        while j >= 0:
            out[i, j] = True
            j = up[j]
    return out


def attention(cache, q, q_pos, start, end, scale, causal=True, window=0, softcap=0.0, slopes=None, prefix=None):
    """out [rows, nq, hd], lse [rows, nq] and sum p |v|; rows of no sequence are NaN."""
    nq, nkv = q.shape[1], cache["k"].shape[1]
    out, mag, lse = np.full(q.shape, np.nan), np.full(q.shape, np.nan), np.full(q.shape[:2], np.nan)
    for s in range(len(start) - 1):
        a, b = int(start[s]), int(start[s + 1])
        where = P.rows_of(cache, s)
        base = len(where) - (b - a)
        tree = ancestors(end[a:b])
        slots = np.array([r for r, w in enumerate(where) if w is not None], dtype=int)
        page, r = np.array([where[x][0] for x in slots], dtype=int), np.array([where[x][1] for x in slots], dtype=int)
        for h in range(nkv):
            k, v, pk = cache["k"][page, h, r], cache["v"][page, h, r], cache["pos"][page, h, r].astype(np.int64)[None]
            pq = q_pos[a:b].astype(np.int64)[:, None]
            m = P.sees(pq, pk, causal, window, None if prefix is None else int(prefix[s]))
            new = slots >= base
            m[:, new] &= tree[:, slots[new] - base]
            for g in range(nq // nkv):
                i = h * (nq // nkv) + g
                t = P.scores(q[a:b, i], k, pq, pk, scale, softcap, 0.0 if slopes is None else slopes[i])
                for n in range(b - a):
                    at = np.flatnonzero(m[n])
                    if not len(at):
                        out[a + n, i], mag[a + n, i], lse[a + n, i] = 0.0, 0.0, -np.inf
                        continue
                    e = np.exp(t[n, at] - t[n, at].max())
                    out[a + n, i], mag[a + n, i] = e @ v[at] / e.sum(), e @ np.abs(v[at]) / e.sum()
                    lse[a + n, i] = t[n, at].max() + np.log(e.sum())
    return out, lse, mag


def sample(logits, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, largest=np.finfo(np.float32).max):
    """token, prob and how near a border came: the smallest distance of a running sum to a threshold that it was compared
    with, relative to the sum of all weights there."""
    x = np.where(np.isnan(logits), -np.inf, np.minimum(logits.astype(np.float64), largest))
    if not (x > -np.inf).any():
        return -1, 0.0, 1.0
    order = np.argsort(-x, kind="stable")
    if not temperature >= 2.0 ** -64:
        return int(order[0]), 1.0, 1.0
    with np.errstate(over="ignore", invalid="ignore"):
        w = np.exp((x - x.max()) / temperature) if np.isfinite(temperature) else (x > -np.inf).astype(np.float64)
    w[~(x > -np.inf)] = 0.0
    near = 1.0
    if top_k > 0:
        order = order[:top_k]
    if top_p < 1:
        run = np.cumsum(w[order])
        before, goal = run - w[order], max(0.0, float(top_p)) * run[-1]
        near = min(near, np.abs(run - goal).min() / run[-1])
        order = order[: max(1, int((before < goal).sum()))]
    if min_p > 0:
        least = min(float(min_p), 1.0)
        if least < 1.0:
            near = min(near, np.abs(w[order] - least).min())
        order = order[: max(1, int((w[order] >= least).sum()))]
    kept = np.sort(order)
    run = np.cumsum(w[kept])
    u = 0.0 if not u > 0 else float(u)
    if u >= 1:
        at = int(np.flatnonzero(w[kept] > 0)[-1])
    else:
        near = min(near, np.abs(run - u * run[-1]).min() / run[-1]) if u > 0 else near
        at = int((run <= u * run[-1]).sum())
    return int(kept[at]), float(w[kept[at]] / run[-1]), near


def accept(end, draft, sampled, width):
    """(path, emitted tokens) of one tree; a negative token is none, and its row is not walked."""
    up, path = parents(end), []
    cur = 0 if len(end) else -1
    while cur >= 0 and sampled[cur] >= 0 and len(path) < width:
        path.append(cur)
        cur = next((i for i in range(len(end)) if up[i] == cur and draft[i] == sampled[cur]), -1)
    return path, [int(sampled[i]) for i in path]


def commit(cache, path, count):
    """Changes k, v, pos and weight of the cache; its length is the one after the walk."""
    for s in range(len(count)):
        n = int(count[s])
        where = P.rows_of(cache, s, cache["table"].shape[1] * cache["k"].shape[2])
        base = int(cache["length"][s]) - n
        rows = [(where[base + i], where[base + int(path[s][i])]) for i in range(n)]
        for name in ("k", "v", "pos", "weight"):
            held = [cache[name][of[0], :, of[1]].copy() if of and to else None for to, of in rows]
            for (to, of), x in zip(rows, held):
                if x is not None:
                    cache[name][to[0], :, to[1]] = x
