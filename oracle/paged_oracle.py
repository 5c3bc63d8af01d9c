"""The paged-cache operators in numpy fp64, from their definitions.

A cache is a dict of numpy arrays: k, v [n_pages, kv_heads, page_rows, hd]
(fp64), pos, weight [n_pages, kv_heads, page_rows], table [n_seq, max_pages],
length [n_seq]. Every function works row by row through `rows_of`, so none
shares an index trick with a kernel."""

import numpy as np


def rows_of(cache, s, n=None):
    """(page, row) of the first n (default: all) rows of sequence s; None where the page id is outside the pool."""
    pages, ps = cache["k"].shape[0], cache["k"].shape[2]
    n = min(int(cache["length"][s]), cache["table"].shape[1] * ps) if n is None else n
    out = []
    for r in range(n):
        page = int(cache["table"][s, r // ps])
        out.append((page, r % ps) if 0 <= page < pages else None)
    return out


def head_norm(x, gain, eps):
    """RMSNorm over the last axis; gain None: x itself."""
    if gain is None:
        return x
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * gain


def rotate(x, pos, pair_axis, theta, neox):
    """x [heads, hd] rotated at pos [n_axes]: pair i by pos[pair_axis[i]] * theta ** (-i / pairs)."""
    y = x.copy()
    pairs = len(pair_axis)
    for i, axis in enumerate(pair_axis):
        angle = float(pos[axis]) * theta ** (-i / pairs)
        a, b = (i, i + pairs) if neox else (2 * i, 2 * i + 1)
        y[:, a] = x[:, a] * np.cos(angle) - x[:, b] * np.sin(angle)
        y[:, b] = x[:, b] * np.cos(angle) + x[:, a] * np.sin(angle)
    return y


def append(cache, q, k, v, row_pos, start, rope_pos, pair_axis, theta, neox, q_norm, k_norm, eps):
    """Changes the cache; returns the rotated q (rows of no sequence as given)."""
    out = q.copy()
    for s in range(len(start) - 1):
        a, b = int(start[s]), int(start[s + 1])
        where = rows_of(cache, s)
        for t in range(a, b):
            p = rope_pos[:, t] if len(pair_axis) else []
            out[t] = rotate(head_norm(q[t], q_norm, eps), p, pair_axis, theta, neox)
            slot = len(where) - (b - t)
            if slot < 0 or where[slot] is None:
                continue
            page, r = where[slot]
            cache["k"][page, :, r] = rotate(head_norm(k[t], k_norm, eps), p, pair_axis, theta, neox)
            cache["v"][page, :, r] = v[t]
            cache["pos"][page, :, r] = row_pos[t]
            cache["weight"][page, :, r] = 0.0
    return out


def sees(pq, pk, causal, window, prefix):
    """pq [n, 1], pk [1, m] -> bool [n, m]."""
    d = pq - pk
    m = np.ones(d.shape, dtype=bool)
    if causal:
        m &= d >= 0
    if window > 0:
        m &= np.abs(d) <= window
    return m | (pk < prefix) if prefix is not None else m


def scores(q, k, pq, pk, scale, softcap, slope):
    """q [n, hd], k [m, hd] -> t [n, m], and the largest sum of |q k| of a row (for error bounds)."""
    with np.errstate(invalid="ignore", over="ignore"):
        t = q @ k.T * scale
        if softcap:
            t = softcap * np.tanh(t / softcap)
        return t - slope * np.abs(pq - pk)


def _visit(cache, q, q_pos, start, scale, causal, window, softcap, slopes, prefix):
    """(s, kv head, query head, new rows, places, mask, t) of every sequence and head."""
    nq, nkv = q.shape[1], cache["k"].shape[1]
    for s in range(len(start) - 1):
        new = np.arange(int(start[s]), int(start[s + 1]))
        where = [w for w in rows_of(cache, s) if w is not None]
        page, r = np.array([w[0] for w in where], dtype=int), np.array([w[1] for w in where], dtype=int)
        for h in range(nkv):
            k, pk = cache["k"][page, h, r], cache["pos"][page, h, r].astype(np.int64)[None]
            pq = q_pos[new].astype(np.int64)[:, None]
            m = sees(pq, pk, causal, window, None if prefix is None else int(prefix[s]))
            for g in range(nq // nkv):
                i = h * (nq // nkv) + g
                t = scores(q[new, i], k, pq, pk, scale, softcap, 0.0 if slopes is None else slopes[i])
                yield s, h, i, new, (page, r), m, t


def attention(cache, q, q_pos, start, scale, causal=True, window=0, softcap=0.0, slopes=None, prefix=None):
    """out [rows, nq, hd], lse [rows, nq] and sum p |v| (the scale of rounding errors); rows of no sequence are NaN."""
    out = np.full(q.shape, np.nan)
    mag = np.full(q.shape, np.nan)
    lse = np.full(q.shape[:2], np.nan)
    for s, h, i, new, (page, r), m, t in _visit(cache, q, q_pos, start, scale, causal, window, softcap, slopes, prefix):
        v = cache["v"][page, h, r]
        for n, row in enumerate(new):
            at = np.flatnonzero(m[n])
            if not len(at):
                out[row, i], mag[row, i], lse[row, i] = 0.0, 0.0, -np.inf
                continue
            x = t[n, at]
            top = x.max()
            e = np.exp(x - top)
            out[row, i] = e @ v[at] / e.sum()
            mag[row, i] = e @ np.abs(v[at]) / e.sum()
            lse[row, i] = top + np.log(e.sum())
    return out, lse, mag


def key_weight(cache, q, q_pos, start, lse, weight, decay, weight_out, scale, causal=True, window=0, softcap=0.0, slopes=None, prefix=None):
    """weight_out (changed) and, in the same layout, the number of terms of each sum."""
    terms = np.zeros(weight_out.shape)
    got = np.zeros(weight_out.shape)
    for s, h, i, new, (page, r), m, t in _visit(cache, q, q_pos, start, scale, causal, window, softcap, slopes, prefix):
        for n, row in enumerate(new):
            if lse[row, i] == -np.inf:
                continue
            at = np.flatnonzero(m[n])
            got[page[at], h, r[at]] += np.exp(t[n, at] - lse[row, i])
            terms[page[at], h, r[at]] += 1
    for s in range(len(start) - 1):
        for w in rows_of(cache, s):
            if w is not None:
                old = 0.0 if weight is None else weight[w[0], :, w[1]]
                weight_out[w[0], :, w[1]] = decay * old + got[w[0], :, w[1]]
    return weight_out, terms


def evict(cache, budget, recent, next_pos, weight_out, pos_out):
    """Changes k, v of the cache, weight_out and pos_out; returns the new lengths."""
    lengths = []
    weight, pos = cache["weight"].copy(), cache["pos"].copy()
    for s in range(cache["table"].shape[0]):
        where = rows_of(cache, s)
        n = len(where)
        lengths.append(min(n, budget))
        for h in range(cache["k"].shape[1]):
            def rank(i):
                page, r = where[i]
                w = weight[page, h, r]
                if pos[page, h, r] >= int(next_pos[s]) - recent:
                    w = np.inf
                return (1, 0.0, i) if np.isnan(w) else (0, -w, i)
            keep = set(sorted(range(n), key=rank)[:budget])
            holes = [i for i in range(min(n, budget)) if i not in keep]
            late = [i for i in range(budget, n) if i in keep]
            for i in range(min(n, budget)):
                if i in keep:
                    page, r = where[i]
                    weight_out[page, h, r], pos_out[page, h, r] = weight[page, h, r], pos[page, h, r]
            assert len(holes) == len(late)
            for to, of in zip(holes, late):
                (pt, rt), (pf, rf) = where[to], where[of]
                cache["k"][pt, h, rt] = cache["k"][pf, h, rf]
                cache["v"][pt, h, rt] = cache["v"][pf, h, rf]
                weight_out[pt, h, rt], pos_out[pt, h, rt] = weight[pf, h, rf], pos[pf, h, rf]
    return np.array(lengths, dtype=np.int32)
