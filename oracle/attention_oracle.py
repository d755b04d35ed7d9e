"""fp64 CPU reference of the operators after the q/k/v projection: the rotation
and the norm before it, tree masks, attention over a paged cache, and the move
of an accepted path.  Straight from the formulas, one token and one head at a
time; test infrastructure only.

Arrays are numpy; 16-bit inputs are passed as float64 (exact).  Every function
that computes an output also returns the magnitude its roundings are relative
to, from which the tests derive their tolerances.
"""

import math

import numpy as np


def rope_angles(positions, inv_freq):
    """[n, rot / 2] angles in fp64."""
    return np.asarray(positions, np.float64)[:, None] * np.asarray(inv_freq, np.float64)[None]


def norm_heads(x, weight, eps):
    """x [T, h, d] times weight / sqrt(mean(x^2) + eps)."""
    r = 1.0 / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps)
    return x * r * (1.0 if weight is None else weight)


def rotate_heads(x, table, positions, layout):
    """x [T, h, d] with its first table.shape[1] elements turned by
    table[positions] (cos | sin).  Returns (y, magnitude): |a| + |b| of each
    element's pair, |x| where nothing turns.  Rows of positions outside the
    table are NaN (nothing of them is written)."""
    rot = table.shape[1]
    half = rot // 2
    y, mag = x.copy(), np.abs(x)
    for i in range(half):
        ia, ib = (i, i + half) if layout == "half" else (2 * i, 2 * i + 1)
        for t, p in enumerate(positions):
            if not 0 <= p < table.shape[0]:
                y[t] = np.nan
                continue
            c, s = table[p, i], table[p, half + i]
            a, b = x[t, :, ia], x[t, :, ib]
            y[t, :, ia], y[t, :, ib] = a * c - b * s, b * c + a * s
            mag[t, :, ia] = mag[t, :, ib] = np.abs(a) + np.abs(b)
    return y, mag


def ancestors(parents):
    """[n, n] booleans: node i sees node j (itself and the nodes on its way)."""
    n = len(parents)
    sees = np.zeros((n, n), bool)
    for i in range(n):
        at = i
        while True:
            sees[i, at] = True
            nxt = int(parents[at])
            if not 0 <= nxt < at:
                break
            at = nxt
    return sees


def cache_rows_of(page_table_row, positions, page_size, n_pages):
    """Row page * page_size + place of each position, -1 where there is no page."""
    rows = []
    for p in positions:
        col = int(p) // page_size
        page = int(page_table_row[col]) if col < len(page_table_row) else -1
        rows.append(page * page_size + int(p) % page_size if 0 <= page < n_pages else -1)
    return np.array(rows, np.int64)


def attend(q, k_cache, v_cache, page_table, context, q_start, sees, scale):
    """q [T, hq, d]; caches [pages, hk, page, d]; sees: one [n, n] matrix a
    sequence.  Returns (out, lse, spread, score): out [T, hq, d]; lse [T, hq];
    spread [T, hq, d] the weighted mean of |v|; score [T, hq] the largest
    scale * sum |q| |k| of the row's keys."""
    T, hq, d = q.shape
    hk, page = k_cache.shape[1:3]
    out, spread = np.full((T, hq, d), np.nan), np.zeros((T, hq, d))
    lse, score = np.full((T, hq), np.nan), np.zeros((T, hq))
    for b in range(len(context)):
        n, ctx = q_start[b + 1] - q_start[b], int(context[b])
        rows = cache_rows_of(page_table[b], np.arange(ctx + n), page, k_cache.shape[0])
        for i in range(n):
            t = q_start[b] + i
            seen = np.concatenate([np.ones(ctx, bool), sees[b][i]]) & (rows >= 0)
            at = rows[seen]
            for h in range(hq):
                kv = h // (hq // hk)
                if not len(at):
                    out[t, h], lse[t, h] = 0.0, -math.inf
                    continue
                k, v = k_cache[at // page, kv, at % page], v_cache[at // page, kv, at % page]
                with np.errstate(invalid="ignore", over="ignore"):
                    s = scale * (k @ q[t, h])
                    m = s.max()
                    w = np.exp(s - m)
                    out[t, h] = (w[:, None] * v).sum(0) / w.sum()
                    lse[t, h] = m + math.log(w.sum()) if w.sum() > 0 else math.nan
                    spread[t, h] = (w[:, None] * np.abs(v)).sum(0) / w.sum()
                    score[t, h] = abs(scale) * (np.abs(k) @ np.abs(q[t, h])).max()
    return out, lse, spread, score


def keep(cache, page_table, context, path, n_kept):
    """cache [pages, hk, page, d] (changed in place)."""
    page = cache.shape[2]
    for b in range(len(context)):
        last = -1
        for j in range(max(0, min(int(n_kept[b]), path.shape[1]))):
            node = int(path[b, j])
            if node <= last:
                break
            last = node
            to, of = cache_rows_of(page_table[b], [int(context[b]) + j, int(context[b]) + node], page, cache.shape[0])
            if to >= 0 and of >= 0:
                cache[to // page, :, to % page] = cache[of // page, :, of % page]
    return cache
