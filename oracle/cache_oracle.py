"""fp64 CPU reference of a cache held in 8 bits and of the pages of a cache: what
a byte holds, the store, the move of an accepted path, and the pool's calls, one
entry at a time.  Test infrastructure only.

A cache is a dict of numpy arrays: k, v (the bytes' numbers, float64, NaN where
the byte is one) [pages, heads, page, d], k_exp, v_exp (int) [pages, heads,
blocks]; fmt "e4m3" or "int8".
"""

import math

import numpy as np

LARGEST = {"e4m3": 448.0, "int8": 127.0}
TOP = {"e4m3": 119, "int8": 121}
LOW = -126


def e4m3_numbers():
    """The number of each of the 256 bytes."""
    out = np.zeros(256)
    for b in range(256):
        sign, exp, man = b >> 7, (b >> 3) & 15, b & 7
        x = math.ldexp(8 + man, exp - 10) if exp else math.ldexp(man, -9)
        out[b] = (-x if sign else x) if (exp, man) != (15, 7) else math.nan
    return out


def nearest(x, fmt):
    """The nearest number that a byte holds, ties to even; beyond the largest, it."""
    if math.isnan(x):
        return math.nan if fmt == "e4m3" else 0.0
    most = LARGEST[fmt]
    if abs(x) >= most:
        return math.copysign(most, x)
    if fmt == "int8":
        return float(round(x))  # Python rounds ties to even
    step = math.ldexp(1.0, max(math.frexp(x)[1] - 1, -6) - 3)
    return math.copysign(round(abs(x) / step) * step, x)


def least_exponent(most, fmt):
    for e in range(LOW, TOP[fmt]):
        if most <= math.ldexp(LARGEST[fmt], e):
            return e
    return TOP[fmt]


def clamp_exponent(e, fmt):
    return min(max(int(e), LOW), TOP[fmt])


def values(c, of):
    """float64 values of c["k"] or c["v"]."""
    held, exp = c[of], c[of + "_exp"]
    block = held.shape[2] // exp.shape[2]
    e = np.clip(exp, LOW, TOP[c["fmt"]]).repeat(block, 2)[..., None]
    return np.ldexp(held, e)


_nearest = np.vectorize(nearest, otypes=[float])


def _place(c, of, h, rows, data, needs):
    """Values data [m, d] into the rows (page, row), in whose blocks exponents become
    no smaller than each row's `needs`; rows of a block before its first new one live on."""
    fmt, held, exp = c["fmt"], c[of], c[of + "_exp"]
    block = held.shape[2] // exp.shape[2]
    blocks = {}
    for (page, row), x, e in zip(rows, data, needs):
        blocks.setdefault((page, row // block), []).append((row, x, e))
    for (page, j), new in blocks.items():
        first = min(r for r, _, _ in new) - j * block
        e = max(n for _, _, n in new)
        old = clamp_exponent(exp[page, h, j], fmt)
        if first > 0 and old >= e:
            e = old
        elif first > 0:
            part = held[page, h, j * block:j * block + first]
            part[:] = _nearest(np.ldexp(part, old - e), fmt)
        exp[page, h, j] = e
        for r, x, _ in new:
            held[page, h, r] = _nearest(np.ldexp(x, -e), fmt)


def store(c, k, v, cache_rows):
    """k, v [T, heads, d] into c, in place."""
    pages, heads, page, _ = c["k"].shape
    exp = c["k_exp"]
    block = page // exp.shape[2]
    there = [t for t, r in enumerate(cache_rows) if 0 <= r < pages * page]
    for of, x in (("k", k), ("v", v)):
        for h in range(heads):
            # the least exponent of a block is that of its largest finite number, so a row's own will do
            needs = []
            for t in there:
                a = np.abs(x[t, h])
                a = a[np.isfinite(a)]
                needs.append(least_exponent(a.max(initial=0.0), c["fmt"]))
            _place(c, of, h, [(int(cache_rows[t]) // page, int(cache_rows[t]) % page) for t in there],
                   [x[t, h] for t in there], needs)
    return c


def keep(c, page_table, context, path, n_kept):
    """The accepted rows behind the context, in place."""
    pages, heads, page, _ = c["k"].shape
    block = page // c["k_exp"].shape[2]

    def row_of(b, pos):
        col = pos // page
        p = int(page_table[b][col]) if col < len(page_table[b]) else -1
        return (p, pos % page) if 0 <= p < pages else None

    for b in range(len(context)):
        moves, last = [], -1
        for j in range(max(0, min(int(n_kept[b]), path.shape[1]))):
            node = int(path[b, j])
            if node <= last:
                break
            last = node
            to, of = row_of(b, int(context[b]) + j), row_of(b, int(context[b]) + node)
            if to and of:
                moves.append((to, of))
        # what lives in a destination block before the first kept row: the context's rows
        for name in ("k", "v"):
            vals, exp = values(c, name), np.clip(c[name + "_exp"], LOW, TOP[c["fmt"]])
            for h in range(heads):
                by_block = {}
                for to, of in moves:
                    by_block.setdefault((to[0], to[1] // block), []).append((to, of))
                for (p, j), some in by_block.items():
                    # the context's rows in this block, whether or not the first kept row follows them
                    lives = [i for i in range(block) if any(
                        row_of(b, pos) == (p, j * block + i) for pos in range(max(0, int(context[b]) - block), int(context[b])))]
                    e = max(int(exp[of[0], h, of[1] // block]) for _, of in some)
                    old = int(exp[p, h, j])
                    if lives and old >= e:
                        e = old
                    elif lives:
                        for i in lives:
                            c[name][p, h, j * block + i] = _nearest(np.ldexp(c[name][p, h, j * block + i], old - e), c["fmt"])
                    c[name + "_exp"][p, h, j] = e
                    for to, of in some:
                        if to == of and e == old:
                            continue
                        c[name][to[0], h, to[1]] = _nearest(np.ldexp(vals[of[0], h, of[1]], -e), c["fmt"])
    return c


# ---- pages -------------------------------------------------------------------

def _free(refs):
    return [p for p in range(len(refs)) if refs[p] <= 0]


def _names(entry, n):
    return 0 <= entry < n


def reserve(refs, table, lengths, page):
    """Returns the number of entries that got no page."""
    free, missing = _free(refs), 0
    for b in range(len(table)):
        for col in range(min(-(-max(int(lengths[b]), 0) // page), table.shape[1])):
            if _names(table[b, col], len(refs)):
                continue
            if free:
                table[b, col] = free.pop(0)
                refs[table[b, col]] = 1
            else:
                table[b, col] = -1
                missing += 1
    return missing


def fork(refs, from_table, to_table, parents, children, lengths, page):
    """Returns (pairs of pages to copy, forks without a page)."""
    free, pairs, missing, old = _free(refs), [], 0, from_table.copy()
    for parent, child, n in zip(parents, children, lengths):
        if not 0 <= child < len(to_table):
            continue
        row = np.full(to_table.shape[1], -1)
        if 0 <= parent < len(old) and n > 0:
            for col in range(min(n // page, len(row))):
                if _names(old[parent, col], len(refs)):
                    row[col] = old[parent, col]
                    refs[row[col]] += 1
            col = n // page
            if n % page and col < len(row) and _names(old[parent, col], len(refs)):
                if free:
                    row[col] = free.pop(0)
                    refs[row[col]] = 1
                    pairs.append((int(old[parent, col]), int(row[col])))
                else:
                    missing += 1
        to_table[child] = row
    return pairs, missing


def release(refs, table, rows, keep, page):
    for i, b in enumerate(rows):
        if not 0 <= b < len(table):
            continue
        first = 0 if keep is None else -(-max(int(keep[i]), 0) // page)
        for col in range(first, table.shape[1]):
            if _names(table[b, col], len(refs)):
                refs[table[b, col]] -= 1
            table[b, col] = -1


def compact(refs, table):
    """Returns (pages in use, moves)."""
    n = int((refs > 0).sum())
    moves = list(zip([p for p in range(n, len(refs)) if refs[p] > 0], [p for p in range(n) if refs[p] <= 0]))
    for of, to in moves:
        refs[to], refs[of] = refs[of], 0
        table[table == of] = to
    return n, moves
