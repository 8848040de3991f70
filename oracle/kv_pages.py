"""Oracle: the cache's page operations (TEST INFRASTRUCTURE ONLY, see the package
docstring).  Plain loops over NumPy arrays, updated in place; caches as in kv.py."""

from __future__ import annotations

import numpy as np


def _copy(cache, src, dst):
    for a in cache:
        if a is not None:
            a[dst] = a[src]


def copy_pages(cache, src, dst):
    n = cache[0].shape[0]
    for s, d in zip(src, dst):
        if 0 <= s < n and 0 <= d < n:
            _copy(cache, s, d)


def fork(cache, table, parents, children, lens, shared, free, page, taken=0):
    """pages_used."""
    rows, blocks = table.shape
    pages = len(shared)
    used = max(0, int(taken))
    for p, c, n in zip(parents, children, lens):
        n = min(max(0, int(n)), blocks * page)
        if not (0 <= p < rows and 0 <= c < rows) or p == c:
            continue
        for j in range(n // page):
            table[c, j] = table[p, j]
            if 0 <= table[p, j] < pages:
                shared[table[p, j]] += 1
        if n % page:
            j, own = n // page, -1
            last = table[p, j]
            if 0 <= last < pages:
                if used < len(free) and 0 <= free[used] < pages:
                    own = int(free[used])
                    _copy(cache, last, own)
                used += 1
            table[c, j] = own
    return used


def release(table, lens, shared, free, page, start=None, end=None, taken=0):
    """The new free list, as long as it is."""
    rows, blocks = table.shape
    pages = len(shared)
    for b in range(rows):
        n = min(max(0, int(lens[b])), blocks * page)
        lo = 0 if start is None else max(0, int(start[b]))
        hi = n if end is None else int(end[b])
        for j in range(-(-n // page)):
            if j * page >= lo and min((j + 1) * page, n) <= hi:
                if 0 <= table[b, j] < pages:
                    shared[table[b, j]] -= 1
                table[b, j] = -1
    out = [int(x) for x in free[max(0, int(taken)):] if 0 <= x < pages]
    for p in range(pages):
        if shared[p] < 0:
            shared[p] = 0
            out.append(p)
    return out


def compact(cache, table, lens, shared, page):
    """(new free list, pages in use)."""
    pages = len(shared)
    live = [(b, j) for b in range(len(lens)) for j in range(min(-(-max(0, int(lens[b])) // page), table.shape[1]))
            if 0 <= table[b, j] < pages]
    used = sorted({int(table[b, j]) for b, j in live})
    n = len(used)
    holes = [p for p in range(n) if p not in set(used)]
    to = {}
    for hole, mover in zip(holes, reversed(used)):
        to[mover] = hole
        _copy(cache, mover, hole)
        shared[hole] = shared[mover]
    for b, j in live:
        table[b, j] = to.get(int(table[b, j]), table[b, j])
    shared[n:] = 0
    return list(range(n, pages)), n


def padded(ids, n):
    out = np.full(n, -1, np.int32)
    out[:min(n, len(ids))] = ids[:n]
    return out
