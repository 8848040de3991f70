"""Oracle: the 4-bit paged key/value cache and attention over it.

TEST INFRASTRUCTURE ONLY (see the package docstring).  Plain loops in fp64,
except that codes, steps and zero points are taken in fp32 as quant.py takes
a weight group's (correctly rounded quotients, half to even).  Caches are NumPy triples (codes u32, scales
fp16, zeros u8 or None) in the layout that include/awq355.h gives.
"""

from __future__ import annotations

import numpy as np

from .quant import ORDER


def quantize_heads(x, zero_point=True):
    """quantize_groups' steps for fp32 values x [..., D], each last dimension a
    group: (codes, steps fp16, zeros or None)."""
    v = np.asarray(x, np.float32)
    if zero_point:
        lo = np.minimum(v.min(-1), np.float32(0))
        hi = np.maximum(v.max(-1), np.float32(0))
        s = np.maximum((hi - lo) / np.float32(15), np.float32(2.0 ** -14)).astype(np.float16)
        sf = s.astype(np.float32)
        z = np.clip(np.rint(-lo / sf), 0, 15)
        q = np.clip(np.rint(v / sf[..., None]) + z[..., None], 0, 15)
        return q.astype(np.uint8), s, z.astype(np.uint8)
    s = np.maximum(np.abs(v).max(-1) / np.float32(7), np.float32(2.0 ** -14)).astype(np.float16)
    q = np.clip(np.rint(v / s.astype(np.float32)[..., None]), -8, 7) + 8
    return q.astype(np.uint8), s, None


def new_cache(pages, heads, D, page, zero_point=True, rng=None):
    """A cache whose slots hold arbitrary bits (rng) or zeros."""
    shape, meta = (pages, 2, heads, page * D // 8), (pages, heads, page, 2)
    if rng is None:
        return (np.zeros(shape, np.uint32), np.zeros(meta, np.float16),
                np.zeros(meta, np.uint8) if zero_point else None)
    return (rng.integers(0, 2 ** 32, shape, dtype=np.uint32),
            rng.integers(0, 2 ** 16, meta, dtype=np.uint16).view(np.float16),
            rng.integers(0, 256, meta, dtype=np.uint8) if zero_point else None)


def _word_index(kv, off, word, D):
    """Index of word `word` of the token at offset `off` in its page's [P * D/8] words."""
    if kv == 0:
        return off * (D // 8) + word
    return (off // 4) * (D // 2) + word * 4 + off % 4


def append(cache, K, V, slots):
    """K, V float32 [T][heads][D] into slots (those outside the cache are skipped)."""
    codes, scales, zeros = cache
    T, heads, D = K.shape
    page = scales.shape[2]
    words = np.arange(D // 8)
    for t in range(T):
        if not 0 <= slots[t] < codes.shape[0] * page:
            continue
        pg, off = divmod(int(slots[t]), page)
        for kv, x in ((0, K[t]), (1, V[t])):
            q, s, z = quantize_heads(x, zeros is not None)
            q = q.reshape(heads, D // 8, 8).astype(np.uint32)
            w = np.zeros((heads, D // 8), np.uint32)
            for nib, ch in enumerate(ORDER):
                w |= q[:, :, ch] << np.uint32(4 * nib)
            codes[pg, kv, :, _word_index(kv, off, words, D)] = w.T
            scales[pg, :, off, kv] = s
            if zeros is not None:
                zeros[pg, :, off, kv] = z


def read(cache, D, slots):
    """(codes - 8, zeros - 8, steps, values) of slots, each for keys and values:
    fp64 [2][n][heads][D], [2][n][heads], [2][n][heads], [2][n][heads][D]."""
    codes, scales, zeros = cache
    heads, page = scales.shape[1], scales.shape[2]
    n = len(slots)
    c = np.zeros((2, n, heads, D))
    z = np.zeros((2, n, heads))
    s = np.zeros((2, n, heads))
    words = np.arange(D // 8)
    for i, slot in enumerate(slots):
        pg, off = divmod(int(slot), page)
        for kv in range(2):
            w = codes[pg, kv][:, _word_index(kv, off, words, D)]
            for nib, ch in enumerate(ORDER):
                c[kv, i, :, ch::8] = ((w >> np.uint32(4 * nib)) & np.uint32(15)).astype(np.float64) - 8
            s[kv, i] = scales[pg, :, off, kv].astype(np.float64)
            if zeros is not None:
                z[kv, i] = zeros[pg, :, off, kv].astype(np.float64) - 8
    return c, z, s, (c - z[..., None]) * s[..., None]


def assign(old, new, table, free, page, num_slots):
    """awq_kv_assign's outputs (table, seq_lens, query_start, slots, pages_used)."""
    table = table.copy()
    slots = np.full(num_slots, -1, np.int32)
    lens, start, used, t = [], [0], 0, 0
    for b in range(len(old)):
        o, n = max(0, int(old[b])), max(0, int(new[b]))
        have = -(-o // page)
        for i in range(n):
            blk, off = divmod(o + i, page)
            pg = -1
            if blk < table.shape[1]:
                if blk < have:
                    pg = int(table[b, blk])
                else:
                    at = used + blk - have
                    pg = int(free[at]) if at < len(free) else -1
                    if off == 0 and t + i < num_slots:
                        table[b, blk] = pg
            if t + i < num_slots and pg >= 0:
                slots[t + i] = pg * page + off
        used += -(-(o + n) // page) - have
        t += n
        lens.append(o + n)
        start.append(t)
    i32 = lambda a: np.asarray(a, np.int32)   # noqa: E731
    return table, i32(lens), i32(start), slots, i32([used])


def attention64(Q, cache, table, lens, start, scale, causal=True, window=0, out_eps=2.0 ** -11,
                weighted=False):
    """(O, lse, bound, lse_bound) in fp64 for Q fp64 [T][num_heads][D]; rows of no
    request NaN.

    `bound` (and lse_bound likewise) says how far a result of the documented arithmetic may be from O:
      the output's rounding                       out_eps |o|
      the weights' rounding to fp16               2^-11 sum p vs |c| / l, c the integer
                                                  that a kernel multiplies (code - 8 or
                                                  code - zero, the larger)
      weights below fp16's normal range           n 2^-21 max vs: a step of 2^-24 each,
                                                  halved, times |c| <= 8 or 15, where the
                                                  largest weight is at least 2^-1 max vs
      fp32 logits of D products, the zero term    dl = (D + 8) 2^-24 a scale, a = ks sum |q|
      and the scaling                             (code + zero); moves p by 2 dl at most
      fp32 sums over n keys (and exp2)            (n + 64) 2^-24 sum p vs (code + zero)
    With `weighted`, weights are taken as they are documented to be: multiplied by
    code - zero, and small ones rounded to steps of 2^-24 where the row's (or its
    part's) largest weight times step is at least 2^2, n 15 2^-27 max (p vs).
    """
    codes, scales, _ = cache
    pages, page = codes.shape[0], scales.shape[2]
    T, heads, D = Q.shape
    Hkv = scales.shape[1]
    group = heads // Hkv
    O = np.full(Q.shape, np.nan)
    lse = np.full(Q.shape[:2], np.nan)
    bound = np.zeros(Q.shape)
    lse_bound = np.zeros(Q.shape[:2])
    for b in range(len(lens)):
        kv = min(max(0, int(lens[b])), table.shape[1] * page)
        q0, q1 = int(start[b]), int(start[b + 1])
        pos = np.arange(kv)
        ids = table[b, pos // page].astype(np.int64)
        held = (ids >= 0) & (ids < pages)
        c, z, s, val = read(cache, D, np.where(held, ids, 0) * page + pos % page)
        for i in range(q1 - q0):
            last = kv - (q1 - q0) + i if causal else kv - 1
            seen = held & (pos <= last)
            if window:
                seen &= pos > last - window
            at = np.flatnonzero(seen)
            for j in range(heads):
                h = j // group
                q = Q[q0 + i, j]
                if not len(at):
                    O[q0 + i, j], lse[q0 + i, j] = 0.0, -np.inf
                    continue
                a = (val[0, at, h] @ q) * scale
                m = a.max()
                p = np.exp(a - m)
                l = p.sum()
                p /= l
                o = p @ val[1, at, h]
                O[q0 + i, j], lse[q0 + i, j] = o, m + np.log(l)
                mag = s[0, at, h] * ((c[0, at, h] + z[0, at, h][:, None] + 16) @ np.abs(q))
                dl = (D + 8) * 2.0 ** -24 * abs(scale) * mag.max()
                vs = s[1, at, h]
                cv = np.maximum(np.abs(c[1, at, h]), np.abs(c[1, at, h] - z[1, at, h][:, None]))
                n = len(at)
                lse_bound[q0 + i, j] = dl + (n + 64) * 2.0 ** -24 + 2.0 ** -22 * abs(lse[q0 + i, j])
                small = n * 2.0 ** -21 * vs.max()
                if weighted:
                    cv = np.abs(c[1, at, h] - z[1, at, h][:, None])
                    small = n * 15 * 2.0 ** -27 * (p * vs).max()
                bound[q0 + i, j] = (out_eps * np.abs(o) + 2.0 ** -11 * ((p * vs) @ cv) + small
                                    + 2 * dl * (p @ np.abs(val[1, at, h]))
                                    + (n + 64) * 2.0 ** -24 * ((p * vs) @ (c[1, at, h] + z[1, at, h][:, None] + 16)))
    return O, lse, bound, lse_bound
