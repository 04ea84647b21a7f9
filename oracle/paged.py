"""Serving over a paged K/V cache: request tables, multi-axis rotary
positions, cache append and attention over the pages (float64, loops).

Test infrastructure only; the CUDA library shares no code with it.
"""

from __future__ import annotations

import numpy as np


def extend(lens, add, table, free, n_free, page, max_rows):
    """Grants pages request by request until one does not fit; returns
    (lens, cu, slots, pos, n_free) and changes `table`."""
    n, width = table.shape
    n_free = min(max(int(n_free), 0), len(free))
    lens_out, cu = [int(x) for x in lens], [0]
    slots, pos = np.full(max_rows, -1, dtype=np.int64), np.zeros(max_rows, dtype=np.int64)
    rows, stopped = 0, False
    for r in range(n):
        ln, a = int(lens[r]), int(add[r])
        ok = not stopped and ln >= 0 and a >= 0
        if ok:
            have, end = -(-ln // page), -(-(ln + a) // page)
            ok = end <= width and end - have <= n_free and rows + a <= max_rows
        if not ok:
            stopped = True
            cu.append(rows)
            continue
        for j in range(have, end):
            n_free -= 1
            table[r, j] = free[n_free]
        for i in range(a):
            p = ln + i
            pos[rows + i] = p
            slots[rows + i] = table[r, p // page] * page + p % page
        rows += a
        lens_out[r] = ln + a
        cu.append(rows)
    return np.array(lens_out), np.array(cu), slots, pos, n_free


def release(lens, done, table, free, n_free, page):
    """Returns (lens, n_free) and changes `table` and `free`; entries below zero
    hold no page."""
    lens_out = [int(x) for x in lens]
    n_free = min(max(int(n_free), 0), len(free))
    for r in range(len(lens)):
        if not done[r]:
            continue
        for j in range(min(-(-max(int(lens[r]), 0) // page), table.shape[1])):
            if table[r, j] >= 0 and n_free < len(free):
                free[n_free] = table[r, j]
                n_free += 1
            table[r, j] = -1
        lens_out[r] = 0
    return np.array(lens_out), n_free


def pair_axes(sections, interleaved, restart):
    """(axis, exponent) of every rotated pair."""
    n = sum(sections)
    if not interleaved:
        order = [a for a, s in enumerate(sections) for _ in range(s)]
    else:
        left, order = list(sections), []
        while len(order) < n:
            for a in range(len(sections)):
                if left[a]:
                    order.append(a)
                    left[a] -= 1
    seen = [0] * len(sections)
    out = []
    for i, a in enumerate(order):
        out.append((a, seen[a] / sections[a] if restart else i / n))
        seen[a] += 1
    return out


def rope_axes(x, pos, sections, base=10000.0, interleaved=False, restart=False, adjacent=False, inverse=False):
    """x [rows, heads, d] float64, pos [axes, rows] whole numbers."""
    y = np.array(x, dtype=np.float64)
    n = sum(sections)
    for i, (a, e) in enumerate(pair_axes(sections, interleaved, restart)):
        ang = np.asarray(pos[a], dtype=np.float64) * float(base) ** -e
        c, s = np.cos(ang)[:, None], np.sin(ang)[:, None] * (-1.0 if inverse else 1.0)
        u, w = (2 * i, 2 * i + 1) if adjacent else (i, i + n)
        y[:, :, u], y[:, :, w] = x[:, :, u] * c - x[:, :, w] * s, x[:, :, w] * c + x[:, :, u] * s
    return y


def attention(q, k_cache, v_cache, table, cu, lens, causal=True, window=0, scale=None):
    """q [rows, H, d], caches [pages, page, Hkv, d] -> O [rows, H, d], L [rows, H]
    (rows of no request: NaN).  Only visible keys are touched."""
    rows, H, d = q.shape
    page, hkv = k_cache.shape[1], k_cache.shape[2]
    scale = 1.0 / np.sqrt(d) if scale is None else scale
    o, lse = np.full((rows, H, d), np.nan), np.full((rows, H), np.nan)
    for r in range(len(lens)):
        c0, c1, kv = int(cu[r]), int(cu[r + 1]), int(lens[r])
        for t in range(c0, c1):
            i = kv - (c1 - c0) + (t - c0)
            hi = min(kv, i + 1) if causal else kv
            lo = max(0, i - window + 1) if window else 0
            j = np.arange(lo, max(lo, hi))
            o[t], lse[t] = 0.0, -np.inf
            if len(j) == 0:
                continue
            pg = np.asarray(table[r])[j // page]
            for h in range(H):
                g = h // (H // hkv)
                kk = np.asarray(k_cache[pg, j % page, g], dtype=np.float64)
                vv = np.asarray(v_cache[pg, j % page, g], dtype=np.float64)
                s = scale * (kk @ np.asarray(q[t, h], dtype=np.float64))
                m = s.max()
                w = np.exp(s - m)
                lse[t, h] = m + np.log(w.sum())
                o[t, h] = (w / w.sum()) @ vv
    return o, lse
