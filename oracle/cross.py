"""Cross attention of packed sequences in float64 (loops over sequences and
heads): bias of the relative position by buckets, dropout from Philox4x32,
gradients by the formulas.

Test infrastructure only; the CUDA library shares no code with it.
"""

from __future__ import annotations

import math

import numpy as np


def bucket_starts(per, max_distance):
    e = per // 2
    return list(range(e)) + [math.ceil(e * (max_distance / e) ** (t / (per - e)) * (1 - 1e-12)) for t in range(per - e)]


def buckets(rel, n, max_distance, both):
    """Bucket of every relative position (key - query) of an integer array."""
    per = n // 2 if both else n
    starts = bucket_starts(per, max_distance)
    away = np.abs(rel) if both else np.maximum(-rel, 0)
    out = np.zeros(rel.shape, dtype=np.int64)
    for b, s in enumerate(starts):
        out[away >= s] = b
    return out + (per * (rel > 0) if both else 0)


def philox(ctr, key, rounds=7):
    """Philox4x32: four arrays of counter words and two of key words (Python or numpy uint64 below 2^32)."""
    m32 = np.uint64(0xFFFFFFFF)
    c = [np.asarray(x, dtype=np.uint64) for x in ctr]
    k = [int(x) for x in key]
    for _ in range(rounds):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> np.uint64(32)) ^ c[1] ^ np.uint64(k[0]), b & m32, (a >> np.uint64(32)) ^ c[3] ^ np.uint64(k[1]), a & m32]
        k = [(k[0] + 0x9E3779B9) % 2 ** 32, (k[1] + 0xBB67AE85) % 2 ** 32]
    return c


def keep(nq, nk, seq_head, p, seed, offset):
    """Which pairs dropout keeps, and the probability that it drops with."""
    cut = round(p * 32768)  # halves to even
    i, j = np.meshgrid(np.arange(nq), np.arange(nk), indexing="ij")
    words = philox((j // 8, i, np.full_like(i, seq_head), np.full_like(i, offset % 2 ** 32)),
                   (seed % 2 ** 32, (seed >> 32) % 2 ** 32))
    e = j % 8
    word = np.choose(e // 2, words)
    piece = (word >> (16 * (e % 2)).astype(np.uint64)) & np.uint64(0x7FFF)
    return piece >= cut, cut / 32768


def attention(q, k, v, seqs, do=None, causal=False, scale=None, table=None, rel=None, p=0.0, rng=(0, 0)):
    """seqs: (first query row, queries, first key row, keys) of every sequence.  Returns a dict
    with o, lse and, with do, dq, dk, dv and dtable; rows of no sequence hold zeros.  mag_* are the same sums
    of magnitudes, which error bounds go by."""
    H, Hkv, d = q.shape[1], k.shape[1], q.shape[2]
    scale = 1 / math.sqrt(d) if scale is None else scale
    out = dict(o=np.zeros_like(q), lse=np.zeros(q.shape[:2]), mag_o=np.zeros_like(q), top=0.0)
    if do is not None:
        for m in ("", "mag_"):
            out.update({m + "dq": np.zeros_like(q), m + "dk": np.zeros_like(k), m + "dv": np.zeros_like(v)})
            if table is not None:
                out[m + "dtable"] = np.zeros_like(table)
    for b, (q0, nq, k0, nk) in enumerate(seqs):
        if nq == 0:
            continue
        out["lse"][q0:q0 + nq] = -np.inf
        if nk == 0:
            continue
        x = np.arange(nk)[None] - (np.arange(nq)[:, None] + nk - nq)
        see = x <= 0 if causal else np.ones(x.shape, dtype=bool)
        if table is not None:
            bk = buckets(x, *rel)
        for h in range(H):
            g = h // (H // Hkv)
            qh, kh, vh = q[q0:q0 + nq, h], k[k0:k0 + nk, g], v[k0:k0 + nk, g]
            s = scale * (qh @ kh.T)
            ok = see
            if table is not None:
                s = s + table[bk, h]
                ok = see & (table[bk, h] >= -1e30)
            s = np.where(ok, s, -np.inf)
            top = np.max(s, axis=1)
            some = top > -np.inf
            e = np.exp(s - np.where(some, top, 0)[:, None])
            total = e.sum(1)
            with np.errstate(divide="ignore"):
                out["lse"][q0:q0 + nq, h] = np.where(some, top + np.log(total), -np.inf)
            prob = e / np.where(some, total, 1)[:, None]
            mask = np.ones(x.shape)
            if p > 0:
                kept, pe = keep(nq, nk, b * H + h, p, *rng)
                mask = kept / (1 - pe)
            o = (prob * mask) @ vh
            out["o"][q0:q0 + nq, h] = o
            out["mag_o"][q0:q0 + nq, h] = (prob * mask) @ np.abs(vh)
            out["top"] = max(out["top"], float(np.max(np.abs(s[ok]), initial=0)))
            if do is None:
                continue
            dh = do[q0:q0 + nq, h]
            ds = prob * (mask * (dh @ vh.T) - (dh * o).sum(1)[:, None])
            out["dq"][q0:q0 + nq, h] = scale * ds @ kh
            out["dk"][k0:k0 + nk, g] += scale * ds.T @ qh
            out["dv"][k0:k0 + nk, g] += (prob * mask).T @ dh
            if table is not None:
                for t in range(len(table)):
                    out["dtable"][t, h] += ds[bk == t].sum()
            mds = prob * (mask * (np.abs(dh) @ np.abs(vh).T) + (np.abs(dh) * out["mag_o"][q0:q0 + nq, h]).sum(1)[:, None])
            out["mag_dq"][q0:q0 + nq, h] = scale * mds @ np.abs(kh)
            out["mag_dk"][k0:k0 + nk, g] += scale * mds.T @ np.abs(qh)
            out["mag_dv"][k0:k0 + nk, g] += (prob * mask).T @ np.abs(dh)
            if table is not None:
                for t in range(len(table)):
                    out["mag_dtable"][t, h] += mds[bk == t].sum()
    return out
