"""Attention of encoder-decoder and bias-position models: cases, plain forms and work.

Three operators on the attention of packed query sequences over packed key
sequences of other lengths (forward, and backward for training):

* ``cross``: the attention itself: a decoder's queries over an encoder's states, from one token up;
* ``bias``:  with a learned bias of the relative position by buckets, and the gradient of its table;
* ``drop``:  with dropout of the probabilities from a counter-based generator, whose mask is never stored.

With ``own`` false, ``run`` computes them from elementary torch operations in 32
bits (long sums and bucket borders in 64); with ``own`` true it calls the library.

Definitions.  Sequence b has nq queries and nk keys.  With causal, query i sees
the keys j <= i + nk - nq (the ends are aligned), else all.  With buckets, the
score of (i, j) is s = scale q_i . k_j + table[bucket(j - (i + nk - nq)), h].  With
dropout, the probability of (i, j) is multiplied by keep(i, j) / (1 - p): of
Philox4x32 with 7 rounds, counter (j // 8, i, b * heads + h, offset) and the
seed as its key, piece j % 8 is the low 15 bits of half (j % 2) of word
(j % 8) // 2, and keep is piece >= round(p * 2^15); 1 - p is taken after that rounding.
"""

import math

import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one sentence answered token by token against its encoder's states: latency
        dict(name="cross_one_token", op="cross", seqs=1, nq=1, nk=777, spread=0.0, hq=32, hkv=8, d=128, dtype="bf16"),
        # a decode batch over encoder states whose lengths are spread like the packed benchmark's
        dict(name="cross_decode_batch", op="cross", seqs=64, nq=1, nk=1808, spread=1.0, hq=32, hkv=8, d=128, dtype="bf16",
             padded=True),
        # a training step's cross attention: ragged targets over ragged sources, K and V halves of one projection
        dict(name="cross_train", op="cross", seqs=16, nq=509, nk=2048, spread=0.5, hq=32, hkv=8, d=128, dtype="bf16",
             train=True, fused=True),
        # a long question over a very long context, scored in one pass
        dict(name="cross_long", op="cross", seqs=1, nq=4096, nk=32768, spread=0.0, hq=32, hkv=8, d=128, dtype="bf16"),
        # short pairs in float32, as a small model's tests and fine-tuning run them
        dict(name="cross_f32", op="cross", seqs=5, nq=100, nk=333, spread=0.5, hq=8, hkv=2, d=64, dtype="f32", train=True),
        # a bidirectional encoder's training step: self attention under a bias by buckets
        dict(name="bias_encoder", op="bias", seqs=8, nq=0, nk=1808, spread=0.5, hq=16, hkv=16, d=64, dtype="bf16",
             buckets=32, distance=128, both=True, train=True),
        # its decoder answering: one token each over cached keys, the bias looking back
        dict(name="bias_one_token", op="bias", seqs=32, nq=1, nk=1024, spread=0.5, hq=16, hkv=16, d=64, dtype="bf16",
             buckets=32, distance=128, both=False, causal=True),
        # short sentences in float32, the smallest training call
        dict(name="bias_f32", op="bias", seqs=3, nq=0, nk=77, spread=0.3, hq=4, hkv=4, d=64, dtype="f32", buckets=32,
             distance=128, both=True, train=True),
        # a decoder's causal self attention with dropout, whole sequences
        dict(name="drop_causal", op="drop", seqs=2, nq=0, nk=4096, spread=0.0, hq=32, hkv=8, d=128, dtype="bf16", p=0.1,
             causal=True, train=True),
        # many short ragged pairs with dropout: fine-tuning on sentences
        dict(name="drop_short", op="drop", seqs=32, nq=200, nk=300, spread=0.5, hq=16, hkv=16, d=64, dtype="bf16", p=0.1,
             train=True),
        # bias and dropout together, as a decoder of this kind trains: causal, ragged
        dict(name="drop_bias", op="drop", seqs=6, nq=0, nk=1500, spread=0.5, hq=16, hkv=16, d=64, dtype="bf16", p=0.1,
             causal=True, buckets=32, distance=128, both=False, train=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    op = rng.choice(["cross", "bias", "drop"])
    hq, hkv = rng.choice([(32, 8), (32, 32), (32, 4), (28, 4), (8, 1), (16, 16), (16, 2), (4, 2), (6, 6), (40, 8)])
    c = dict(op=op, hq=hq, hkv=hkv, d=rng.choice([128, 64]), dtype=rng.choice(["bf16", "bf16", "bf16", "f32"]),
             spread=rng.choice([0.0, 0.5, 1.0]), fused=rng.random() < 0.3, padded=rng.random() < 0.3)
    c["train"] = rng.random() < 0.5
    most = 2 ** (26 if c["dtype"] == "f32" else 30) // hq  # pairs of a head
    form = rng.choice(["one", "few", "self", "cross", "cross"])
    c["seqs"] = _log_int(rng, 1, 128 if form in ("one", "few") else 32)
    if form in ("one", "few"):
        c["nq"] = 1 if form == "one" else rng.randint(2, 9)
        c["train"] = c["train"] and form == "few"
        c["nk"] = _log_int(rng, 1, min(65536, most // (c["seqs"] * c["nq"] * 4), 2 ** 19 // c["seqs"] * 8 // hkv))
    elif form == "self":
        c["nq"], c["nk"] = 0, _log_int(rng, 1, int(math.sqrt(most / c["seqs"] / 4)))
    else:
        c["nq"] = _log_int(rng, 1, 4096)
        c["nk"] = _log_int(rng, 1, min(16384, max(2, most // (c["seqs"] * c["nq"] * 4))))
    c["causal"] = form != "cross" and rng.random() < 0.5 or rng.random() < 0.1
    if op == "bias" or (op == "drop" and rng.random() < 0.3):
        c["both"] = rng.random() < 0.5
        c["buckets"] = 2 * rng.choice([2, 4, 8, 16, 16, 32]) if c["both"] else rng.choice([2, 5, 16, 32, 32, 64])
        c["distance"] = _log_int(rng, c["buckets"], 600)
        if c["dtype"] == "f32" and c["train"]:
            # A table's gradient sums dS, whose rows sum to 0: with n keys and all but w of them in one bucket it
            # loses a factor of sqrt(n / w), which float32 P cannot give back.
            c["buckets"], c["distance"] = max(c["buckets"], 16), max(c["distance"], 16, c["nk"] // 16)
    if op == "drop":
        c["p"] = rng.choice([0.1, 0.1, rng.uniform(0.0, 0.6)])
    return c


# ------------------------------------------------------------------ shapes ---
def _lengths(case):
    """Queries and keys of every sequence: a part of the case, the same for every seed."""
    rng = np.random.default_rng(4321)
    n = case["seqs"]

    def some(mean):
        x = np.full(n, mean, dtype=np.float64)
        if case["spread"] > 0:
            x = np.minimum(x * np.exp(case["spread"] * np.clip(rng.standard_normal(n), -2.5, 2.5)), 2 * mean)
        return np.maximum(0 if mean > 1 and n > 2 else 1, np.round(x)).astype(np.int64)

    nk = some(case["nk"])
    if case["nq"] == 0:
        nq = nk.copy()
    elif case["nq"] < 10:
        nq = np.full(n, case["nq"], dtype=np.int64)
    else:
        nq = some(case["nq"])
    return nq, nk


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(g, shape, dtype):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).to(dtype)


def _i32(x):
    return torch.tensor(np.asarray(x, dtype=np.int32), device=DEV)


def prepare(case, seed):
    g = _gen(seed)
    dt, hq, hkv, d = TYPES[case["dtype"]], case["hq"], case["hkv"], case["d"]
    nq, nk = _lengths(case)
    rows_q = int(nq.sum())
    starts_q = np.concatenate([[0], np.cumsum(nq)])
    if case.get("padded"):  # every source in a place of the longest one's size
        starts_k = np.arange(len(nk) + 1) * int(nk.max())
    else:
        starts_k = np.concatenate([[0], np.cumsum(nk)])
    rows_k = int(starts_k[-1])
    s = dict(case=case, nq=nq.tolist(), nk=nk.tolist(), q0=starts_q.tolist(), k0=starts_k.tolist())
    s["q"] = _randn(g, (rows_q, hq, d), dt)
    if case.get("fused"):
        kv = _randn(g, (rows_k, 2, hkv, d), dt)
        s["k"], s["v"] = kv[:, 0], kv[:, 1]
    else:
        s["k"], s["v"] = _randn(g, (rows_k, hkv, d), dt), _randn(g, (rows_k, hkv, d), dt)
    s["cu_q"], s["cu_k"] = _i32(starts_q), _i32(starts_k)
    s["len_k"] = _i32(nk) if case.get("padded") else None
    if case.get("train"):
        s["do"] = _randn(g, (rows_q, hq, d), dt)
    s["table"] = _randn(g, (case["buckets"], hq), dt) if case.get("buckets") else None
    if case.get("p") is not None:
        s["seed"], s["offset"] = (seed * 0x9E3779B97F4A7C15 + 12345) % 2 ** 63, seed % 1000 + 7
        s["rng"] = torch.tensor([s["seed"], s["offset"]], dtype=torch.int64, device=DEV)
    else:
        s["rng"] = None
    if own:
        from tile_attention_lse_gb300 import api
        rel = api.RelBuckets(case["buckets"], case["distance"], case["both"]) if case.get("buckets") else None
        s["plan"] = api.CrossProblem(heads_q=hq, heads_kv=hkv, head_dim=d, dtype=dt, causal=case.get("causal", False),
                                     max_q=int(nq.max()), rel=rel, dropout=case.get("p") or 0.0)
        s["ws"] = api.cross_workspace(s["plan"], len(nq), rows_q, rows_k, backward=bool(case.get("train")))
    return s


# --------------------------------------------------------------------- run ---
def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(s):
    from tile_attention_lse_gb300 import api
    at = dict(len_k=s["len_k"], bias=s["table"], rng=s["rng"], ws=s["ws"])
    if not s["case"].get("train"):
        o, lse = api.cross_attn_fwd(s["plan"], s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], **at)
        return dict(o=o, lse=lse)
    # rest: what o lost to its rounding, where the table's gradient needs it
    o, lse, rest = api.cross_attn_fwd(s["plan"], s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], for_backward=True, **at)
    dq, dk, dv, dtable = api.cross_attn_bwd(s["plan"], s["q"], s["k"], s["v"], o, lse, s["do"], s["cu_q"], s["cu_k"],
                                            rest=rest, **at)
    out = dict(o=o, lse=lse, dq=dq, dk=dk, dv=dv)
    if dtable is not None:
        out["dtable"] = dtable
    return out


def _bucket_row(case, lo, hi):
    """Buckets of the relative positions lo .. hi (host)."""
    both, n = case["both"], case["buckets"]
    per = n // 2 if both else n
    near = per // 2
    starts = list(range(near))
    for t in range(per - near):
        x = near * (case["distance"] / near) ** (t / (per - near)) if near else float(t)
        starts.append(math.ceil(x * (1 - 1e-12)))
    starts = np.array(starts)
    rel = np.arange(lo, hi + 1)
    away = np.abs(rel) if both else np.maximum(-rel, 0)
    row = np.searchsorted(starts, away, side="right") - 1
    return row + (per * (rel > 0) if both else 0)


M32 = 0xFFFFFFFF


def _philox(c0, c1, c2, c3, k0, k1):
    """Philox4x32 with 7 rounds on int64 tensors that hold 32-bit words."""
    for _ in range(7):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = ((b >> 32) & M32) ^ c1 ^ k0, b & M32, ((a >> 32) & M32) ^ c3 ^ k1, a & M32
        k0, k1 = (k0 + 0x9E3779B9) & M32, (k1 + 0xBB67AE85) & M32
    return c0, c1, c2, c3


def _keep(s, b, h0, h1, nq, nk):
    case = s["case"]
    block = torch.arange((nk + 7) // 8, device=DEV)[None, None, :]
    i = torch.arange(nq, device=DEV)[None, :, None]
    bh = (b * case["hq"] + torch.arange(h0, h1, device=DEV))[:, None, None]
    shape = (h1 - h0, nq, block.shape[2])
    c = [x.expand(shape) for x in (block, i, bh)] + [torch.full(shape, s["offset"] & M32, device=DEV)]
    words = _philox(*c, s["seed"] & M32, s["seed"] >> 32)
    pieces = [(w >> sh) & 0x7FFF for w in words for sh in (0, 16)]
    return torch.stack(pieces, -1).flatten(2)[..., :nk] >= round(case["p"] * 32768)


def _run_plain(s):
    case = s["case"]
    hq, hkv, d, train = case["hq"], case["hkv"], case["d"], case.get("train")
    grp = hq // hkv
    dt, scale = s["q"].dtype, 1.0 / math.sqrt(d)
    # a float32 table's gradient is a long sum of what nearly cancels
    wide_t = torch.float64 if train and case.get("buckets") and case["dtype"] == "f32" else torch.float32
    o = torch.empty_like(s["q"])
    lse = torch.empty(s["q"].shape[:2], dtype=torch.float32, device=DEV)
    if train:
        dq = torch.empty_like(s["q"])
        dk, dv = (torch.zeros(s["k"].shape, dtype=dt, device=DEV) for _ in range(2))
        dtable = torch.zeros((case["buckets"], hq), dtype=torch.float64, device=DEV) if case.get("buckets") else None
    p_eff = round(case["p"] * 32768) / 32768 if case.get("p") is not None else 0.0
    for b, (nq, nk) in enumerate(zip(s["nq"], s["nk"])):
        if nq == 0:
            continue
        q0, k0 = s["q0"][b], s["k0"][b]
        if case.get("buckets") and nk > 0:
            row = torch.tensor(_bucket_row(case, -(nk - 1), nq - 1), device=DEV)  # index: rel + nk - 1
            rel = torch.arange(nk, device=DEV)[None] - (torch.arange(nq, device=DEV)[:, None] + nk - nq) + nk - 1
        heads = max(1, min(hkv, int(2 ** 30 // max(1, nq * nk * grp))))  # kv-heads at once
        for g0 in range(0, hkv, heads):
            g1 = min(hkv, g0 + heads)
            h0, h1 = g0 * grp, g1 * grp
            q = s["q"][q0:q0 + nq, h0:h1].to(wide_t).permute(1, 0, 2).reshape(g1 - g0, grp * nq, d)
            k, v = (s[x][k0:k0 + nk, g0:g1].to(wide_t).permute(1, 0, 2) for x in ("k", "v"))
            x = (q @ k.transpose(1, 2)).reshape(h1 - h0, nq, nk) * scale
            if case.get("buckets") and nk > 0:
                x = x + s["table"][:, h0:h1].to(wide_t).t()[:, row][:, rel]
            if case.get("causal"):
                hide = torch.arange(nk, device=DEV)[None] > torch.arange(nq, device=DEV)[:, None] + nk - nq
                x = x.masked_fill(hide, -math.inf)
            if nk > 0:
                top = x.amax(2, keepdim=True).clamp(min=-3e38)
                e = torch.exp(x - top)
                total = e.sum(2, keepdim=True)
                prob = e / total.clamp(min=1e-30)
                lse[q0:q0 + nq, h0:h1] = torch.where(total > 0, top + torch.log(total), -math.inf)[..., 0].t().float()
            else:
                prob = x
                lse[q0:q0 + nq, h0:h1] = -math.inf
            used = prob
            if case.get("p") is not None and nk > 0:
                factor = _keep(s, b, h0, h1, nq, nk).to(wide_t) / (1 - p_eff)
                used = prob * factor
            wide = used.reshape(g1 - g0, grp * nq, nk)
            res = (wide @ v).reshape(h1 - h0, nq, d)
            o[q0:q0 + nq, h0:h1] = res.permute(1, 0, 2).to(dt)
            if not train:
                continue
            do = s["do"][q0:q0 + nq, h0:h1].to(wide_t).permute(1, 0, 2)
            dow = do.reshape(g1 - g0, grp * nq, d)
            dp = (dow @ v.transpose(1, 2)).reshape(h1 - h0, nq, nk)
            if case.get("p") is not None and nk > 0:
                dp = dp * factor
            ds = prob * (dp - (do * res).sum(2, keepdim=True))
            dsw = ds.reshape(g1 - g0, grp * nq, nk)
            dq[q0:q0 + nq, h0:h1] = ((dsw @ k) * scale).reshape(h1 - h0, nq, d).permute(1, 0, 2).to(dt)
            dk[k0:k0 + nk, g0:g1] = ((dsw.transpose(1, 2) @ q) * scale).permute(1, 0, 2).to(dt)
            dv[k0:k0 + nk, g0:g1] = (wide.transpose(1, 2) @ dow).permute(1, 0, 2).to(dt)
            if dtable is not None and nk > 0:
                # sums of the diagonals: rows turned about and shifted so that column r holds rel + nk - 1 = r
                z = torch.nn.functional.pad(ds, (0, nq)).flip(1).flatten(1)[:, :nq * (nk + nq - 1)]
                diag = z.reshape(h1 - h0, nq, nk + nq - 1).sum(1, dtype=torch.float64)
                dtable[:, h0:h1].index_add_(0, row, diag.t())
    out = dict(o=o, lse=lse)
    if train:
        out.update(dq=dq, dk=dk, dv=dv)
        if dtable is not None:
            out["dtable"] = dtable.to(dt)
    return out


# -------------------------------------------------------------------- work ---
def work(case):
    nq, nk = _lengths(case)
    size, hq, hkv, d = (2 if case["dtype"] == "bf16" else 4), case["hq"], case["hkv"], case["d"]
    pairs = 0
    for a, b in zip(nq.tolist(), nk.tolist()):
        if case.get("causal"):  # row i sees max(0, min(b, i + b - a + 1)) keys
            m = min(a, b)
            pairs += m * (2 * b - m + 1) // 2
        else:
            pairs += a * b
    rows_q, rows_k = int(nq.sum()), int(nk.sum())
    moved = rows_q * hq * (2 * d * size + 4) + 2 * rows_k * hkv * d * size + (case.get("buckets") or 0) * hq * size
    flops = 4.0 * d * hq * pairs
    if case.get("train"):  # dO read, dQ, dK, dV and the table's gradient written; five products on top of the two
        moved += rows_q * hq * 2 * d * size + 2 * rows_k * hkv * d * size + (case.get("buckets") or 0) * hq * size
        flops += 10.0 * d * hq * pairs
    return {"bytes": float(moved), "flops": flops}


# ------------------------------------------------------------------- exact ---
def _mul_high_low(a, m):
    """High and low 32 bits of a * m from 16-bit parts, no product above 2^33."""
    al, ah, ml, mh = a & 0xFFFF, a >> 16, m & 0xFFFF, m >> 16
    low = al * ml
    mid1, mid2 = ah * ml, al * mh
    carry = (low >> 16) + (mid1 & 0xFFFF) + (mid2 & 0xFFFF)
    return ah * mh + (mid1 >> 16) + (mid2 >> 16) + (carry >> 16), ((carry & 0xFFFF) << 16) | (low & 0xFFFF)


def _exact_keep(case, s, b, h, nq, nk):
    i, j = torch.meshgrid(torch.arange(nq, device=DEV), torch.arange(0, nk, 8, device=DEV) // 8, indexing="ij")
    ctr = [j, i, torch.full_like(i, b * case["hq"] + h), torch.full_like(i, s["offset"])]
    key = [s["seed"] % 2 ** 32, s["seed"] // 2 ** 32]
    for _ in range(7):
        h0, l0 = _mul_high_low(ctr[0], 0xD2511F53)
        h1, l1 = _mul_high_low(ctr[2], 0xCD9E8D57)
        ctr = [h1 ^ ctr[1] ^ key[0], l1, h0 ^ ctr[3] ^ key[1], l0]
        key = [(key[0] + 0x9E3779B9) % 2 ** 32, (key[1] + 0xBB67AE85) % 2 ** 32]
    out = torch.empty((nq, j.shape[1] * 8), dtype=torch.bool, device=DEV)
    for e in range(8):
        word = ctr[e // 2] // (65536 if e % 2 else 1)
        out[:, e::8] = word % 32768 >= round(case["p"] * 32768)
    return out[:, :nk]


def exact(case, seed):
    if work(case)["flops"] > 5e12:
        return None
    s = prepare(case, seed)
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    train = bool(case.get("train"))
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device=DEV)
    grads = {x: torch.zeros(s[x].shape, dtype=torch.float64, device=DEV) for x in ("q", "k", "v")} if train else None
    dtable = torch.zeros_like(s["table"], dtype=torch.float64) if train and s["table"] is not None else None
    for b, (nq, nk) in enumerate(zip(s["nq"], s["nk"])):
        if nq == 0 or nk == 0:
            continue
        at_q, at_k = slice(s["q0"][b], s["q0"][b] + nq), slice(s["k0"][b], s["k0"][b] + nk)
        i, j = torch.arange(nq, device=DEV)[:, None], torch.arange(nk, device=DEV)[None]
        rel = j - (i + nk - nq)
        if s["table"] is not None:
            per = case["buckets"] // 2 if case["both"] else case["buckets"]
            near = per // 2
            away = rel.abs() if case["both"] else (-rel).clamp(min=0)
            step = torch.log(away.clamp(min=1).double() / near) / math.log(case["distance"] / near) * (per - near) \
                if case["distance"] > near and near else torch.full(away.shape, float(per), dtype=torch.float64, device=DEV)
            far = near + torch.floor(step + 1e-9).long().clamp(max=per - near - 1)
            bucket = torch.where(away < near, away, far) + (per * (rel > 0).long() if case["both"] else 0)
        for h in range(hq):
            g = h // (hq // hkv)
            q, k, v = s["q"][at_q, h].double(), s["k"][at_k, g].double(), s["v"][at_k, g].double()
            leaves = [q, k, v]
            if s["table"] is not None:
                leaves.append(s["table"][:, h].double())
            if train:
                for x in leaves:
                    x.requires_grad_(True)
            score = q @ k.t() / math.sqrt(d)
            if s["table"] is not None:
                score = score + leaves[3][bucket]
            sees = torch.ones_like(rel, dtype=torch.bool) if not case.get("causal") else rel <= 0
            some = sees.any(1)
            score = score.masked_fill(~sees, -math.inf)
            lse[at_q, h] = torch.logsumexp(score.detach(), 1)
            prob = torch.softmax(score.masked_fill(~some[:, None], 0.0), 1) * some[:, None]
            if case.get("p") is not None:
                prob = prob * _exact_keep(case, s, b, h, nq, nk) / (1 - round(case["p"] * 32768) / 32768)
            res = prob @ v
            o[at_q, h] = res.detach()
            if train:
                got = torch.autograd.grad(res, leaves, s["do"][at_q, h].double())
                grads["q"][at_q, h] = got[0]
                grads["k"][at_k, g] += got[1]
                grads["v"][at_k, g] += got[2]
                if dtable is not None:
                    dtable[:, h] += got[3]
    out = dict(o=o, lse=lse)
    if train:
        out.update(dq=grads["q"], dk=grads["k"], dv=grads["v"])
        if dtable is not None:
            out["dtable"] = dtable
    return out
