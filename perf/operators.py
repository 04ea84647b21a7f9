"""Serving operators over a paged K/V cache: cases, plain forms and work.

Four operators that a serving step runs one after the other:

* ``extend``: block tables, slot maps and positions from the lengths of the requests;
* ``rope``: rotary positions with several axes on Q and K (and the transpose, a gradient);
* ``append``: new K/V rows into the pages of the cache, K and Q rotated on the way;
* ``attn``: attention of each request's new tokens over its pages.

With ``own`` false, ``run`` computes them from elementary torch operations in 32
bits (angles in 64); with ``own`` true it calls the library.
"""

import math

import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one request answering token by token on a short context: latency
        dict(name="attn_one_token", op="attn", reqs=1, new="one", ctx=777, spread=0.0, hq=32, hkv=8, d=128, page=16,
             dtype="bf16", window=0, causal=True),
        # a decode batch whose context lengths are spread like the packed benchmark's lengths
        dict(name="attn_decode_batch", op="attn", reqs=64, new="one", ctx=1808, spread=1.0, hq=32, hkv=8, d=128, page=64,
             dtype="bf16", window=0, causal=True),
        # few requests on the longest context: the key axis is split
        dict(name="attn_decode_long", op="attn", reqs=4, new="one", ctx=131072, spread=0.0, hq=32, hkv=8, d=128, page=128,
             dtype="bf16", window=0, causal=True),
        # one chunk of a long prompt over what is cached already
        dict(name="attn_chunk", op="attn", reqs=1, new="all", tokens=2048, ctx=30720, spread=0.0, hq=32, hkv=8, d=128, page=64,
             dtype="bf16", window=0, causal=True),
        # single tokens and chunks of odd lengths in one batch, with a sliding window
        dict(name="attn_mixed_window", op="attn", reqs=24, new="mixed", tokens=509, ctx=6000, spread=0.5, hq=32, hkv=8, d=128,
             page=32, dtype="bf16", window=4096, causal=True),
        # float32, head_dim 64, short odd chunks
        dict(name="attn_f32_short", op="attn", reqs=7, new="all", tokens=33, ctx=1000, spread=0.7, hq=8, hkv=2, d=64, page=16,
             dtype="f32", window=0, causal=True),
        # Q and K of a training sequence of images and text, rotated along time, height and width
        dict(name="rope_train", op="rope", tokens=32768, hq=32, hkv=8, d=128, sections="16,24,24", interleaved=False,
             restart=False, adjacent=False, inverse=False, dtype="bf16"),
        # the gradient's way back on a short odd sequence, adjacent pairs, frequencies of each axis from its own start
        dict(name="rope_back_f32", op="rope", tokens=1021, hq=4, hkv=2, d=64, sections="8,12,12", interleaved=False,
             restart=True, adjacent=True, inverse=True, dtype="f32"),
        # a decode batch's new tokens
        dict(name="append_decode", op="append", tokens=64, hq=32, hkv=8, d=128, page=64, sections="64", interleaved=False,
             restart=False, adjacent=False, dtype="bf16"),
        # the chunk of a prompt with image tokens
        dict(name="append_chunk", op="append", tokens=8191, hq=32, hkv=8, d=128, page=16, sections="24,20,20", interleaved=True,
             restart=False, adjacent=False, dtype="bf16"),
        # one decode step's tables
        dict(name="extend_decode", op="extend", reqs=256, add=1, ctx=2000, page=16, width=1024, short=False),
        # prompts of odd lengths that arrive together, more than the free pages hold
        dict(name="extend_prompts", op="extend", reqs=61, add=1500, ctx=300, page=32, width=512, short=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "attn", "rope", "append", "extend"])
    page = rng.choice([8, 16, 32, 64, 128, 256])
    hq, hkv = rng.choice([(32, 8), (32, 32), (32, 4), (28, 4), (8, 1), (16, 2), (4, 2), (6, 6), (40, 8)])
    d = rng.choice([128, 128, 64])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op == "attn":
        new = rng.choice(["one", "one", "few", "all", "mixed"])
        tokens = {"one": 1, "few": rng.randint(2, 8)}.get(new) or _log_int(rng, 9, 2048)
        reqs = _log_int(rng, 1, 128 if new in ("one", "few") else 24)
        # the drawn cost stays within the listed chunk's and the longest decode's
        most = min(131072, int(2 ** 31 / (reqs * hq * tokens)) - tokens, int(2 ** 19 / reqs * 8 / hkv))
        if dtype == "f32":
            most = min(most, int(2 ** 28 / (reqs * hq * tokens)) - tokens)
        ctx = _log_int(rng, 1, max(2, most // 3))
        return dict(op=op, reqs=reqs, new=new, tokens=tokens, ctx=ctx, spread=rng.choice([0.0, 0.5, 1.0]), hq=hq, hkv=hkv, d=d,
                    page=page, dtype=dtype, window=rng.choice([0, 0, _log_int(rng, 1, 5000)]), causal=rng.random() < 0.85)
    half = d // 2
    a = 8 * rng.randint(0, half // 16)
    sections = rng.choice(["%d" % half, "%d,%d" % (half - 8, 8), "%d,%d,%d" % (half - 2 * (half // 4 + half // 16),
                           half // 4 + half // 16, half // 4 + half // 16), "%d,%d,%d,%d" % (half // 4, half // 4, half // 4, half // 4),
                           "%d" % max(8, half - a)])
    if op == "rope":
        return dict(op=op, tokens=_log_int(rng, 1, 32768), hq=hq if hq < 40 else 32, hkv=min(hkv, 8), d=d, sections=sections,
                    interleaved=rng.random() < 0.5, restart=rng.random() < 0.3, adjacent=rng.random() < 0.3,
                    inverse=rng.random() < 0.5, dtype=rng.choice(["bf16", "f32"]) if hq < 28 else "bf16")
    if op == "append":
        return dict(op=op, tokens=_log_int(rng, 1, 8192), hq=hq if hq < 40 else 32, hkv=hkv, d=d, page=page, sections=sections,
                    interleaved=rng.random() < 0.5, restart=rng.random() < 0.3, adjacent=rng.random() < 0.3, dtype=dtype)
    reqs = _log_int(rng, 1, 600)
    add = rng.choice([1, _log_int(rng, 1, max(2, 60000 // reqs))])
    ctx = _log_int(rng, 1, 8000)
    return dict(op=op, reqs=reqs, add=add, ctx=ctx, page=page, width=-(-(4 * ctx + 2 * add + 8) // page), short=rng.random() < 0.3)


# ------------------------------------------------------------------ shapes ---
def _lengths(case):
    """New tokens and cached lengths (before them) of every request: a part of the case, the same for every seed."""
    rng = np.random.default_rng(1234)
    n = case["reqs"]
    full = case.get("tokens", 1)
    if case["new"] == "one":
        new = np.ones(n, dtype=np.int64)
    elif case["new"] in ("few", "all"):
        new = np.full(n, full, dtype=np.int64)
        if case["new"] == "all" and n > 1:
            new = np.maximum(1, (full * rng.uniform(0.3, 1.0, n)).astype(np.int64))
            new[0] = full
    else:  # one request in six brings a chunk
        new = np.where(np.arange(n) % 6 == 2, np.maximum(1, (full * rng.uniform(0.5, 1.0, n)).astype(np.int64)), 1)
        new[min(2, n - 1)] = full
    ctx = np.full(n, case["ctx"], dtype=np.float64)
    if case["spread"] > 0:
        ctx = np.minimum(ctx * np.exp(case["spread"] * np.clip(rng.standard_normal(n), -2.5, 2.5)) , 3 * case["ctx"])
    old = np.maximum(0, np.round(ctx)).astype(np.int64)
    if case["new"] == "one":
        old = np.maximum(0, old - 1)
    return new, old


def _sections(case):
    return [int(x) for x in case["sections"].split(",")]


def _axis_and_step(case):
    """Axis and frequency exponent of every pair."""
    sec = _sections(case)
    n = sum(sec)
    if case["interleaved"]:
        left, axis = list(sec), []
        while len(axis) < n:
            for a in range(len(sec)):
                if left[a] > 0:
                    left[a] -= 1
                    axis.append(a)
    else:
        axis = [a for a, s in enumerate(sec) for _ in range(s)]
    if case["restart"]:
        seen, step = [0] * len(sec), []
        for a in axis:
            step.append(seen[a] / sec[a])
            seen[a] += 1
    else:
        step = [i / n for i in range(n)]
    return axis, step


def _grid_positions(case, rng):
    """Positions of text runs and image patches: [axes, tokens]."""
    n, t = len(_sections(case)), case["tokens"]
    start = int(rng.integers(0, 100000))
    i = np.arange(t)
    if n == 1:
        return (start + i)[None]
    w = 2 + t % 37
    rows = [start + i // (w * w), start + (i // w) % w, start + i % w, start + (i * 7) % 11]
    pos = np.stack(rows[:n])
    text = (i // 256) % 3 == 0
    pos[:, text] = start + i[text]
    return pos


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _randn(g, shape, dtype):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).to(dtype)


def _i32(x):
    return torch.from_numpy(np.ascontiguousarray(x).astype(np.int32)).to(DEV)


# ----------------------------------------------------------------- prepare ---
def prepare(case, seed):
    g, rng, op = _gen(seed), np.random.default_rng(seed), case["op"]
    s = dict(case=case, op=op)
    if op == "extend":
        n, p = case["reqs"], case["page"]
        lens = np.minimum(rng.integers(0, 2 * case["ctx"] + 1, n), case["width"] * p - 2 * case["add"])
        lens = np.maximum(lens, 0)
        add = np.full(n, 1) if case["add"] == 1 else rng.integers(0, 2 * case["add"] + 1, n)
        have = -(-lens // p)
        need = -(-(lens + add) // p) - have
        free = int(need.sum()) if not case["short"] else int(need.sum()) * 2 // 3
        spare = 0 if case["short"] else 64
        pages = rng.permutation(int(have.sum()) + free + spare)
        table = np.full((n, case["width"]), -1, dtype=np.int64)
        at = 0
        for r in range(n):
            table[r, :have[r]] = pages[at:at + have[r]]
            at += have[r]
        rows = int(n if case["add"] == 1 else 2 * case["add"] * n)
        s.update(table=_i32(table), lens=_i32(lens), add=_i32(add), free=_i32(pages[at:]), n_free=_i32([free + spare]), rows=rows,
                 page=p)
        return s
    hq, hkv, d, dt = case["hq"], case["hkv"], case["d"], TYPES[case["dtype"]]
    if op == "rope":
        t = case["tokens"]
        s["q"], s["k"] = _randn(g, (t, hq, d), dt), _randn(g, (t, hkv, d), dt)
        s["pos"] = _i32(_grid_positions(case, rng))
        s["freq"] = _freq(case)
        if own:
            from tile_attention_lse_gb300 import api
            s["rope"] = api.Rope(_sections(case), interleaved=case["interleaved"], restart=case["restart"], adjacent=case["adjacent"])
        return s
    p = case["page"]
    if op == "append":
        t = case["tokens"]
        pages = -(-t // p) + 3
        s["k_cache"], s["v_cache"] = _randn(g, (pages, p, hkv, d), dt), _randn(g, (pages, p, hkv, d), dt)
        qkv = _randn(g, (t, hq + 2 * hkv, d), dt)  # the rows of one fused projection
        s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        order = torch.from_numpy(rng.permutation(pages)).to(DEV)
        i = torch.arange(t, device=DEV) + 3
        s["slots"] = (order[i // p] * p + i % p).to(torch.int32)
        s["pos"] = _i32(_grid_positions(case, rng))
        s["freq"] = _freq(case)
        s["q_out"] = torch.empty((t, hq, d), dtype=dt, device=DEV)
        if own:
            from tile_attention_lse_gb300 import api
            s["kv"] = api.PagedKV(s["k_cache"], s["v_cache"])
            s["rope"] = api.Rope(_sections(case), interleaved=case["interleaved"], restart=case["restart"], adjacent=case["adjacent"])
        return s
    new, old = _lengths(case)
    n, lens = case["reqs"], old + new
    used = -(-lens // p)
    pages, width = int(used.sum()) + 2, int(used.max()) + 1
    s["k_cache"], s["v_cache"] = _randn(g, (pages, p, hkv, d), dt), _randn(g, (pages, p, hkv, d), dt)
    order = rng.permutation(pages)
    table = np.full((n, width), -1, dtype=np.int64)  # no page behind a request's last
    at = 0
    for r in range(n):
        table[r, :used[r]] = order[at:at + used[r]]
        at += used[r]
    rows = int(new.sum())
    s["q"] = _randn(g, (rows, hq + 2 * hkv, d), dt)[:, :hq]  # the first heads of one fused projection
    s["table"], s["lens"] = _i32(table), _i32(lens)
    s["cu"] = _i32(np.concatenate([[0], np.cumsum(new)]))
    s["most"] = int(new.max())
    if own:
        from tile_attention_lse_gb300 import api
        s["kv"] = api.PagedKV(s["k_cache"], s["v_cache"])
        s["p"] = api.PagedProblem(s["kv"], heads_q=hq, max_new=s["most"], causal=case["causal"], window=case["window"])
        s["ws"] = api.paged_workspace(s["p"])
    return s


def _freq(case):
    axis, step = _axis_and_step(case)
    return dict(axis=torch.tensor(axis, device=DEV), inv=torch.tensor([10000.0 ** -e for e in step], dtype=torch.float64, device=DEV))


# --------------------------------------------------------------------- run ---
def run(state):
    if own:
        return _run_own(state)
    return {"attn": _plain_attn, "rope": _plain_rope, "append": _plain_append, "extend": _plain_extend}[state["op"]](state)


def _run_own(s):
    from tile_attention_lse_gb300 import api
    c = s["case"]
    if s["op"] == "attn":
        o, lse = api.paged_attn_fwd(s["p"], s["q"], s["table"], s["cu"], s["lens"], ws=s["ws"])
        return dict(o=o, lse=lse)
    if s["op"] == "rope":
        q, k = api.rope_axes(s["rope"], s["pos"], s["q"], s["k"], inverse=c["inverse"])
        return dict(q=q, k=k)
    if s["op"] == "append":
        api.kv_append(s["kv"], s["slots"], s["k"], s["v"], rope=s["rope"], pos=s["pos"], q=s["q"], q_out=s["q_out"])
        return dict(q=s["q_out"], k_cache=s["k_cache"], v_cache=s["v_cache"])
    lens, cu, slots, pos, n_free = api.kv_extend(s["page"], s["table"], s["lens"], s["add"], s["free"], s["n_free"], s["rows"])
    return dict(table=s["table"], lens=lens, cu=cu, slots=slots, pos=pos, n_free=n_free)


def _plain_attn(s):
    c, table, lens, cu = s["case"], s["table"].long(), s["lens"].long(), s["cu"].long()
    n, hq, hkv, d = c["reqs"], c["hq"], c["hkv"], c["d"]
    length = table.shape[1] * c["page"]
    k = s["k_cache"][table.clamp(min=0)].float().reshape(n, length, hkv, d)
    v = s["v_cache"][table.clamp(min=0)].float().reshape(n, length, hkv, d)
    key = torch.arange(length, device=DEV)
    i = torch.arange(s["most"], device=DEV)
    new = cu[1:] - cu[:-1]
    row = (cu[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)                              # [n, most]
    q = s["q"][row].float().reshape(n, s["most"], hkv, hq // hkv, d)
    pos = (lens - new)[:, None] + i                                                       # position of each query
    seen = (key < lens[:, None])[:, None, :].expand(n, s["most"], length)
    if c["causal"]:
        seen = seen & (key <= pos[:, :, None])
    if c["window"]:
        seen = seen & (pos[:, :, None] - key < c["window"])
    v = torch.where((key < lens[:, None])[:, :, None, None], v, 0.0)
    x = torch.matmul(q.permute(0, 2, 3, 1, 4).reshape(n, hkv, -1, d), k.permute(0, 2, 3, 1)) * (1.0 / math.sqrt(d))
    x = x.reshape(n, hkv, hq // hkv, s["most"], length).masked_fill(~seen[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    x = torch.exp(x - m)
    z = x.sum(-1, keepdim=True)
    o = torch.matmul(x.reshape(n, hkv, -1, length), v.permute(0, 2, 1, 3)).reshape(n, hkv, hq // hkv, s["most"], d)
    o = o / torch.where(z == 0, 1.0, z)
    lse = (m + torch.log(z))[..., 0]
    take = (i < new[:, None]).reshape(-1)
    o = o.permute(0, 3, 1, 2, 4).reshape(n * s["most"], hq, d)[take]
    lse = lse.permute(0, 3, 1, 2).reshape(n * s["most"], hq)[take]
    return dict(o=o.to(s["q"].dtype), lse=lse)


def _plain_turn(s, x, inverse):
    c, f = s["case"], s["freq"]
    ang = s["pos"].double()[f["axis"]].T * f["inv"]                                       # [tokens, pairs]
    cos, sin = ang.cos().float()[:, None], ang.sin().float()[:, None]
    if inverse:
        sin = -sin
    x = x.float()
    n = f["inv"].numel()
    if c["adjacent"]:
        a, b = x[..., 0:2 * n:2], x[..., 1:2 * n:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :n], x[..., n:2 * n]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([y, x[..., 2 * n:]], -1)


def _plain_rope(s):
    inv, dt = s["case"]["inverse"], s["q"].dtype
    return dict(q=_plain_turn(s, s["q"], inv).to(dt), k=_plain_turn(s, s["k"], inv).to(dt))


def _plain_append(s):
    dt, p = s["q"].dtype, s["case"]["page"]
    slot = s["slots"].long()
    s["k_cache"][slot // p, slot % p] = _plain_turn(s, s["k"], False).to(dt)
    s["v_cache"][slot // p, slot % p] = s["v"]
    s["q_out"].copy_(_plain_turn(s, s["q"], False).to(dt))
    return dict(q=s["q_out"], k_cache=s["k_cache"], v_cache=s["v_cache"])


def _plain_extend(s):
    p, table, rows = s["page"], s["table"], s["rows"]
    lens, add, free, n_free = s["lens"].long(), s["add"].long(), s["free"].long(), s["n_free"].long()
    n, width = table.shape
    have = (lens + p - 1) // p
    need = (lens + add + p - 1) // p - have
    upto = need.cumsum(0)
    fits = (upto <= n_free) & (have + need <= width) & (add.cumsum(0) <= rows)
    fits = fits.long().cumprod(0) > 0                      # served in order: nothing behind the first that does not fit
    given = torch.where(fits, add, 0)
    cu = torch.cat([given.new_zeros(1), given.cumsum(0)])
    col = torch.arange(width, device=DEV)
    j = col - have[:, None]                                # new page of this column
    fresh = (j >= 0) & (j < need[:, None]) & fits[:, None]
    take = (n_free - 1 - (upto - need)[:, None] - j).clamp(0, max(0, free.numel() - 1))
    table.copy_(torch.where(fresh, free[take] if free.numel() else -1, table.long()))
    t = torch.arange(rows, device=DEV)
    r = torch.searchsorted(cu[1:].contiguous(), t, right=True).clamp(max=n - 1)
    real = t < cu[-1]
    pos = torch.where(real, lens[r] + t - cu[:-1][r], 0)
    slots = torch.where(real, table.long()[r, (pos // p).clamp(max=width - 1)] * p + pos % p, -1)
    left = n_free - torch.where(fits, need, 0).sum()
    i32 = torch.int32
    return dict(table=table, lens=(lens + given).to(i32), cu=cu.to(i32), slots=slots.to(i32), pos=pos.to(i32), n_free=left.to(i32))


# -------------------------------------------------------------------- work ---
def _visible(case):
    """Visible (query, key) pairs over all requests, and the keys that some query of each request sees."""
    new, old = _lengths(case)
    pairs = keys = 0
    for q, o in zip(new.tolist(), old.tolist()):
        pos = o + np.arange(q)
        hi = pos + 1 if case["causal"] else np.full(q, o + q)
        lo = np.maximum(0, pos - case["window"] + 1) if case["window"] else np.zeros(q, dtype=np.int64)
        pairs += int(np.maximum(0, hi - lo).sum())
        keys += int(hi.max() - lo.min())
    return pairs, keys, int(new.sum())


def work(case):
    if case["op"] == "extend":
        n = case["reqs"]
        rows = n if case["add"] == 1 else 2 * case["add"] * n
        return {"bytes": 4.0 * (5 * n + 3 + 2 * rows + 2 * n * case["add"] / case["page"]), "flops": 0.0}
    size = 2 if case["dtype"] == "bf16" else 4
    row = case["d"] * size
    if case["op"] == "attn":
        pairs, keys, rows = _visible(case)
        return {"bytes": float(2 * keys * case["hkv"] * row + rows * case["hq"] * (2 * row + 4)),
                "flops": 4.0 * case["d"] * case["hq"] * pairs}
    t, pairs = case["tokens"], sum(_sections(case))
    heads = case["hq"] + case["hkv"]
    moved = heads + (case["hkv"] if case["op"] == "append" else 0)
    return {"bytes": float(t * (2 * moved * row + 4 * len(_sections(case)) + (4 if case["op"] == "append" else 0))),
            "flops": 6.0 * t * heads * pairs}


# ------------------------------------------------------------------- exact ---
def exact(case, seed):
    op = case["op"]
    if op == "extend":
        return None  # whole numbers
    s = prepare(case, seed)
    if op == "attn":
        return _exact_attn(case, s)

    axis, step = _axis_and_step(case)
    n = len(axis)
    turn = torch.empty((case["tokens"], n), dtype=torch.complex128, device=DEV)
    for i in range(n):
        a = s["pos"][axis[i]].double() * 10000.0 ** -step[i]
        turn[:, i] = torch.polar(torch.ones_like(a), -a if case.get("inverse") else a)

    def rotated(x):
        y = x.double().clone()
        one, two = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if case["adjacent"] else (slice(0, n), slice(n, 2 * n))
        z = torch.complex(y[..., one], y[..., two]) * turn[:, None]
        y[..., one], y[..., two] = z.real, z.imag
        return y

    if op == "rope":
        return dict(q=rotated(s["q"]), k=rotated(s["k"]))
    kc, vc = (s[x].double().flatten(0, 1) for x in ("k_cache", "v_cache"))
    kc[s["slots"].long()] = rotated(s["k"])
    vc[s["slots"].long()] = s["v"].double()
    shape = s["k_cache"].shape
    return dict(q=rotated(s["q"]), k_cache=kc.reshape(shape), v_cache=vc.reshape(shape))


def _exact_attn(case, s):
    new, old = _lengths(case)
    hq, hkv, d, p = case["hq"], case["hkv"], case["d"], case["page"]
    out = torch.zeros((int(new.sum()), hq, d), dtype=torch.float64, device=DEV)
    lse = torch.full((int(new.sum()), hq), -math.inf, dtype=torch.float64, device=DEV)
    t0 = 0
    for r in range(case["reqs"]):
        t1, length = t0 + int(new[r]), int(new[r] + old[r])
        pages = s["table"][r, :-(-length // p)].long()
        first = 0
        if case["window"]:
            first = max(0, int(old[r]) - case["window"] + 1)
        j = torch.arange(first, length, device=DEV)
        i = torch.arange(int(old[r]), length, device=DEV)
        hide = torch.zeros((i.numel(), j.numel()), dtype=torch.bool, device=DEV)
        if case["causal"]:
            hide |= j[None] > i[:, None]
        if case["window"]:
            hide |= i[:, None] - j[None] >= case["window"]
        for g in range(hkv):
            kk = s["k_cache"][pages, :, g].reshape(-1, d)[first:length].double()
            vv = s["v_cache"][pages, :, g].reshape(-1, d)[first:length].double()
            for h in range(g * (hq // hkv), (g + 1) * (hq // hkv)):
                x = (s["q"][t0:t1, h].double() @ kk.T) / math.sqrt(d)
                x[hide] = -math.inf
                lse[t0:t1, h] = torch.logsumexp(x, 1)
                w = torch.exp(x - lse[t0:t1, h, None])
                out[t0:t1, h] = torch.nan_to_num(w, nan=0.0) @ vv
        t0 = t1
    return dict(o=out, lse=lse)
