"""Serving operators on the GPU against plain float64 implementations: request
tables, multi-axis rotary positions, cache append, attention over the pages,
and a run of them together.

Tolerances (u32 = 2^-24, u16 = 2^-8: half a step of float32 and bfloat16,
relative to the value):
* a rotated element: two products and a sum of elements of magnitude at most A
  with sines and cosines that are off by at most 2^-25 half turns pi + 2 u32,
  so 2 A (2^-24 pi / 2 + 2 u32 + 2 u32) < 12 A u32, and the output's rounding;
* a score: a sum of d products, off by at most 6 sqrt(d) u32 |q| |k| scale (six
  standard deviations of independent roundings) plus the scale's and the
  exponent's own 4 u32; a weight is off by twice that and exp2's 2 ulp;
* O: every weight's error times max |v| at most; with bfloat16, u16 max |v|
  more for the weights' rounding and u16 |O| for the output's.  In the mean
  the two roundings stay below u16 |O| each: the 2-norm is held to 2 u16.
"""

import os
import subprocess
import sys
import threading

import numpy as np
import pytest
import torch

from oracle import paged as P
from tile_attention_lse_gb300 import api

from helpers import f64

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U32, U16 = 2.0 ** -24, 2.0 ** -8
I32 = dict(dtype=torch.int32, device=DEV)
HALF = {torch.float32: U32, torch.bfloat16: U16}


def dev(x, dtype=torch.int32):
    return torch.from_numpy(np.ascontiguousarray(x)).to(DEV).to(dtype)


def host(x):
    return x.cpu().numpy()


@pytest.fixture(autouse=True)
def no_device_error():
    yield
    assert api.device_error() == 0


# ------------------------------------------------------------------ tables ---
def table_case(n, page, width, add, lens, rows, free_spare, seed):
    rng = np.random.default_rng(seed)
    lens, add = np.asarray(lens), np.asarray(add)
    have = np.minimum(-(-np.maximum(lens, 0) // page), width)
    need = int(np.maximum(0, -(-np.maximum(lens + add, 0) // page) - have).sum())
    pages = rng.permutation(int(have.sum()) + need + 7)
    table = np.full((n, width), -7, dtype=np.int64)
    at = 0
    for r in range(n):
        table[r, :have[r]] = pages[at:at + have[r]]
        at += have[r]
    free = pages[at:]
    return table, lens, add, free, max(0, need + free_spare), rows


rng0 = np.random.default_rng(0)
TABLES = {
    "one": table_case(1, 16, 8, [1], [0], 1, 0, 0),
    "page_ends_and_begins": table_case(6, 16, 8, [1, 1, 1, 16, 17, 0], [15, 16, 17, 16, 31, 32], 40, 7, 1),
    "nothing_new": table_case(3, 8, 4, [0, 0, 0], [5, 0, 32], 5, 0, 2),
    "no_rows": table_case(3, 8, 4, [0, 1, 0], [5, 0, 32], 0, 0, 2),
    "short_of_pages": table_case(9, 16, 16, [40] * 9, [3, 0, 100, 7, 16, 16, 0, 0, 9], 400, -5, 3),
    "no_free_page": table_case(4, 16, 16, [1, 1, 1, 1], [3, 15, 16, 3], 8, -99, 3),
    "table_too_narrow": table_case(4, 16, 3, [10, 20, 30, 1], [38, 20, 19, 0], 90, 7, 4),
    "too_few_rows": table_case(4, 32, 9, [10, 20, 30, 1], [38, 20, 19, 0], 45, 7, 4),
    "negative": table_case(4, 32, 9, [10, 20, -3, 1], [38, 20, 19, 0], 45, 7, 4),
    "many_requests": table_case(2500, 8, 12, rng0.integers(0, 9, 2500), rng0.integers(0, 80, 2500), 12000, 7, 5),
    "many_rows": table_case(5, 64, 900, [9000, 1, 0, 20001, 3], [100, 64, 3, 0, 999], 29500, 7, 6),
    "odd_page": table_case(3, 5, 9, [7, 11, 0], [3, 5, 10], 20, 7, 7),
    "no_request": table_case(0, 16, 4, [], [], 6, 0, 8),
}


def page_of(name):
    return {"one": 16, "page_ends_and_begins": 16, "nothing_new": 8, "no_rows": 8, "short_of_pages": 16, "no_free_page": 16,
            "table_too_narrow": 16, "too_few_rows": 32, "negative": 32, "many_requests": 8, "many_rows": 64, "odd_page": 5,
            "no_request": 16}[name]


@pytest.mark.parametrize("name", TABLES)
def test_extend(name):
    table, lens, add, free, n_free, rows = TABLES[name]
    page = page_of(name)
    t = dev(table)
    want_t = table.copy()
    want = P.extend(lens, add, want_t, free, n_free, page, rows)
    for _ in range(2):  # the inputs stay as they were: a second call gives the same
        got = api.kv_extend(page, t, dev(lens), dev(add), dev(free), dev([n_free]), rows)
        for g, w, what in zip(got, want, ("lens", "cu", "slots", "pos", "n_free")):
            assert np.array_equal(host(g).ravel(), np.ravel(w)), what
        assert np.array_equal(host(t), want_t)


def test_extend_clamps_the_free_count():
    table, lens, add, free, _, rows = TABLES["page_ends_and_begins"]
    for n_free in (-4, 10 ** 6):
        t, want_t = dev(table), table.copy()
        want = P.extend(lens, add, want_t, free, n_free, 16, rows)
        got = api.kv_extend(16, t, dev(lens), dev(add), dev(free), dev([n_free]), rows)
        assert np.array_equal(host(got[1]), want[1]) and int(got[4]) == want[4] and np.array_equal(host(t), want_t)


@pytest.mark.parametrize("name", ["page_ends_and_begins", "many_requests", "no_request", "odd_page"])
@pytest.mark.parametrize("room", [0, 10000])
def test_release(name, room):
    table, lens, _, free, n_free, _ = TABLES[name]
    page = page_of(name)
    pool = np.concatenate([free, np.zeros(room, dtype=np.int64)])
    done = np.arange(len(lens)) % 3 == 1
    t, f = dev(table), dev(pool)
    want_t, want_f = table.copy(), pool.copy()
    want = P.release(lens, done, want_t, want_f, n_free, page)
    got = api.kv_release(page, t, dev(lens), dev(done), f, dev([n_free]))
    assert np.array_equal(host(got[0]), want[0]) and int(got[1]) == want[1]
    assert np.array_equal(host(t), want_t) and np.array_equal(host(f), want_f)


# -------------------------------------------------------------------- rope ---
ROPES = [
    # sections, interleaved, restart, adjacent, head_dim
    ([64], False, False, False, 128),
    ([16, 24, 24], False, False, False, 128),
    ([24, 20, 20], True, False, False, 128),
    ([8, 12, 12], False, True, True, 64),
    ([32], False, False, True, 128),       # a part of the head
    ([8], False, False, False, 64),
    ([3, 0, 4, 1], True, True, False, 64),
    ([20, 20, 20, 4], False, True, True, 128),
]


def positions(axes, rows, seed):
    pos = np.random.default_rng(seed).integers(-1000, 200000, (axes, rows))
    pos.ravel()[:4] = [0, 2 ** 31 - 1, -2 ** 31, 1][:pos.size]
    return pos


def rope_kw(r):
    return dict(interleaved=r[1], restart=r[2], adjacent=r[3])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("r", ROPES, ids=[str(i) for i in range(len(ROPES))])
@pytest.mark.parametrize("rows,hq,hk", [(1, 1, 1), (37, 5, 2), (4099, 2, 17)])
def test_rope(r, dtype, rows, hq, hk):
    d, axes = r[4], len(r[0])
    rope = api.Rope(r[0], base=10000.0, **rope_kw(r))
    pos = positions(axes, rows, 3)
    g = torch.Generator().manual_seed(rows)
    x = torch.randn((rows, hq + hk + 1, d), generator=g).to(dtype).to(DEV)
    q, k = x[:, :hq], x[:, hq:hq + hk]
    for inverse in (False, True):
        gq, gk = api.rope_axes(rope, dev(pos), q, k, inverse=inverse)
        for got, src in ((gq, q), (gk, k)):
            want = P.rope_axes(f64(src), pos, r[0], inverse=inverse, **rope_kw(r))
            big = float(src.abs().max())
            # a position of 2^31 turns the fastest pair 2^31 / 2 pi times: the
            # 53-bit fraction and the oracle's own product leave 2^-21 radians
            tol = 12 * big * U32 + HALF[dtype] * 1.5 * big
            far = np.any(np.abs(pos) > 2 ** 24, axis=0)
            err = np.abs(f64(got) - want)
            assert err[~far].max(initial=0.0) <= tol
            assert err[far].max(initial=0.0) <= tol + 2 * big * 2.0 ** -21
    alone = api.rope_axes(rope, dev(pos), k, inverse=True)
    assert torch.equal(alone, gk)


def test_rope_one_axis_is_the_gathers_rope():
    rows, h, d = 256, 3, 128
    x = torch.randn((1, rows, h, d), generator=torch.Generator().manual_seed(1)).to(DEV)
    p = api.Problem(batch=1, heads_q=h, heads_kv=h, head_dim=d, cp=1, seqlen=rows, dtype=torch.float32)
    idx, _ = api.partition_indices(p)
    want = api.permute_rope(p, idx, x)[0]
    got = api.rope_axes(api.Rope([64]), torch.arange(rows, **I32), x[0][idx.long()[0]].contiguous())
    assert float((got - want).abs().max()) <= 24 * U32 * float(x.abs().max())


def test_rope_in_place_and_what_is_not_rotated():
    r = api.Rope([8, 8])
    x = torch.randn((9, 4, 128), generator=torch.Generator().manual_seed(2)).to(DEV)
    x[0, 0, 40] = float("inf")
    x[0, 1, 100] = float("nan")
    pos = dev(positions(2, 9, 5))
    want = api.rope_axes(r, pos, x)
    y = x.clone()
    assert api.rope_axes(r, pos, y, q_out=y) is y
    assert torch.equal(torch.nan_to_num(y), torch.nan_to_num(want))
    same = lambda a, b: bool(((a == b) | (a.isnan() & b.isnan())).all())  # noqa: E731
    assert same(want[..., 32:], x[..., 32:]) and torch.isfinite(want[..., :32]).all()
    with pytest.raises(api.CpError):
        wide = torch.zeros((9, 6, 128), device=DEV)[:, :4]
        api.rope_axes(r, pos, wide, q_out=torch.empty(0, device=DEV).set_(wide.untyped_storage(), 0, (9, 4, 128), (512, 128, 1)))


def test_rope_gradient_against_differences():
    # the rotation is linear, so a central difference of any width is exact
    # up to float32 rounding: L = <c, R x>, dL/dx = R^T c
    r, rows, d = api.Rope([16, 24, 24], restart=True), 3, 128
    pos = dev(positions(3, rows, 7) % 5000)
    g = torch.Generator().manual_seed(3)
    x, c = (torch.randn((rows, 1, d), generator=g).to(DEV) for _ in range(2))
    grad = api.rope_axes(r, pos, c, inverse=True)
    for i in range(0, d, 5):
        e = torch.zeros_like(x)
        e[:, 0, i] = 1.0
        diff = (c * (api.rope_axes(r, pos, x + e).double() - api.rope_axes(r, pos, x - e).double())).sum(-1) / 2
        tol = 2 * 12 * U32 * (float(x.abs().max()) + 1) * 2 * float(c.abs().max())
        assert float((diff - grad[..., i]).abs().max()) <= tol


# ------------------------------------------------------------------ append ---
def make_cache(pages, page, hkv, d, dtype, order, fill=float("nan")):
    if order == "token":
        k, v = (torch.full((pages, page, hkv, d), fill, dtype=dtype, device=DEV) for _ in range(2))
    elif order == "head":
        k, v = (torch.full((pages, hkv, page, d), fill, dtype=dtype, device=DEV).transpose(1, 2) for _ in range(2))
    else:  # K and V of a page side by side
        kv = torch.full((pages, 2, page, hkv, d), fill, dtype=dtype, device=DEV)
        k, v = kv[:, 0], kv[:, 1]
    return api.PagedKV(k, v)


@pytest.mark.parametrize("order", ["token", "head", "beside"])
@pytest.mark.parametrize("dtype,d,rows,hq,hkv,page", [
    (torch.bfloat16, 128, 1, 4, 1, 8), (torch.bfloat16, 128, 70, 7, 3, 16), (torch.float32, 64, 33, 2, 2, 32),
    (torch.float32, 128, 5, 3, 1, 256), (torch.bfloat16, 64, 4100, 1, 1, 64)])
def test_append(dtype, d, rows, hq, hkv, page, order):
    pages = -(-rows // page) + 2
    sections = [d // 8, d // 8, d // 4]
    kv = make_cache(pages, page, hkv, d, dtype, order)
    g = torch.Generator().manual_seed(5)
    qkv = torch.randn((rows, hq + 2 * hkv, d), generator=g).to(dtype).to(DEV)
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    slots = np.random.default_rng(1).permutation(pages * page)[:rows]
    if rows > 4:  # rows that have no slot
        slots[1], slots[3], slots[4] = -1, pages * page, 2 ** 31 - 1
    there = (slots >= 0) & (slots < pages * page)
    pos = positions(3, rows, 2)
    pos = pos % 10000
    q_out = torch.full((rows, hq, d), 7.0, dtype=dtype, device=DEV)
    api.kv_append(kv, dev(slots), k, v, rope=api.Rope(sections), pos=dev(pos), q=q, q_out=q_out)
    want_k, want_v = (np.full((pages * page, hkv, d), np.nan) for _ in range(2))
    want_k[slots[there]] = P.rope_axes(f64(k), pos, sections)[there]
    want_v[slots[there]] = f64(v)[there]
    big = float(qkv.abs().max())
    tol = 12 * big * U32 + HALF[dtype] * 1.5 * big
    got_k, got_v = f64(kv.k_cache).reshape(-1, hkv, d), f64(kv.v_cache).reshape(-1, hkv, d)
    assert np.array_equal(np.isnan(got_k), np.isnan(want_k)) and np.array_equal(got_v, want_v, equal_nan=True)
    assert np.nanmax(np.abs(got_k - want_k)) <= tol
    want_q = P.rope_axes(f64(q), pos, sections)
    assert np.abs(f64(q_out) - want_q)[there].max() <= tol
    assert (f64(q_out)[~there] == 7.0).all()
    # without a rotation: plain copies
    kv2 = make_cache(pages, page, hkv, d, dtype, order)
    assert api.kv_append(kv2, dev(slots), k, v) is None
    want_k[slots[there]] = f64(k)[there]
    assert np.array_equal(f64(kv2.k_cache).reshape(-1, hkv, d), want_k, equal_nan=True)


# --------------------------------------------------------------- attention ---
def paged_inputs(new, lens, hq, hkv, d, page, dtype, order="token", seed=0, window=0, spread=1.0, tail=0):
    """Pages that hold NaN wherever no visible token is; table entries that no
    row needs are far out of range."""
    rng = np.random.default_rng(seed)
    g = torch.Generator().manual_seed(seed)
    n = len(lens)
    used = -(-np.asarray(lens) // page)
    pages, width = int(used.sum()) + 3, max(1, int(used.max(initial=1)) + 1)
    kv = make_cache(pages, page, hkv, d, dtype, order)
    ids = rng.permutation(pages)
    table = np.full((n, width), 2 ** 31 - 1, dtype=np.int64)
    at = 0
    for r in range(n):
        table[r, :used[r]] = ids[at:at + used[r]]
        at += used[r]
        ln = int(lens[r])
        if ln == 0:
            continue
        first = max(0, ln - new[r] - window + 1) if window else 0
        k, v = (spread * torch.randn((ln, hkv, d), generator=g) for _ in range(2))
        j = np.arange(first, ln)
        pg, tk = dev(table[r][j // page], torch.int64), dev(j % page, torch.int64)
        kv.k_cache[pg, tk] = k[first:].to(dtype).to(DEV)
        kv.v_cache[pg, tk] = v[first:].to(dtype).to(DEV)
        table[r, :first // page] = -1  # pages in front of the window were given back
    cu = np.concatenate([[0], np.cumsum(new)])
    rows = int(cu[-1]) + tail
    q = torch.randn((rows, hq + 2, d), generator=g).to(dtype).to(DEV)[:, 1:hq + 1]
    return kv, q, table, cu


def check_attention(kv, q, table, cu, lens, o, lse, causal=True, window=0, scale=None):
    dtype, d = q.dtype, q.shape[2]
    qh, kh, vh = f64(q), f64(kv.k_cache), f64(kv.v_cache)
    want_o, want_l = P.attention(qh, kh, vh, table, cu, lens, causal, window, scale)
    end = int(cu[-1])
    got_o, got_l = f64(o)[:end], f64(lse)[:end]
    want_o, want_l = want_o[:end], want_l[:end]
    if end == 0:
        return
    none = np.isneginf(want_l)
    assert np.array_equal(none, np.isneginf(got_l)) and np.isfinite(got_o).all()
    assert (got_o[none] == 0).all()
    sc = 1 / np.sqrt(d) if scale is None else scale
    vmax = np.nanmax(np.abs(vh))
    score = sc * np.sqrt((qh ** 2).sum(-1)).max() * np.sqrt(np.nanmax((kh ** 2).sum(-1)))
    e_s = U32 * (6 * np.sqrt(d) + 4) * score
    keys = max(lens)
    e_w = 2 * e_s + 4 * U32 + 6 * np.sqrt(keys) * U32
    tol = 2 * vmax * e_w + U32 * vmax
    if dtype == torch.bfloat16:
        tol = tol + U16 * vmax + U16 * np.abs(want_o)
    err = np.abs(got_o - want_o)
    assert (err <= tol).all(), float((err - tol).max())
    assert np.abs(got_l[~none] - want_l[~none]).max(initial=0.0) <= e_w + 4 * U32 * np.abs(want_l[~none]).max(initial=0.0)
    if dtype == torch.bfloat16:
        assert np.linalg.norm(got_o - want_o) <= 2 * U16 * np.linalg.norm(want_o)


ATTN = [
    # name, new, lens, hq, hkv, causal, window
    ("one_key", [1], [1], 4, 4, True, 0),
    ("lengths_around_a_slice", [1] * 9, [0, 1, 15, 16, 17, 63, 64, 65, 130], 8, 2, True, 0),
    ("long", [1], [9001], 8, 1, True, 0),
    ("few_new", [3, 1, 8, 2], [3, 200, 77, 1000], 8, 4, True, 0),
    ("chunks", [70, 129, 1, 33], [70, 300, 129, 700], 4, 2, True, 0),
    ("wide_chunk", [260], [777], 28, 4, True, 0),
    ("tile_ends_in_the_last_page", [65, 129, 66], [65, 190, 1100], 8, 2, True, 0),
    ("window_in_chunks", [200, 70, 1, 300], [900, 70, 500, 301], 8, 2, True, 77),
    ("ends_of_pages", [64, 70, 70, 70, 70], [128, 129, 192, 255, 257], 4, 1, True, 0),
    ("no_new_and_empty", [0, 2, 0, 5, 0], [9, 0, 0, 5, 33], 4, 1, True, 0),
    ("more_new_than_cached", [20, 3], [7, 50], 4, 2, True, 0),
    ("window", [1, 40, 5, 1], [600, 333, 5, 20], 8, 2, True, 50),
    ("window_one", [1, 17], [40, 17], 4, 4, True, 1),
    ("not_causal", [1, 9, 40], [30, 40, 400], 10, 2, False, 0),
    ("not_causal_window", [6, 40], [30, 200], 2, 2, False, 33),
    ("wide_group", [2, 5], [300, 20], 40, 1, True, 0),
]


@pytest.mark.parametrize("dtype,d", [(torch.float32, 64), (torch.float32, 128), (torch.bfloat16, 64), (torch.bfloat16, 128)])
@pytest.mark.parametrize("case", ATTN, ids=[c[0] for c in ATTN])
def test_attention(case, dtype, d):
    _, new, lens, hq, hkv, causal, window = case
    i = ATTN.index(case)
    page, order = [8, 16, 32, 64, 128, 256][i % 6], ["token", "head", "beside"][i % 3]
    kv, q, table, cu = paged_inputs(new, lens, hq, hkv, d, page, dtype, order, seed=i, window=window, tail=3)
    p = api.PagedProblem(kv, hq, max_new=max(new), causal=causal, window=window)
    ws = api.paged_workspace(p)
    ws.fill_(255)                                            # NaN: nothing is read before it is written
    o = torch.full((q.shape[0], hq, d), 7.0, dtype=dtype, device=DEV)
    lse = torch.full((q.shape[0], hq), 7.0, device=DEV)
    args = (dev(table), dev(cu), dev(lens))
    api.paged_attn_fwd(p, q, *args, ws=ws, out=o, lse=lse)
    assert (o[int(cu[-1]):] == 7).all() and (lse[int(cu[-1]):] == 7).all()  # rows of no request
    check_attention(kv, q, table, cu, lens, o, lse, causal, window)
    o2, lse2 = api.paged_attn_fwd(p, q, *args)               # the same bits again
    end = int(cu[-1])
    assert torch.equal(o2[:end], o[:end]) and torch.equal(lse2[:end], lse[:end])


@pytest.mark.parametrize("dtype,d", [(torch.float32, 64), (torch.bfloat16, 64), (torch.bfloat16, 128)])
@pytest.mark.parametrize("max_new", [0, 1, 4, 5000])
def test_attention_with_any_hint(dtype, d, max_new):
    new, lens, hq, hkv = [1, 30, 140], [64, 65, 300], 6, 2
    kv, q, table, cu = paged_inputs(new, lens, hq, hkv, d, 16, dtype, seed=3)
    p = api.PagedProblem(kv, hq, max_new=max_new)
    o, lse = api.paged_attn_fwd(p, q, dev(table), dev(cu), dev(lens))
    check_attention(kv, q, table, cu, lens, o, lse)


@pytest.mark.parametrize("dtype,d", [(torch.float32, 128), (torch.bfloat16, 128)])
@pytest.mark.parametrize("new", [[1, 1], [200, 64]])
def test_attention_with_scores_that_rise_and_a_scale(dtype, d, new):
    # keys whose scores rise along the sequence: the running maximum moves again and again
    lens, hq, hkv = [700, 300], 4, 2
    kv, q, table, cu = paged_inputs(new, lens, hq, hkv, d, 32, dtype, seed=4)
    for r, ln in enumerate(lens):
        j = np.arange(ln)
        pg, tk = dev(table[r][j // 32], torch.int64), dev(j % 32, torch.int64)
        ramp = (1 + 12 * torch.arange(ln, device=DEV) / ln)[:, None, None]
        kv.k_cache[pg, tk] = (kv.k_cache[pg, tk].float() * ramp).to(dtype)
    for scale in (0.0, 0.25):
        p = api.PagedProblem(kv, hq, max_new=max(new), softmax_scale=scale)
        o, lse = api.paged_attn_fwd(p, q, dev(table), dev(cu), dev(lens))
        check_attention(kv, q, table, cu, lens, o, lse, scale=scale or None)


def test_attention_many_requests():
    rng = np.random.default_rng(8)
    n = 1100
    lens = rng.integers(0, 40, n)
    new = np.minimum(rng.integers(0, 3, n), lens)
    kv, q, table, cu = paged_inputs(new, lens, 4, 2, 64, 8, torch.bfloat16, seed=9)
    p = api.PagedProblem(kv, 4, max_new=2)
    o, lse = api.paged_attn_fwd(p, q, dev(table), dev(cu), dev(lens))
    check_attention(kv, q, table, cu, lens, o, lse)


def test_attention_page_outside_the_cache_is_reported():
    # the division test and the refusals on the host come first; here the
    # kernel's own check of the page number keeps it from being read
    for dtype, max_new in ((torch.bfloat16, 1), (torch.float32, 1), (torch.bfloat16, 64)):
        new, lens = [1, 1] if max_new == 1 else [64, 20], [70, 90]
        kv, q, table, cu = paged_inputs(new, lens, 4, 2, 128, 16, dtype, seed=5)
        p = api.PagedProblem(kv, 4, max_new=max_new)
        for bad in (-1, kv.n_pages, 2 ** 31 - 1, -2 ** 31):
            t = table.copy()
            t[1, 2] = bad
            o, lse = api.paged_attn_fwd(p, q, dev(t), dev(cu), dev(lens))
            assert api.device_error() == -1                    # CP_ERR_INVALID_ARG
            end = new[0]                                       # the other request is not touched by it
            check_attention(kv, q[:end], table[:1], cu[:2], lens[:1], o[:end], lse[:end])
            assert torch.isfinite(o.float()).all()
        api.paged_attn_fwd(p, q, dev(table), dev(cu), dev(lens))


@pytest.mark.parametrize("dtype,d,max_new", [(torch.bfloat16, 128, 1), (torch.bfloat16, 128, 96), (torch.float32, 64, 4)])
def test_attention_captured_and_replayed_on_new_lengths(dtype, d, max_new):
    lens0, new0 = [500, 90, 33], [max_new, 1, max_new]
    kv, q, table, cu = paged_inputs(new0, lens0, 8, 2, d, 16, dtype, seed=6)
    p = api.PagedProblem(kv, 8, max_new=max_new)
    t, c, n = dev(table), dev(cu), dev(lens0)
    ws, o, lse = api.paged_workspace(p), torch.empty(q.shape, dtype=dtype, device=DEV), torch.empty(q.shape[:2], device=DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        api.paged_attn_fwd(p, q, t, c, n, ws=ws, out=o, lse=lse)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            api.paged_attn_fwd(p, q, t, c, n, ws=ws, out=o, lse=lse)
    torch.cuda.current_stream().wait_stream(s)
    for lens in ([500, 90, 33], [17, 90, 2], [499, 1, 33]):
        new = np.minimum(new0, lens)
        cu2 = np.concatenate([[0], np.cumsum(new)])
        c.copy_(dev(cu2))
        n.copy_(dev(lens))
        o.fill_(3.0)
        graph.replay()
        check_attention(kv, q, table, cu2, lens, o, lse)


def test_calls_from_two_threads_and_streams():
    new, lens = [[1, 1, 1], [33, 2]], [[400, 7, 120], [200, 64]]
    jobs = []
    for i in range(2):
        kv, q, table, cu = paged_inputs(new[i], lens[i], 8, 2, 128, 16, torch.bfloat16, seed=20 + i)
        jobs.append((api.PagedProblem(kv, 8, max_new=max(new[i])), q, dev(table), dev(cu), dev(lens[i]), table, cu))
    torch.cuda.synchronize()
    out, errors = [None, None], []

    def work(i):
        try:
            p, q, t, c, n, _, _ = jobs[i]
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                for _ in range(20):
                    out[i] = api.paged_attn_fwd(p, q, t, c, n)
                s.synchronize()
        except Exception as e:  # reported on the main thread
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    for i in range(2):
        p, q, *_, table, cu = jobs[i]
        check_attention(p.kv, q, table, cu, lens[i], *out[i])


def test_state_merges_with_other_partial_states():
    # attention over a prefix in the cache, merged with attention over other
    # keys by the library's own merge, is attention over both
    d, hq, hkv, lens = 64, 4, 2, [150, 30]
    kv, q, table, cu = paged_inputs([1, 1], lens, hq, hkv, d, 16, torch.float32, seed=11)
    p = api.PagedProblem(kv, hq, max_new=1)
    whole = api.paged_attn_fwd(p, q, dev(table), dev(cu), dev(lens))
    cut = [64, 16]
    front = api.paged_attn_fwd(p, q, dev(table), dev(cu), dev(cut))
    rest = np.stack([np.concatenate([table[r, c // 16:], table[r, :c // 16]]) for r, c in enumerate(cut)])
    back = api.paged_attn_fwd(p, q, dev(rest), dev(cu), dev([n - c for n, c in zip(lens, cut)]))
    o, lse = api.merge_partials(torch.stack([front[0], back[0]]), torch.stack([front[1], back[1]]))
    assert float((o - whole[0]).abs().max()) <= 1e-5 and float((lse - whole[1]).abs().max()) <= 1e-5


# ---------------------------------------------------------------- together ---
def test_serving_steps_together():
    """Requests of different lengths run through prompt chunks and single
    tokens; what every step answers is the plain attention over all that the
    request has brought so far."""
    n, page, hq, hkv, d, dtype = 5, 16, 8, 2, 128, torch.bfloat16
    sections, pages, width = [16, 24, 24], 40, 12
    kv = make_cache(pages, page, hkv, d, dtype, "beside")
    rope = api.Rope(sections, interleaved=True)
    g = torch.Generator().manual_seed(30)
    rng = np.random.default_rng(31)
    table, lens = torch.full((n, width), -1, **I32), torch.zeros(n, **I32)
    free, n_free = dev(rng.permutation(pages)), dev([pages])
    table_h, lens_h, free_h, n_free_h = host(table).astype(np.int64), np.zeros(n, dtype=np.int64), host(free), pages
    keys, values = [[] for _ in range(n)], [[] for _ in range(n)]
    for step, add in enumerate([[70, 3, 0, 33, 1], [1, 64, 40, 1, 1], [1, 1, 1, 1, 1], [20, 0, 1, 1, 90], [1, 1, 1, 1, 1]]):
        rows = sum(add) + 4                                     # a padded batch
        lens2, cu, slots, pos, n_free2 = api.kv_extend(page, table, lens, dev(add), free, n_free, rows)
        want = P.extend(lens_h, add, table_h, free_h, n_free_h, page, rows)
        for got, w in zip((lens2, cu, slots, pos, n_free2), want):
            assert np.array_equal(host(got).ravel(), np.ravel(w))
        p3 = torch.stack([pos, pos // 7, pos % 7]).contiguous()
        x = torch.randn((rows, hq + 2 * hkv, d), generator=g).to(dtype).to(DEV)
        q = api.kv_append(kv, slots, x[:, hq:hq + hkv], x[:, hq + hkv:], rope=rope, pos=p3, q=x[:, :hq],
                          q_out=torch.zeros((rows, hq, d), dtype=dtype, device=DEV))
        p = api.PagedProblem(kv, hq, max_new=max(add))
        o, lse = api.paged_attn_fwd(p, q, table, cu, lens2)
        assert api.device_error() == 0
        # the plain way: rotate, round as stored, keep per request
        ph, cu_h = host(p3), want[1]
        kr = P.rope_axes(f64(x[:, hq:hq + hkv]), ph, sections, interleaved=True)
        qr = P.rope_axes(f64(x[:, :hq]), ph, sections, interleaved=True)
        rnd = lambda a: f64(torch.from_numpy(a).to(dtype))  # noqa: E731
        kr, qr, vr = rnd(kr), rnd(qr), f64(x[:, hq + hkv:])
        for r in range(n):
            keys[r] += list(kr[cu_h[r]:cu_h[r + 1]])
            values[r] += list(vr[cu_h[r]:cu_h[r + 1]])
        for r in range(n):
            if cu_h[r + 1] == cu_h[r]:
                continue
            kk, vv = (np.stack(a)[None] for a in (keys[r], values[r]))
            wo, wl = P.attention(qr[cu_h[r]:cu_h[r + 1]], kk, vv, np.zeros((1, 1), dtype=np.int64),
                                 [0, cu_h[r + 1] - cu_h[r]], [kk.shape[1]])
            go, gl = f64(o)[cu_h[r]:cu_h[r + 1]], f64(lse)[cu_h[r]:cu_h[r + 1]]
            # the stored K and Q may sit one rounding (2 u16 of the value) from the plain ones'
            # where float32 and float64 fall on two sides of a tie; in the mean that stays below u16
            assert np.linalg.norm(go - wo) <= 4 * U16 * np.linalg.norm(wo)
            assert np.abs(gl - wl).max() <= 2 * U16 * 8
        lens, n_free = lens2, n_free2
        lens_h, n_free_h = want[0], want[4]
    # requests end, their pages come back, and a new one takes them
    lens, n_free = api.kv_release(page, table, lens, dev([1, 0, 1, 0, 0]), free, n_free)
    lens_h, n_free_h = P.release(lens_h, [1, 0, 1, 0, 0], table_h, free_h, n_free_h, page)
    assert np.array_equal(host(table), table_h) and np.array_equal(host(lens), lens_h) and int(n_free) == n_free_h
    lens2, cu, slots, pos, n_free = api.kv_extend(page, table, lens, dev([30, 1, 0, 0, 0]), free, n_free, 31)
    want = P.extend(lens_h, [30, 1, 0, 0, 0], table_h, free_h, n_free_h, page, 31)
    assert np.array_equal(host(slots), want[2]) and np.array_equal(host(table), table_h)


def test_prompt_through_the_pages_is_the_ring_forward():
    b, s, hq, hkv, d = 2, 512, 4, 2, 128
    g = torch.Generator().manual_seed(40)
    q, k, v = (torch.randn((b, s, h, d), generator=g).to(torch.bfloat16).to(DEV) for h in (hq, hkv, hkv))
    rp = api.Problem(batch=b, heads_q=hq, heads_kv=hkv, head_dim=d, cp=2, seqlen=s)
    want_o, want_l = api.ring_attn_fwd(rp, q, k, v)
    page = 64
    kv = make_cache(b * s // page, page, hkv, d, torch.bfloat16, "head")
    order = torch.randperm(b * s // page, generator=g)
    table = order.view(b, -1).to(**I32)
    slots = (table.long()[:, :, None] * page + torch.arange(page, device=DEV)).view(-1).to(torch.int32)
    api.kv_append(kv, slots, k.flatten(0, 1), v.flatten(0, 1))
    p = api.PagedProblem(kv, hq, max_new=s)
    o, lse = api.paged_attn_fwd(p, q.flatten(0, 1), table, dev([0, s, 2 * s]), dev([s, s]))
    assert float((lse.view(b, s, hq) - want_l).abs().max()) <= 1e-5 * 8
    diff = (o.view(b, s, hq, d).double() - want_o.double())
    assert float(diff.norm()) <= 2 * U16 * float(want_o.double().norm())


def test_multi_axis_positions_through_the_ring_and_back():
    # Q and K rotated, ring attention forward and backward, gradients turned
    # back: against the plain formula in float64
    from oracle import attention as A
    s, hq, hkv, d, sections = 256, 2, 1, 64, [8, 12, 12]
    g = torch.Generator().manual_seed(41)
    q, k, v, do = (torch.randn((1, s, h, d), generator=g).to(DEV) for h in (hq, hkv, hkv, hq))
    pos = np.stack([np.arange(s) // 64, np.arange(s) % 64 // 8, np.arange(s) % 8])
    rope = api.Rope(sections)
    qr, kr = api.rope_axes(rope, dev(pos), q[0], k[0])
    p = api.Problem(batch=1, heads_q=hq, heads_kv=hkv, head_dim=d, cp=2, seqlen=s, dtype=torch.float32)
    o, lse = api.ring_attn_fwd(p, qr[None], kr[None], v)
    dq, dk, dv = api.ring_attn_bwd(p, qr[None], kr[None], v, o, lse, do)
    dq, dk = api.rope_axes(rope, dev(pos), dq[0], dk[0], inverse=True)
    qh, kh = P.rope_axes(f64(q)[0], pos, sections), P.rope_axes(f64(k)[0], pos, sections)
    ro, _ = A.attention_forward_bshd(qh[None], kh[None], f64(v))
    rq, rk, rv = A.attention_backward_bshd(qh[None], kh[None], f64(v), f64(do))
    rq, rk = P.rope_axes(rq[0], pos, sections, inverse=True), P.rope_axes(rk[0], pos, sections, inverse=True)
    for got, want in ((o, ro), (dq, rq), (dk, rk), (dv, rv)):
        assert np.abs(f64(got) - want).max() <= 1e-5 * max(1.0, np.abs(want).max())


def test_offsets_past_32_bits():
    # 40000 pages of 64 tokens, 8 heads, 128: the last pages start past 2^31 elements
    pages, page, hkv, d, hq = 40000, 64, 8, 128, 16
    kv = api.PagedKV(*(torch.empty((pages, page, hkv, d), dtype=torch.bfloat16, device=DEV) for _ in range(2)))
    assert (pages - 3) * kv.k_cache.stride(0) > 2 ** 31
    lens = [130, 70]
    table = np.array([[39999, 7, 39990], [39995, 39998, -1]])
    g = torch.Generator().manual_seed(50)
    rows = sum(lens)
    k, v = (torch.randn((rows, hkv, d), generator=g).to(torch.bfloat16).to(DEV) for _ in range(2))
    slots = np.concatenate([table[r][np.arange(n) // page] * page + np.arange(n) % page for r, n in enumerate(lens)])
    api.kv_append(kv, dev(slots), k, v)
    at = torch.from_numpy(slots).to(DEV)
    assert torch.equal(kv.k_cache.view(-1, hkv, d)[at], k) and torch.equal(kv.v_cache.view(-1, hkv, d)[at], v)
    few_k, few_v = (np.zeros((6, page, hkv, d)) for _ in range(2))  # the five pages alone, for the plain way
    small = np.array([[0, 1, 2], [3, 4, 5]])
    for big, little in zip(table.ravel()[:5], small.ravel()):
        few_k[little], few_v[little] = f64(kv.k_cache[int(big)]), f64(kv.v_cache[int(big)])
    for new in ([1, 1], [40, 30]):
        cu = np.concatenate([[0], np.cumsum(new)])
        q = torch.randn((sum(new), hq, d), generator=g).to(torch.bfloat16).to(DEV)
        p = api.PagedProblem(kv, hq, max_new=max(new))
        o, lse = api.paged_attn_fwd(p, q, dev(table), dev(cu), dev(lens))
        wo, wl = P.attention(f64(q), few_k, few_v, small, cu, lens)
        assert np.linalg.norm(f64(o) - wo) <= 2 * U16 * np.linalg.norm(wo)
        assert np.abs(f64(lse) - wl).max() <= 1e-4


def test_a_group_wider_than_a_pairs_tile():
    new, lens, hq = [3, 1, 9], [40, 130, 9], 130
    for dtype, d in ((torch.bfloat16, 128), (torch.bfloat16, 64), (torch.float32, 64)):
        kv, q, table, cu = paged_inputs(new, lens, hq, 1, d, 16, dtype, seed=51)
        p = api.PagedProblem(kv, hq, max_new=9)
        o, lse = api.paged_attn_fwd(p, q, dev(table), dev(cu), dev(lens))
        check_attention(kv, q, table, cu, lens, o, lse)


def test_a_serving_step_captured_and_replayed():
    """extend, append with a rotation and attention in one graph; between
    replays the host only copies the lengths that the step left and new rows."""
    n, page, hq, hkv, d, dtype, width, pages, rows = 3, 16, 4, 2, 64, torch.bfloat16, 8, 24, 5
    kv = make_cache(pages, page, hkv, d, dtype, "token")
    rope = api.Rope([32], adjacent=True)
    table, free = torch.full((n, width), -1, **I32), torch.arange(pages, **I32)
    lens, add, n_free = torch.zeros(n, **I32), torch.zeros(n, **I32), torch.full((1,), pages, **I32)
    x = torch.zeros((rows, hq + 2 * hkv, d), dtype=dtype, device=DEV)
    p = api.PagedProblem(kv, hq, max_new=3)
    ws = api.paged_workspace(p)
    o, lse = torch.zeros((rows, hq, d), dtype=dtype, device=DEV), torch.zeros((rows, hq), device=DEV)
    q_out = torch.zeros((rows, hq, d), dtype=dtype, device=DEV)

    def step():
        lens2, cu, slots, pos, n_free2 = api.kv_extend(page, table, lens, add, free, n_free, rows)
        api.kv_append(kv, slots, x[:, hq:hq + hkv], x[:, hq + hkv:], rope=rope, pos=pos, q=x[:, :hq], q_out=q_out)
        api.paged_attn_fwd(p, q_out, table, cu, lens2, ws=ws, out=o, lse=lse)
        lens.copy_(lens2)
        n_free.copy_(n_free2)
        return cu

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()                                                  # nothing to add
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            cu = step()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.Generator().manual_seed(52)
    keys, values = [[] for _ in range(n)], [[] for _ in range(n)]
    for adds in ([2, 0, 3], [1, 3, 1], [1, 1, 1], [0, 2, 0]) * 3:
        add.copy_(dev(adds))
        x.copy_(torch.randn(x.shape, generator=g).to(dtype))
        before = host(lens)
        graph.replay()
        c = host(cu)
        assert c.tolist() == [0] + np.cumsum(adds).tolist() and (host(lens) == before + adds).all()
        pos = np.zeros((1, rows), dtype=np.int64)
        for r in range(n):
            pos[0, c[r]:c[r + 1]] = before[r] + np.arange(adds[r])
        rnd = lambda a: f64(torch.from_numpy(a).to(dtype))  # noqa: E731
        qr = rnd(P.rope_axes(f64(x[:, :hq]), pos, [32], adjacent=True))
        kr, vr = rnd(P.rope_axes(f64(x[:, hq:hq + hkv]), pos, [32], adjacent=True)), f64(x[:, hq + hkv:])
        for r in range(n):
            keys[r] += list(kr[c[r]:c[r + 1]])
            values[r] += list(vr[c[r]:c[r + 1]])
            if adds[r] == 0:
                continue
            kk, vv = (np.stack(a)[None] for a in (keys[r], values[r]))
            wo, wl = P.attention(qr[c[r]:c[r + 1]], kk, vv, np.zeros((1, 1), dtype=np.int64), [0, adds[r]], [kk.shape[1]])
            assert np.linalg.norm(f64(o)[c[r]:c[r + 1]] - wo) <= 4 * U16 * np.linalg.norm(wo)
            assert np.abs(f64(lse)[c[r]:c[r + 1]] - wl).max() <= 2 * U16 * 8


FIRST_CALL = """
import torch
from tile_attention_lse_gb300 import api
g = torch.Generator().manual_seed(60)
i32 = dict(dtype=torch.int32, device="cuda:0")
kv = api.PagedKV(*(torch.randn((9, 16, 2, 128), generator=g).to("cuda:0", torch.bfloat16) for _ in range(2)))
x = torch.randn((40, 8, 128), generator=g).to("cuda:0", torch.bfloat16)
lens, add = torch.tensor([20, 0], **i32), torch.tensor([39, 1], **i32)
table, free, n_free = torch.tensor([[3, 4, -1, -1], [-1] * 4], **i32), torch.arange(5, 9, **i32), torch.tensor([4], **i32)
rope = api.Rope([64])
p = api.PagedProblem(kv, 4, max_new=MAX_NEW)
ws = api.paged_workspace(p)

def step():
    t = table.clone()
    lens2, cu, slots, pos, _ = api.kv_extend(16, t, lens, add, free, n_free, 40)
    q = api.kv_append(kv, slots, x[:, 4:6], x[:, 6:], rope=rope, pos=pos, q=x[:, :4])
    return api.paged_attn_fwd(p, q, t, cu, lens2, ws=ws)

torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    o, lse = step()
graph.replay()
o2, lse2 = step()
assert torch.equal(o, o2) and torch.equal(lse, lse2) and bool(torch.isfinite(lse).all()) and api.device_error() == 0
"""


@pytest.mark.parametrize("max_new", [1, 39])
def test_the_first_calls_of_a_process_are_captured(max_new):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    res = subprocess.run([sys.executable, "-c", FIRST_CALL.replace("MAX_NEW", str(max_new))], cwd=root,
                         capture_output=True, text=True, timeout=300)
    assert res.returncode == 0, res.stderr[-2000:]


def test_serving_launches_are_counted_and_timed():
    kv, q, table, cu = paged_inputs([1, 60], [40, 100], 4, 2, 64, 16, torch.bfloat16, seed=61)
    p = api.PagedProblem(kv, 4, max_new=60)
    args = (p, q, dev(table), dev(cu), dev([40, 100]))
    plain = api.paged_attn_fwd(*args)
    api.profile_read()
    api.profile_enable(True)
    timed = api.paged_attn_fwd(*args)
    api.rope_axes(api.Rope([32]), dev(np.arange(61)), q)
    api.kv_release(16, dev(table), dev([40, 100]), dev([0, 0]), dev([0]), dev([0]))
    api.profile_enable(False)
    got = api.profile_read()
    assert all(torch.equal(a, b) for a, b in zip(plain, timed))
    want = {"paged": 2, "paged_merge": 1, "head_rows": 1, "kv_tables": 1}
    assert {k: n for k, (_, n) in got.items() if n} == want and all(got[k][0] > 0 for k in want)


@pytest.mark.parametrize("dtype,new,max_new", [(torch.bfloat16, 3, 3), (torch.bfloat16, 8, 8), (torch.bfloat16, 90, 90),
                                               (torch.float32, 1, 1), (torch.float32, 11, 11)])
@pytest.mark.parametrize("ctx", [40, 9000])
def test_a_row_that_is_not_a_number_says_so(dtype, new, max_new, ctx):
    """A NaN in a row of q is in its O and its LSE, whether its tile is whole
    or cut into pieces, and in no other row."""
    lens = [ctx + new, 70]
    kv, q, table, cu = paged_inputs([new, 1], lens, 4, 1, 128, 64, dtype, seed=62)
    p = api.PagedProblem(kv, 4, max_new=max_new)
    row = new // 2
    bad = q.clone()
    bad[row, 2, 5] = float("nan")
    o, lse = api.paged_attn_fwd(p, bad, dev(table), dev(cu), dev(lens))
    assert bool(torch.isnan(o[row, 2]).all()) and bool(torch.isnan(lse[row, 2]))
    o[row, 2], lse[row, 2] = 0, 0
    keep = torch.ones_like(lse, dtype=torch.bool)
    keep[row, 2] = False
    want_o, want_lse = api.paged_attn_fwd(p, q, dev(table), dev(cu), dev(lens))
    assert bool(torch.isfinite(o).all()) and bool(torch.isfinite(lse).all())
    # the other rows' states may be rescaled at other tiles: a few float32 roundings, and O's own
    assert float((lse - want_lse)[keep].abs().max()) <= 64 * U32 * 16
    assert float((o.double() - want_o.double())[keep].abs().max()) <= 2 * HALF[dtype] * float(want_o.abs().max()) + 64 * U32


# The first table call of its process: no earlier, larger one has raised the
# kernel's limit of dynamic shared memory.
EXTEND_FIRST = """
import torch
from tile_attention_lse_gb300 import api
n, i32 = N_REQS, dict(dtype=torch.int32, device="cuda:0")
table, free = torch.full((n, 2), -1, **i32), torch.arange(n, **i32)
lens, cu, slots, pos, n_free = api.kv_extend(16, table, torch.zeros(n, **i32), torch.ones(n, **i32), free,
                                             torch.full((1,), n, **i32), n)
at = torch.arange(n + 1, **i32)
assert torch.equal(lens, torch.ones_like(lens)) and torch.equal(cu, at) and int(n_free) == 0
assert torch.equal(slots, (n - 1 - at[:n]) * 16) and not bool(pos.any())
assert torch.equal(table[:, 0], n - 1 - at[:n]) and bool((table[:, 1] == -1).all())
"""


@pytest.mark.parametrize("n", [6016, 6017, 6079, 6144, 6145])
def test_the_first_extend_of_a_process_takes_any_number_of_requests(n):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    res = subprocess.run([sys.executable, "-c", EXTEND_FIRST.replace("N_REQS", str(n))], cwd=root, capture_output=True,
                         text=True, timeout=300)
    assert res.returncode == 0, res.stderr[-2000:]


@pytest.mark.parametrize("n", [6078, 6079, 6144, 6145, 16384])
def test_extend_of_thousands_of_requests(n):
    rng = np.random.default_rng(n)
    table, lens, add, free, n_free, rows = table_case(n, 16, 4, rng.integers(0, 3, n), rng.integers(0, 60, n), 2 * n, 7, n)
    t, want_t = dev(table), table.copy()
    want = P.extend(lens, add, want_t, free, n_free, 16, rows)
    got = api.kv_extend(16, t, dev(lens), dev(add), dev(free), dev([n_free]), rows)
    for g, w, what in zip(got, want, ("lens", "cu", "slots", "pos", "n_free")):
        assert np.array_equal(host(g).ravel(), np.ravel(w)), what
    assert np.array_equal(host(t), want_t)


def test_calls_by_public_functions_alone():
    # where PyTorch lacks the private shortcuts to streams and tensors
    script = """
import sys
import torch
del torch._C._cuda_getCurrentRawStream
sys.modules["torch._C._dynamo.guards"] = None
""" + FIRST_CALL.replace("MAX_NEW", "39")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    res = subprocess.run([sys.executable, "-c", script], cwd=root, capture_output=True, text=True, timeout=300)
    assert res.returncode == 0, res.stderr[-2000:]


@pytest.mark.parametrize("room", [0, 40, 5000])
def test_release_passes_over_pages_that_were_given_back(room):
    # requests with a window: -1 in front (all of the table, some, none), a hole,
    # more than 1024 pages in one request, the pool too small for all
    page, width = 16, 1300
    lens = np.array([20800, 0, 33, 400, 16 * 1100, 70, 1, 64])
    rng = np.random.default_rng(70)
    have = -(-lens // page)
    table = np.full((len(lens), width), -7, dtype=np.int64)
    ids = rng.permutation(int(have.sum()))
    at = 0
    for r, n in enumerate(have):
        table[r, :n] = ids[at:at + n]
        at += n
    table[0, :1100] = -1
    table[3, :have[3]] = -1
    table[4, [0, 7, 1024, 1099]] = [-1, -5, -2 ** 31, -1]
    done = np.array([1, 1, 0, 1, 1, 1, 0, 1])
    pool, n_free = np.concatenate([[100001, 100002], np.full(room, -9)]), 2
    t, f = dev(table), dev(pool)
    want_t, want_f = table.copy(), pool.copy()
    want = P.release(lens, done, want_t, want_f, n_free, page)
    got = api.kv_release(page, t, dev(lens), dev(done), f, dev([n_free]))
    assert np.array_equal(host(got[0]), want[0]) and int(got[1]) == want[1]
    assert np.array_equal(host(t), want_t) and np.array_equal(host(f), want_f)
    # what the pool then holds is exactly the pages of the requests that ended, each once
    freed = sorted(x for r in np.nonzero(done)[0] for x in table[r, :have[r]] if x >= 0)
    back = sorted(host(f)[n_free:want[1]])
    assert min(back, default=0) >= 0 and len(back) == min(len(freed), room)
    assert back == freed if room >= len(freed) else set(back) <= set(freed)


def test_window_pages_given_back_are_granted_again():
    # a request slides its window, the caller gives the pages in front back, the
    # request ends, a new one takes all pages: each once, none missing
    page, width, pages = 16, 8, 8
    table, lens = torch.full((2, width), -1, **I32), torch.zeros(2, **I32)
    free, n_free = torch.arange(pages, **I32), torch.full((1,), pages, **I32)
    lens, _, _, _, n_free = api.kv_extend(page, table, lens, dev([100, 0]), free, n_free, 100)
    gone = host(table)[0, :3]                        # the caller: three pages in front of the window
    free[int(n_free):int(n_free) + 3] = dev(gone)
    table[0, :3] = -1
    n_free = n_free + 3
    lens, n_free = api.kv_release(page, table, lens, dev([1, 0]), free, n_free)
    assert int(n_free) == pages and sorted(host(free)) == list(range(pages))
    lens, cu, slots, pos, n_free = api.kv_extend(page, table, lens, dev([0, 128]), free, n_free, 128)
    assert int(n_free) == 0 and sorted(host(slots)) == list(range(128)) and sorted(host(table)[1]) == list(range(pages))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new,lens", [([700], [9000]), ([1, 300, 1, 90], [5000, 4000, 64, 900]), ([3, 1], [20, 9000])])
def test_the_schedule_is_the_launches_division(d, new, lens):
    # the states that the launches leave in the workspace are those of the pieces that
    # the host's division cuts: the same slots, the same rows of each
    hq, hkv, page = 8, 2, 16
    kv, q, table, cu = paged_inputs(new, lens, hq, hkv, d, page, torch.bfloat16, seed=71)
    p = api.PagedProblem(kv, hq, max_new=max(new))
    pieces, grid = api.paged_schedule(p, cu, lens, int(cu[-1]), table.shape[1])
    ws = api.paged_workspace(p)
    ws.fill_(255)
    api.paged_attn_fwd(p, q, dev(table), dev(cu), dev(lens), ws=ws)
    pair, some = max(new) * hq // hkv > 32, len(new) > 1
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    R = (256 if pair else 16, 16)                              # packed rows of a state
    blocks = (sms // 2 if pair else sms, sms if pair and some else 0)
    states = sum(2 * n * r for n, r in zip(blocks, R))
    part_l = ws.view(torch.int32)[states * d:states * (d + 1)]
    wrote = host(part_l != -1).astype(bool)
    first = grid - sms if pair and some else grid               # blocks of the pair launch, or of the only one
    want = np.zeros(states, dtype=bool)
    for block, r, h, row0, nrows, k0, k1, slot in pieces.tolist():
        if slot < 0:
            continue
        at = slot * R[0] if block < first else 2 * blocks[0] * R[0] + (slot - 2 * first) * R[1]
        want[at:at + nrows] = True
    assert want.any() and np.array_equal(wrote, want)


def exact_turns(base, pairs, pos):
    """Sine and cosine of pos base^(-i / pairs) for i < pairs, from 70 decimal digits."""
    from decimal import Decimal, getcontext
    getcontext().prec = 70
    two_pi = 2 * Decimal("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899863")
    ln = Decimal(base).ln()
    out = np.zeros((2, pairs))
    for i in range(pairs):
        x = (Decimal(int(pos)) * (-ln * i / pairs).exp()) % two_pi
        x -= two_pi * (x / two_pi).to_integral_value()
        term, sums = Decimal(1), [Decimal(0), Decimal(0)]
        for n in range(60):                                     # x^59 / 59! < 1e-50 for |x| <= pi
            sums[n % 2] += term if n % 4 < 2 else -term
            term = term * x / (n + 1)
        out[:, i] = float(sums[1]), float(sums[0])
    return out


@pytest.mark.parametrize("pos", [2 ** 31 - 1, -2 ** 31, 2 ** 30 + 12345, -987654321, 2 ** 24 + 1, 1000003, -131071, 17])
@pytest.mark.parametrize("base", [10000.0, 500000.0, 1.0])
def test_angles_are_as_exact_as_the_header_says(pos, base):
    # a pair (1, 0) turns into its cosine and sine: off by the angle's error, 2^-26
    # + 2^-32 + |pos| 2^-53 turns, and by one unit in the last place of sincospif
    x = torch.zeros((1, 1, 128), device=DEV)
    x[..., :64] = 1.0
    y = f64(api.rope_axes(api.Rope([64], base=base), dev([pos]), x))[0, 0]
    sine, cosine = exact_turns(int(base), 64, pos)
    tol = 2 * np.pi * (2.0 ** -26 + 2.0 ** -32 + abs(pos) * 2.0 ** -53) + 2.0 ** -23
    assert np.abs(y[:64] - cosine).max() <= tol and np.abs(y[64:] - sine).max() <= tol


@pytest.mark.parametrize("dtype,d", [(torch.bfloat16, 128), (torch.bfloat16, 64), (torch.float32, 64)])
@pytest.mark.parametrize("order", [(1, 0, 2), (2, 0, 1), (2, 1, 0), (1, 2, 0), (0, 2, 1)])
def test_pages_tokens_and_heads_in_any_order(order, dtype, d):
    # order: the memory order of pages (0), tokens (1) and heads (2), outermost first
    new, lens, hq, hkv, page = [1, 90, 2], [300, 200, 33], 8, 2, 32
    kv, q, table, cu = paged_inputs(new, lens, hq, hkv, d, page, dtype, seed=72)
    back = [order.index(i) for i in range(3)]
    k, v = (x.permute(*order, 3).contiguous().permute(*back, 3) for x in (kv.k_cache, kv.v_cache))
    other = api.PagedKV(k, v)
    assert tuple(np.argsort([-s for s in k.stride()[:3]], kind="stable")) == order
    # every token is written again through the slots
    rows = sum(lens)
    slots = np.concatenate([table[r][np.arange(n) // page] * page + np.arange(n) % page for r, n in enumerate(lens)])
    at = torch.from_numpy(slots).to(DEV)
    flat = [x.reshape(-1, hkv, d)[at].contiguous() for x in (kv.k_cache, kv.v_cache)]
    other.k_cache.fill_(float("nan")), other.v_cache.fill_(float("nan"))
    api.kv_append(other, dev(slots), *flat)
    for a, b in ((other.k_cache, flat[0]), (other.v_cache, flat[1])):
        assert torch.equal(a.reshape(-1, hkv, d)[at], b) and int(torch.isnan(a[..., 0]).sum()) == (a.shape[0] * page - rows) * hkv
    for max_new in (90, 2):
        args = (q, dev(table), dev(cu), dev(lens))
        o, lse = api.paged_attn_fwd(api.PagedProblem(other, hq, max_new=max_new), *args)
        check_attention(kv, q, table, cu, lens, o, lse)
        want = api.paged_attn_fwd(api.PagedProblem(kv, hq, max_new=max_new), *args)
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("dtype,max_new", [(torch.bfloat16, 3), (torch.bfloat16, 64), (torch.float32, 3)])
def test_lengths_outside_the_table_and_the_rows_are_clamped(dtype, max_new):
    # the same bits as a call with the clamped lengths: a request longer than its
    # table, one of negative length, offsets in front of and behind the rows of q
    lens, page = [48, 48, 48], 16
    kv, q, table, _ = paged_inputs([0, 0, 0], lens, 4, 2, 128, page, dtype, seed=73, tail=9)
    table = table[:, :3]                                     # 48 keys of each
    p = api.PagedProblem(kv, 4, max_new=max_new)
    for cu, n, cu_c, n_c in (([-3, 2, 99, 120], [1000, -5, 7], [0, 2, 9, 9], [48, 0, 7]),
                             ([0, 0, -4, 6], [48, 2 ** 31 - 1, 2 ** 31 - 1], [0, 0, 0, 6], [48, 48, 48]),
                             ([4, 9, 9, 9], [-2 ** 31, 3, 1], [4, 9, 9, 9], [0, 3, 1])):
        got, want = [], []
        for c, x, out in ((cu, n, got), (cu_c, n_c, want)):
            o, lse = torch.full(q.shape, 7.0, dtype=dtype, device=DEV), torch.full(q.shape[:2], 7.0, device=DEV)
            out += api.paged_attn_fwd(p, q, dev(table), dev(c), dev(x), out=o, lse=lse)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        inside = np.zeros(q.shape[0], dtype=bool)
        inside[cu_c[0]:cu_c[-1]] = True
        assert np.array_equal(host((got[1] != 7).all(1)), inside) and np.array_equal(host((got[1] == 7).all(1)), ~inside)
        check = [r for r in range(3) if cu_c[r + 1] > cu_c[r]]
        for r in check:
            rows = slice(cu_c[r], cu_c[r + 1])
            check_attention(kv, q[rows], table[r:r + 1], [0, cu_c[r + 1] - cu_c[r]], n_c[r:r + 1], got[0][rows], got[1][rows])


def test_tables_append_and_release_on_another_stream_captured():
    # every table call in one graph on a stream of its own, replayed until the pool has been through twice;
    # q is rotated in place
    page, n, width, pages, rows = 16, 4, 4, 10, 20
    kv = make_cache(pages, page, 2, 64, torch.float32, "token", fill=0.0)
    rope = api.Rope([8, 24], interleaved=True)
    table, lens, free = torch.full((n, width), -1, **I32), torch.zeros(n, **I32), torch.arange(pages, **I32)
    add, done, n_free = torch.zeros(n, **I32), torch.zeros(n, **I32), torch.full((1,), pages, **I32)
    x = torch.randn((rows, 4, 64), generator=torch.Generator().manual_seed(74)).to(DEV)
    q = torch.zeros((rows, 2, 64), device=DEV)

    def step():
        lens2, cu, slots, pos, free2 = api.kv_extend(page, table, lens, add, free, n_free, rows)
        api.kv_append(kv, slots, x[:, :2], x[:, 2:], rope=rope, pos=torch.stack([pos, pos // 3]), q=q, q_out=q)
        lens3, free3 = api.kv_release(page, table, lens2, done, free, free2)
        lens.copy_(lens3)
        n_free.copy_(free3)
        return slots, pos

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            slots, pos = step()
    torch.cuda.current_stream().wait_stream(s)
    t_h, l_h, f_h, nf_h = np.full((n, width), -1), np.zeros(n, dtype=np.int64), np.arange(pages), pages
    rng = np.random.default_rng(75)
    for i in range(12):
        adds, ends = rng.integers(0, 9, n), (rng.random(n) < 0.4).astype(np.int64)
        add.copy_(dev(adds))
        done.copy_(dev(ends))
        q.copy_(x[:, :2])
        graph.replay()
        l_h, _, want_s, want_p, nf_h = P.extend(l_h, adds, t_h, f_h, nf_h, page, rows)
        l_h, nf_h = P.release(l_h, ends, t_h, f_h, nf_h, page)
        assert np.array_equal(host(slots), want_s) and np.array_equal(host(pos), want_p)
        assert np.array_equal(host(table), t_h) and np.array_equal(host(free), f_h) and int(n_free) == nf_h
        there = want_s >= 0
        want = P.rope_axes(f64(x[:, :2]), np.stack([want_p, want_p // 3]), [8, 24], interleaved=True)
        tol = 12 * float(x.abs().max()) * U32 + U32 * 1.5 * float(x.abs().max())
        assert np.abs(f64(q) - want)[there].max(initial=0.0) <= tol
        assert torch.equal(q[dev(~there, torch.bool)], x[:, :2][dev(~there, torch.bool)])    # rows without a slot stay
        flat = f64(kv.k_cache).reshape(-1, 2, 64)
        assert np.abs(flat[want_s[there]] - want[there]).max(initial=0.0) <= tol
