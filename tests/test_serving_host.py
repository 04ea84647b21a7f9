"""CPU-only checks of the serving entry points: refusals and the division of a
paged attention over the blocks of its launch (no GPU calls)."""

import ctypes
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from tile_attention_lse_gb300 import api

OK, INVALID, ALIGN, UNSUP = 0, -1, -2, -3


def _kv(pages=9, page=16, hkv=2, d=128, dtype=torch.bfloat16):
    t = torch.zeros((pages, page, hkv, d), dtype=dtype)
    return api.PagedKV(t, t.clone())


def _problem(heads_q=8, kv=None, **kw):
    return api.PagedProblem(_kv() if kv is None else kv, heads_q, **kw)


def test_descriptor_refusals():
    assert api.validate_paged(_problem()) == OK
    assert api.validate_paged(_problem(heads_q=7)) == UNSUP            # not a multiple of 2
    assert api.validate_paged(_problem(heads_q=0)) == INVALID
    assert api.validate_paged(_problem(max_new=-1)) == INVALID
    assert api.validate_paged(_problem(window=-1)) == INVALID
    assert api.validate_paged(_problem(window=1 << 30)) == INVALID
    assert api.validate_paged(_problem(softmax_scale=-1.0)) == INVALID
    assert api.validate_paged(_problem(softmax_scale=float("nan"))) == INVALID
    for page in (4, 12, 512):
        assert api.validate_paged(_problem(kv=_kv(page=page))) == UNSUP
    assert api.validate_paged(_problem(kv=_kv(d=96))) == UNSUP
    assert api.lib().cp_validate_paged_desc(None) == INVALID
    for dt in (torch.float32, torch.bfloat16):
        for d in (64, 128):
            assert api.paged_workspace_bytes(_problem(kv=_kv(d=d, dtype=dt))) > 0
    assert api.paged_workspace_bytes(_problem(heads_q=7)) == 0


def test_cache_strides():
    t = torch.zeros((5, 2, 16, 2, 128), dtype=torch.bfloat16)          # K and V side by side
    assert api.validate_paged(_problem(kv=api.PagedKV(t[:, 0], t[:, 1]))) == OK
    h = torch.zeros((5, 2, 16, 128), dtype=torch.bfloat16)             # head-major pages
    assert api.validate_paged(_problem(kv=api.PagedKV(h.transpose(1, 2), h.transpose(1, 2)))) == OK
    odd = torch.zeros((5, 16, 2, 132), dtype=torch.bfloat16)[..., :128]
    assert api.validate_paged(_problem(kv=api.PagedKV(odd, odd))) == ALIGN
    flat = torch.zeros(5 * 16 * 2 * 128 + 1, dtype=torch.bfloat16)[1:].view(5, 16, 2, 128)
    assert api.validate_paged(_problem(kv=api.PagedKV(flat, flat))) == ALIGN
    with pytest.raises(ValueError):
        api.PagedKV(t[:, 0], h)
    with pytest.raises(ValueError):
        api.PagedKV(h[0], h[0])


def _attn(p, n=2, rows=5, blocks=4, q=256, stride=1024, table=256, cu=256, lens=256, o=256, lse=256, ws=256,
          ws_bytes=1 << 40):
    # pointers are never read: every call here is refused on the host or has no work
    return api.lib().cp_paged_attn_fwd(p._ref, n, rows, blocks, q, stride, table, cu, lens, o, lse, ws, ws_bytes, None)


def test_attention_argument_refusals():
    p = _problem()
    assert _attn(p, n=-1) == INVALID and _attn(p, rows=-1) == INVALID and _attn(p, blocks=0) == INVALID
    for name in ("q", "table", "cu", "lens", "o", "lse", "ws"):
        assert _attn(p, **{name: None}) == INVALID, name
    assert _attn(p, ws=128) == INVALID                                   # 256-byte alignment
    assert _attn(p, stride=1023) == INVALID and _attn(p, stride=1028) == ALIGN
    assert _attn(p, q=264) == ALIGN and _attn(p, o=264) == ALIGN
    assert _attn(p, ws_bytes=api.paged_workspace_bytes(p) - 1) == -4
    assert _attn(p, blocks=1 << 28) == UNSUP and _attn(p, rows=1 << 30) == UNSUP
    assert _attn(p, n=0, q=None) == OK and _attn(p, rows=0, q=None) == OK  # no work: nothing is read


def _rope(**kw):
    kw = dict(dict(sections=[16, 24, 24]), **kw)
    return api.Rope(kw.pop("sections"), **kw)


def _rope_call(r, rows=3, d=128, dtype=1, hq=2, q=256, qs=256, qo=512, hk=0, k=None, ks=0, ko=None, pos=256):
    return api.lib().cp_rope_axes(None if r is None else r._ref, pos, rows, d, dtype, hq, q, qs, qo, hk, k, ks, ko, 0, None)


def test_rope_refusals():
    assert _rope_call(None) == INVALID
    assert _rope_call(_rope(), rows=0) == OK
    assert _rope_call(_rope(sections=[16, 24, 23])) == UNSUP             # 63 pairs
    assert _rope_call(_rope(sections=[40, 40])) == INVALID               # 80 pairs of 64
    assert _rope_call(_rope(sections=[-8, 16])) == INVALID
    assert _rope_call(_rope(sections=[0, 0])) == INVALID
    assert _rope_call(_rope(base=0.0)) == INVALID and _rope_call(_rope(base=float("inf"))) == INVALID
    with pytest.raises(ValueError):
        api.Rope([8] * 5)
    r = _rope()
    assert _rope_call(r, d=96) == UNSUP and _rope_call(r, dtype=2) == UNSUP and _rope_call(r, rows=-1) == INVALID
    assert _rope_call(r, hq=0) == INVALID and _rope_call(r, hk=1) == INVALID
    assert _rope_call(r, q=None) == INVALID and _rope_call(r, pos=None) == INVALID and _rope_call(r, qo=None) == INVALID
    assert _rope_call(r, qs=255) == INVALID and _rope_call(r, qs=260) == ALIGN
    assert _rope_call(r, q=264) == ALIGN and _rope_call(r, qo=520) == ALIGN
    assert _rope_call(r, qo=256, qs=512) == INVALID                      # in place with another stride


def _append(kv, rows=3, slots=256, k=256, ks=256, v=256, vs=256, rope=None, pos=None, hq=0, q=None, qs=0, qo=None):
    return api.lib().cp_kv_append(kv._ref, slots, rows, k, ks, v, vs, rope, pos, hq, q, qs, qo, None)


def test_append_refusals():
    kv, r = _kv(), _rope()
    assert _append(kv, rows=0) == OK and _append(kv, rows=-1) == INVALID
    for name in ("slots", "k", "v"):
        assert _append(kv, **{name: None}) == INVALID
    assert _append(kv, ks=255) == INVALID and _append(kv, vs=260) == ALIGN and _append(kv, k=264) == ALIGN
    assert _append(kv, rope=r._ref) == INVALID                           # no positions
    assert _append(kv, hq=2, q=256, qs=256, qo=512) == INVALID           # q without a rotation
    assert _append(kv, rope=r._ref, pos=256, hq=2, q=256, qs=255, qo=512) == INVALID
    assert _append(_kv(page=24), rows=0) == UNSUP


def _extend(n=3, blocks=4, page=16, rows=8, pool=5, lens=256, add=256, free=256, nf=256, table=256, lo=512, cu=512,
            slots=512, pos=512, nfo=512):
    return api.lib().cp_kv_extend(n, blocks, page, rows, pool, lens, add, free, nf, table, lo, cu, slots, pos, nfo, None)


def _release(n=3, blocks=4, page=16, pool=5, lens=256, done=256, free=256, nf=256, table=256, lo=512, nfo=512):
    return api.lib().cp_kv_release(n, blocks, page, pool, lens, done, free, nf, table, lo, nfo, None)


def test_table_refusals():
    for kw in (dict(n=-1), dict(blocks=0), dict(page=0), dict(rows=-1), dict(pool=-1), dict(lens=None), dict(add=None),
               dict(free=None), dict(nf=None), dict(table=None), dict(lo=None), dict(cu=None), dict(slots=None),
               dict(pos=None), dict(nfo=None), dict(lo=256), dict(nfo=256)):
        assert _extend(**kw) == INVALID, kw
    assert _extend(n=16385) == UNSUP and _extend(blocks=1 << 27) == UNSUP and _extend(rows=1 << 31) == UNSUP
    for kw in (dict(n=-1), dict(blocks=0), dict(page=0), dict(pool=-1), dict(lens=None), dict(done=None), dict(free=None),
               dict(nf=None), dict(table=None), dict(lo=None), dict(nfo=None), dict(lo=256), dict(nfo=256)):
        assert _release(**kw) == INVALID, kw
    assert _release(n=16385) == UNSUP and _release(blocks=1 << 27) == UNSUP


def test_python_refusals():
    i32 = dict(dtype=torch.int32)
    kv, z = _kv(), torch.zeros
    p = _problem(kv=kv)
    q, tab, cu, lens = z(4, 8, 128, dtype=torch.bfloat16), z((2, 3), **i32), z(3, **i32), z(2, **i32)
    for bad in (dict(q=q.float()), dict(q=q[:, :4]), dict(q=q[..., ::2]), dict(tab=tab.long()), dict(tab=tab[0]),
                dict(cu=cu[:2]), dict(lens=lens.long()), dict()):       # the last: no CUDA device
        a = dict(dict(q=q, tab=tab, cu=cu, lens=lens), **bad)
        with pytest.raises(ValueError):
            api.paged_attn_fwd(p, a["q"], a["tab"], a["cu"], a["lens"])
    with pytest.raises(ValueError):
        api.kv_append(kv, z(4, **i32), q[:, :2], q[:, :2], rope=_rope())
    with pytest.raises(ValueError):
        api.rope_axes(_rope(), z((2, 4), **i32), q)
    with pytest.raises(ValueError):
        api.kv_extend(16, tab, lens, lens[:1], lens, lens[:1], 4)


# ------------------------------------------------------------ the division ---
SHAPES = [
    # name, new tokens, cached lengths (with them), heads_q, heads_kv, max_new, causal, window
    ("one", [1], [777], 32, 8, 1, True, 0),
    ("one_key", [1], [1], 4, 4, 1, True, 0),
    ("batch", [1] * 64, list(range(1, 6400, 100)), 32, 8, 1, True, 0),
    ("none_and_empty", [0, 1, 0, 3, 0], [50, 0, 0, 3, 7], 8, 2, 3, True, 0),
    ("chunk", [301], [5000], 28, 4, 301, True, 0),
    ("mixed_window", [1, 1, 130, 1], [3000, 90, 1000, 1], 32, 8, 130, True, 128),
    ("not_causal", [9, 40], [40, 400], 40, 8, 40, False, 0),
    ("wide_group", [2, 5], [300, 20], 130, 1, 5, True, 0),
    ("more_new_than_cached", [20], [7], 8, 2, 20, True, 0),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("case", SHAPES, ids=[c[0] for c in SHAPES])
def test_every_visible_key_of_every_row_is_walked_once(case, dtype):
    _, new, lens, hq, hkv, max_new, causal, window = case
    p = _problem(heads_q=hq, kv=_kv(hkv=hkv, dtype=dtype), max_new=max_new, causal=causal, window=window)
    cu = np.concatenate([[0], np.cumsum(new)])
    width = -(-max(lens) // 16)
    pieces, grid = api.paged_schedule(p, cu, lens, int(cu[-1]), width)
    G = hq // hkv
    slots = {}
    seen = {}
    for block, r, h, row0, nrows, k0, k1, slot in pieces.tolist():
        assert 0 <= block < grid and 0 < nrows and row0 + nrows <= new[r] * G and 0 <= h < hkv
        assert 0 <= k0 <= k1 <= lens[r]
        if slot >= 0:
            assert slot // 2 == block and slot not in slots   # two states per block, each its own
            slots[slot] = True
        seen.setdefault((r, h, row0, nrows), []).append((k0, k1, slot, block))
    tiles = set()
    for (r, h, row0, nrows), parts in seen.items():
        tiles |= {(r, h, row0 + i) for i in range(nrows)}
        assert (len(parts) == 1) == (parts[0][2] == -1)
        # a cut tile: blocks in order, only its first piece in a second slot
        assert [b for *_, b in parts] == sorted(b for *_, b in parts)
        assert all(s % 2 == 0 for _, _, s, _ in parts[1:])
        pos = [lens[r] - new[r] + (row0 + i) // G for i in range(nrows)]
        hi = max(min(lens[r], x + 1) if causal else lens[r] for x in pos)
        lo = min(max(0, x - window + 1) if window else 0 for x in pos)
        keys = np.concatenate([np.arange(a, b) for a, b, _, _ in parts])
        assert keys.tolist() == list(range(min(lo, max(hi, 0)), max(hi, 0))), (r, h, row0)
    assert tiles == {(r, h, i) for r in range(len(new)) for h in range(hkv) for i in range(new[r] * G)}


def test_lengths_from_the_device_are_clamped():
    p = _problem(max_new=1)
    # offsets that fall, run past q's rows or are negative; lengths past the table and below zero
    pieces, _ = api.paged_schedule(p, [-3, 2, 1, 99], [1000, -5, 40], 6, 3)
    for block, r, h, row0, nrows, k0, k1, slot in pieces.tolist():
        assert 0 <= k0 <= k1 <= 48
    rows = {r: max(x[3] + x[4] for x in pieces.tolist() if x[1] == r) // 4 for r in {x[1] for x in pieces.tolist()}}
    assert rows == {0: 2, 2: 5}


def test_shares_are_even():
    p = _problem(heads_q=32, kv=_kv(hkv=8), max_new=1)
    lens = [131072, 5, 700, 40000]
    pieces, grid = api.paged_schedule(p, [0, 1, 2, 3, 4], lens, 4, 8192)
    load = np.bincount(pieces[:, 0], weights=(pieces[:, 6] - pieces[:, 5]), minlength=grid)
    # units of 64 keys and two for every tile's ends, in shares that differ by at most one unit
    units = 8 * sum(-(-n // 64) + 2 for n in lens)
    assert load.max() <= 64 * -(-units // grid)
    assert np.median(load) >= 0.97 * load.max()


# A PyTorch that was built without CUDA lacks these private functions.
WITHOUT_CUDA = """
import sys
import torch
del torch._C._cuda_getCurrentRawStream
sys.modules["torch._C._dynamo.guards"] = None
from tile_attention_lse_gb300 import api
t = torch.zeros((9, 16, 2, 128), dtype=torch.bfloat16)
p = api.PagedProblem(api.PagedKV(t, t), 8, max_new=3)
assert api.validate_paged(p) == 0 and api.paged_workspace_bytes(p) > 0
assert len(api.paged_schedule(p, [0, 3], [40], 3, 4)[0]) > 0
assert len(api.hybrid_schedule([128, 256], 4, 128)[0]) == 2
try:
    api.kv_extend(16, *(torch.zeros(s, dtype=torch.int32) for s in ((1, 4), (1,), (1,), (4,), (1,))), 3)
except ValueError:
    print("refused")
"""


def test_the_package_imports_without_cuda_in_pytorch():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    res = subprocess.run([sys.executable, "-c", WITHOUT_CUDA], cwd=root, capture_output=True, text=True, timeout=300,
                         env=dict(os.environ, CUDA_VISIBLE_DEVICES=""))
    assert res.returncode == 0 and res.stdout.strip() == "refused", res.stderr[-2000:]


def test_the_division_refuses_what_the_attention_refuses():
    p = _problem()
    cu, lens = np.array([0, 1], dtype=np.int32), np.array([777], dtype=np.int32)

    def schedule(rows=1, blocks=64, n=1, cu=cu, lens=lens):
        grid, count = ctypes.c_int32(-1), ctypes.c_int64(-1)
        at = [None if x is None else x.ctypes.data for x in (cu, lens)]
        return api.lib().cp_paged_schedule(p._ref, n, rows, blocks, *at, ctypes.byref(grid), ctypes.byref(count), None)

    assert schedule() == OK
    assert schedule(n=0) == INVALID and schedule(rows=-1) == INVALID and schedule(blocks=0) == INVALID
    assert schedule(cu=None) == INVALID and schedule(lens=None) == INVALID
    # table widths and rows at the limits, past them, and where a 32-bit or a
    # 64-bit product would wrap around to a small number
    assert schedule(blocks=1 << 26) == OK
    for blocks in ((1 << 26) + 1, 1 << 27, 1 << 28, 2 ** 31 - 1):
        assert schedule(blocks=blocks) == UNSUP == _attn(p, blocks=blocks), blocks
    assert schedule(rows=(1 << 29) - 257) == OK
    for rows in ((1 << 29) - 256, 1 << 30, 1 << 31, 1 << 60, 1 << 62, 2 ** 63 - 1):
        assert schedule(rows=rows) == UNSUP == _attn(p, rows=rows), rows
