"""CPU-only checks of cross attention: refusals and workspace sizes of its entry
points, and pins of its oracle (no GPU calls)."""

import numpy as np
import pytest
import torch

from oracle import cross as X
from tile_attention_lse_gb300 import api

OK, INVALID, ALIGN, UNSUP, WORK = 0, -1, -2, -3, -4


def problem(heads_q=8, heads_kv=2, head_dim=128, **kw):
    return api.CrossProblem(heads_q, heads_kv, head_dim, **kw)


# ------------------------------------------------------------- descriptor ---
def test_descriptor_refusals():
    v = api.validate_cross
    for dt in (torch.float32, torch.bfloat16):
        for d in (64, 128):
            assert v(problem(head_dim=d, dtype=dt)) == OK
    assert api.lib().cp_validate_cross_desc(None) == INVALID
    assert v(problem(heads_q=7)) == UNSUP
    assert v(problem(heads_q=0)) == INVALID
    assert v(problem(heads_kv=0)) == INVALID
    assert v(problem(head_dim=96)) == UNSUP
    assert v(problem(max_q=-1)) == INVALID
    for s in (-1.0, float("nan"), float("inf")):
        assert v(problem(softmax_scale=s)) == INVALID
    for p in (-0.1, 1.0, 1.5, 0.99999, float("nan")):
        assert v(problem(dropout=p)) == INVALID, p
    assert v(problem(dropout=0.999)) == OK
    bad = problem()
    bad._desc.dtype = 7
    assert v(bad) == UNSUP
    # dropout in bf16 packs a group's heads into one tile
    assert v(problem(heads_q=256, heads_kv=1, dropout=0.1)) == UNSUP
    assert v(problem(heads_q=256, heads_kv=1)) == OK
    assert v(problem(heads_q=256, heads_kv=1, dropout=0.1, dtype=torch.float32)) == OK


@pytest.mark.parametrize("buckets,distance,both,want", [
    (32, 128, True, OK), (32, 128, False, OK), (2, 1, False, OK), (4, 1, True, OK), (64, 65536, True, OK),
    (1, 8, False, INVALID), (2, 8, True, INVALID), (31, 128, True, INVALID), (-2, 8, False, INVALID),
    (32, 7, True, INVALID), (32, 15, False, INVALID), (66, 128, False, UNSUP), (32, 65537, False, UNSUP)])
def test_bucket_refusals(buckets, distance, both, want):
    assert api.validate_cross(problem(rel=api.RelBuckets(buckets, distance, both))) == want


def test_dropout_is_rounded_once():
    """The nearest multiple of 2^-15 of the caller's double, halves to even, which the descriptor's float holds."""
    for k in (0, 1, 2, 3276, 3277, 9830, 20000, 20001, 32766):
        for p in (k / 32768, (k + 0.5) / 32768, np.nextafter((k + 0.5) / 32768, 0), np.nextafter((k + 0.5) / 32768, 1)):
            got = problem(dropout=p)
            assert got._desc.dropout * 32768 == round(p * 32768) == round(got.dropout * 32768), p
    near = problem(dropout=1e-6)                                            # as none: no rng is asked for
    assert near.dropout == 0.0 and fwd(near, wb=16) == WORK


def test_workspace_sizes():
    w = api.cross_workspace_bytes
    p = problem()
    assert w(p, 3, 100, 200) > 0
    assert w(p, 3, 100, 200, True) >= w(p, 3, 100, 200)
    assert w(p, 3, 10 ** 6, 10 ** 6, True) >= 10 ** 6 * 8 * 128 * 4  # dQ's sums
    assert w(p, -1, 100, 200) == 0 and w(p, 3, -1, 200) == 0 and w(p, 3, 100, -1) == 0
    assert w(p, 3, 2 ** 31, 200) == 0 and w(p, 3, 100, 2 ** 30 + 1) == 0 and w(p, 2 ** 29, 100, 200) == 0
    assert w(problem(head_dim=96), 3, 100, 200) == 0
    with pytest.raises(api.CpError):
        api.cross_workspace(problem(head_dim=96), 3, 100, 200, device="cpu")


# ----------------------------------------------------------- calls refused ---
A = 4096  # an aligned address that nothing is read from: every call below is refused before


def fwd(p, n=2, rq=4, rk=6, q=A, qs=None, k=A, ks=None, v=A, vs=None, cu_q=A, cu_k=A, len_q=None, len_k=None, bias=None,
        rng=None, o=A, rest=None, lse=A, ws=A, wb=1 << 40):
    d = p.head_dim
    qs, ks, vs = (p.heads_q * d if qs is None else qs, p.heads_kv * d if ks is None else ks,
                  p.heads_kv * d if vs is None else vs)
    return api.lib().cp_cross_attn_fwd(p._ref, n, rq, rk, q, qs, k, ks, v, vs, cu_q, cu_k, len_q, len_k, bias, rng, o, rest,
                                       lse, ws, wb, None)


def bwd(p, n=2, rq=4, rk=6, q=A, qs=None, k=A, ks=None, v=A, vs=None, o=A, rest=None, lse=A, dout=A, ds=None, cu_q=A, cu_k=A,
        bias=None, rng=None, dq=A, dk=A, dv=A, dbias=None, ws=A, wb=1 << 40):
    d = p.head_dim
    qs, ks, vs, ds = (p.heads_q * d if qs is None else qs, p.heads_kv * d if ks is None else ks,
                      p.heads_kv * d if vs is None else vs, p.heads_q * d if ds is None else ds)
    return api.lib().cp_cross_attn_bwd(p._ref, n, rq, rk, q, qs, k, ks, v, vs, o, rest, lse, dout, ds, cu_q, cu_k, None, None,
                                       bias, rng, dq, dk, dv, dbias, ws, wb, None)


@pytest.mark.parametrize("call", [fwd, bwd])
def test_call_refusals(call):
    p = problem()
    for name in ("q", "k", "v", "cu_q", "cu_k", "o", "lse", "ws"):
        assert call(p, **{name: None}) == INVALID, name
    for name in ("n", "rq", "rk"):
        assert call(p, **{name: -1}) == INVALID, name
    assert call(p, rq=2 ** 31) == UNSUP and call(p, rk=2 ** 30 + 1) == UNSUP
    for name, width in (("qs", 8 * 128), ("ks", 256), ("vs", 256)):
        assert call(p, **{name: width - 8}) == INVALID, name
        assert call(p, **{name: width + 4}) == ALIGN, name
        assert call(p, **{name: 2 ** 40}) == UNSUP, name
    for name in ("q", "k", "v", "o"):
        assert call(p, **{name: A + 8}) == ALIGN, name
    assert call(p, ws=A + 16) == INVALID
    assert call(p, wb=16) == WORK
    assert call(p, bias=A) == INVALID                                       # a bias without buckets
    r = problem(rel=api.RelBuckets(32))
    assert call(r) == INVALID                                               # buckets without a bias
    assert call(problem(dropout=0.1)) == INVALID                            # no rng
    assert call(problem(dropout=0.1), rng=A + 4) == INVALID
    assert call(problem(dtype=torch.float32), rest=A) == INVALID
    assert call(problem(head_dim=96)) == UNSUP


def test_backward_refusals():
    p = problem()
    for name in ("dout", "dq", "dk", "dv"):
        assert bwd(p, **{name: None}) == INVALID, name
        assert bwd(p, **{name: A + 8}) == ALIGN, name
    assert bwd(p, ds=8 * 128 - 8) == INVALID
    assert bwd(p, ds=8 * 128 + 4) == ALIGN
    assert bwd(p, ds=2 ** 40) == UNSUP
    assert bwd(problem(rel=api.RelBuckets(32)), bias=A) == INVALID          # no dbias
    w = api.cross_workspace_bytes(p, 2, 4, 6, True)
    assert bwd(p, wb=w - 1) == WORK


def test_forward_without_rows_is_a_no_op():
    assert fwd(problem(), n=0, q=None, k=None, v=None, cu_q=None, cu_k=None, o=None, lse=None, ws=None, wb=0) == OK
    assert fwd(problem(), rq=0, q=None, o=None, lse=None, ws=None, wb=0) == OK


def test_rest_wants_the_pair_kernel():
    p = problem(heads_q=256, heads_kv=1, rel=api.RelBuckets(32))
    assert fwd(p, bias=A, rest=A) == UNSUP


def test_table_gradient_wants_the_rest():
    """More heads a kv-head than the pair kernel packs: no forward leaves what dbias needs in bf16."""
    rel = api.RelBuckets(32)
    assert bwd(problem(heads_q=256, heads_kv=1, rel=rel), bias=A, dbias=A, wb=16) == UNSUP
    assert bwd(problem(heads_q=128, heads_kv=1, rel=rel), bias=A, dbias=A, wb=16) == WORK
    assert bwd(problem(heads_q=256, heads_kv=1, rel=rel, dtype=torch.float32), bias=A, dbias=A, wb=16) == WORK
    assert bwd(problem(heads_q=256, heads_kv=1), wb=16) == WORK


def test_python_refusals():
    p = problem()
    q, k = torch.zeros((4, 8, 128), dtype=torch.bfloat16), torch.zeros((6, 2, 128), dtype=torch.bfloat16)
    cu = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError):
        api.cross_attn_fwd(p, q, k, k, cu, cu)                              # not on a CUDA device
    for bad in (dict(q=q[:, :7]), dict(q=q.float()), dict(k=k[:, :1]), dict(v=k[:5]), dict(cu_q=cu[:2]), dict(cu_q=cu.long()),
                dict(bias=torch.zeros(32, 8)), dict(len_k=cu), dict(q=q.transpose(0, 1))):
        a = dict(q=q, k=k, v=k, cu_q=cu, cu_k=cu)
        a.update(bad)
        with pytest.raises(ValueError):
            api.cross_attn_fwd(p, **a)
    with pytest.raises(ValueError):
        api.cross_attn_fwd(problem(rel=api.RelBuckets(32)), q, k, k, cu, cu)
    with pytest.raises(ValueError):
        api.cross_attn_fwd(problem(dropout=0.5), q, k, k, cu, cu, rng=torch.zeros(2))


# ------------------------------------------------------------------ oracle ---
def test_generator_against_its_published_vectors():
    """Known answers of Philox4x32 (the paper's test vectors): 7 and 10 rounds."""
    ones = 0xFFFFFFFF
    for rounds, ctr, key, want in (
            (7, (0, 0, 0, 0), (0, 0), (0x5F6FB709, 0x0D893F64, 0x4F121F81, 0x4F730A48)),
            (10, (0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
            (10, (ones,) * 4, (ones,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD))):
        assert tuple(int(x) for x in X.philox(ctr, key, rounds)) == want


def test_kept_share():
    for p in (0.0, 0.1, 0.5, 0.9):
        kept, pe = X.keep(64, 1000, 3, p, 17, 5)
        assert abs(pe - p) <= 2.0 ** -16
        assert abs(kept.mean() - (1 - pe)) <= 5 * np.sqrt(pe * (1 - pe) / kept.size)


@pytest.mark.parametrize("n,distance,both", [(32, 128, True), (32, 128, False), (8, 20, True), (5, 9, False), (2, 1, False)])
def test_buckets(n, distance, both):
    """Every bucket's distances in order; distances below the half have one each; the last one from the distance on."""
    rel = np.arange(-300, 301)
    b = X.buckets(rel, n, distance, both)
    assert b.min() >= 0 and b.max() <= n - 1
    per = n // 2 if both else n
    back = b[rel <= 0][::-1]
    assert np.all(np.diff(back) >= 0) and list(back[:per // 2]) == list(range(per // 2)) and back[distance] == per - 1
    fore = b[rel > 0]
    assert np.array_equal(fore, back[1:] + per) if both else not fore.any()
    # the border of 8 16 32 64 for 16 buckets to 128: powers of two begin a bucket
    if (n, distance, both) == (32, 128, True):
        assert [int(back[x] - back[x - 1]) for x in (8, 16, 32, 64)] == [1, 1, 1, 1]


def test_gradients_against_differences():
    rng = np.random.default_rng(3)
    q, k, v, do = (rng.standard_normal(s) for s in ((7, 4, 8), (9, 2, 8), (9, 2, 8), (7, 4, 8)))
    table = rng.standard_normal((8, 4))
    seqs = [(0, 3, 0, 4), (3, 4, 4, 5)]
    kw = dict(seqs=seqs, causal=True, rel=(8, 4, True), p=0.3, rng=(12345678901234, 9))
    g = X.attention(q, k, v, do=do, table=table, **kw)
    for name, x in (("dq", q), ("dk", k), ("dv", v), ("dtable", table)):
        step = rng.standard_normal(x.shape)
        ends = []
        for h in (1e-5, -1e-5):
            a = dict(q=q, k=k, v=v, table=table)
            a[{"dq": "q", "dk": "k", "dv": "v", "dtable": "table"}[name]] = x + h * step
            ends.append((X.attention(**a, **kw)["o"] * do).sum())
        assert abs((ends[0] - ends[1]) / 2e-5 - (g[name] * step).sum()) <= 1e-6 * np.abs(g[name] * step).sum(), name
