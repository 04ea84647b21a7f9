"""Cross attention on the GPU against its float64 oracle: forward and backward,
bias of the relative position, dropout, and runs of them together.

Tolerances (u32 = 2^-24, u16 = 2^-8: half a step of float32 and bfloat16, relative to
the value), element by element, times the sums of magnitudes that the oracle gives:
* a score: a sum of d products, off by at most 6 sqrt(d) u32 |q| |k| scale (six standard
  deviations of independent roundings), its bias, the exponent and the row's LSE by 8 u32
  of the largest score; P is off by twice all that (its row's sum too): e;
* a sum of n products in float32: 6 sqrt(n) u32 more: f = 2 e + 6 sqrt(n) u32;
* bfloat16: P is rounded before its second product (u16); D's O is rounded (u16) and so
  is dS (2 u16 in all); the outputs are rounded (u16 of the value).  The table's gradient
  takes P and dS in float32 and D to 2^-16.
In the mean the roundings are independent: the 2-norm is held to 2 u16 (the two of dQ and
dK are sqrt(2) u16 / sqrt(3), and the output's u16 / sqrt(3)).
"""

import numpy as np
import pytest
import torch

from oracle import cross as X
from tile_attention_lse_gb300 import api

from helpers import f64

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U32, U16 = 2.0 ** -24, 2.0 ** -8
BF, F32 = torch.bfloat16, torch.float32


def i32(x):
    return torch.tensor(np.asarray(x, dtype=np.int32), device=DEV)


@pytest.fixture(autouse=True)
def no_device_error():
    yield
    assert api.device_error() == 0


class Case:
    """Inputs of a call: sequences (nq, nk), places of the keys (pad: rows behind each sequence)."""

    def __init__(self, seqs, H=4, Hkv=2, d=128, dtype=BF, causal=False, rel=None, p=0.0, fused=False, pad=0, pad_q=0, tail=0,
                 seed=0, max_q=None, junk=1.0,
                 scale=0.0):
        g = torch.Generator().manual_seed(seed)
        nq, nk = [s[0] for s in seqs], [s[1] for s in seqs]
        pq, pk = [n + pad_q for n in nq], [n + pad for n in nk]
        self.cu_q, self.cu_k = np.concatenate([[0], np.cumsum(pq)]), np.concatenate([[0], np.cumsum(pk)])
        self.seqs = [(int(self.cu_q[i]), nq[i], int(self.cu_k[i]), nk[i]) for i in range(len(seqs))]
        rq, rk = int(self.cu_q[-1]) + tail, int(self.cu_k[-1]) + tail

        def rand(*shape):
            return torch.randn(shape, generator=g).to(dtype).to(DEV)

        def fill(x, at):
            """Rows that no sequence owns hold `junk`."""
            own = torch.zeros(x.shape[0], dtype=torch.bool)
            for lo, n in at:
                own[lo:lo + n] = True
            x[~own.to(DEV)] = junk
            return x
        at_q, at_k = [s[:2] for s in self.seqs], [s[2:] for s in self.seqs]
        self.q, self.do = fill(rand(rq, H, d), at_q), fill(rand(rq, H, d), at_q)
        if fused:
            kv = fill(rand(rk, 2, Hkv, d), at_k)
            self.k, self.v = kv[:, 0], kv[:, 1]
        else:
            self.k, self.v = fill(rand(rk, Hkv, d), at_k), fill(rand(rk, Hkv, d), at_k)
        self.rel = rel
        self.table = rand(rel.buckets, H) if rel is not None else None
        self.seed, self.offset = 0x123456789ABCDEF0 + seed, 41 + seed
        self.rng = torch.tensor([self.seed, self.offset], dtype=torch.int64, device=DEV) if p > 0 else None
        self.p, self.causal, self.dtype, self.d = p, causal, dtype, d
        self.problem = api.CrossProblem(H, Hkv, d, dtype=dtype, causal=causal, rel=rel, dropout=p,
                                        max_q=max(nq, default=0) if max_q is None else max_q, softmax_scale=scale)
        self.scale = scale or d ** -0.5
        self.at = dict(len_q=i32(nq) if pad_q else None, len_k=i32(nk) if pad else None, bias=self.table, rng=self.rng)
        self.dcu = (i32(self.cu_q), i32(self.cu_k))

    def forward(self, **kw):
        return api.cross_attn_fwd(self.problem, self.q, self.k, self.v, *self.dcu, for_backward=True, **self.at, **kw)

    def backward(self, o, lse, rest, **kw):
        return api.cross_attn_bwd(self.problem, self.q, self.k, self.v, o, lse, self.do, *self.dcu, rest=rest, **self.at, **kw)

    def oracle(self, grads=True):
        rel = None if self.rel is None else (self.rel.buckets, self.rel.max_distance, self.rel.both)
        return X.attention(f64(self.q), f64(self.k), f64(self.v), self.seqs, do=f64(self.do) if grads else None,
                           causal=self.causal, table=None if self.table is None else f64(self.table), rel=rel, p=self.p,
                           rng=(self.seed, self.offset), scale=self.scale)

    def owned(self, keys):
        n = (self.k if keys else self.q).shape[0]
        own = np.zeros(n, dtype=bool)
        for s in self.seqs:
            lo, m = s[2:] if keys else s[:2]
            own[lo:lo + m] = True
        return own

    def rounding(self, want):
        """e and f of the tolerances."""
        own_q, own_k = self.owned(False), self.owned(True)
        lens = [np.sqrt((f64(x)[own] ** 2).sum(-1)).max(initial=0) for x, own in ((self.q, own_q), (self.k, own_k))]
        e = 2 * (6 * np.sqrt(self.d) * U32 * lens[0] * lens[1] * self.scale + 8 * U32 * max(want["top"], 1.0))
        n = max([self.d] + [m for s in self.seqs for m in (s[1], s[3])]) * 8
        return e, 2 * e + 6 * np.sqrt(n) * U32


def near(name, got, want, mag, share, u, norm=None):
    bad = np.abs(got - want) - (share * mag + u * np.abs(want) + 1e-30)
    assert not np.isnan(got).any(), name
    worst = np.unravel_index(np.argmax(bad), bad.shape) if bad.size else None
    assert bad.size == 0 or bad[worst] <= 0, (name, worst, got[worst], want[worst], mag[worst], share)
    if norm is not None and np.linalg.norm(want) > 0:
        assert np.linalg.norm(got - want) <= norm * np.linalg.norm(want), (name, np.linalg.norm(got - want) / np.linalg.norm(want))


def check_forward(c, o, lse, rest=None, want=None):
    want = c.oracle(False) if want is None else want
    own = c.owned(False)
    e, f = c.rounding(want)
    bf = c.dtype is BF
    ref, lref = want["o"][own], want["lse"][own]
    got = f64(lse)[own]
    assert np.array_equal(np.isneginf(got), np.isneginf(lref))
    fine = np.isfinite(lref)
    assert np.all(np.abs(got[fine] - lref[fine]) <= e + 4 * U32 * np.abs(lref[fine]))
    # with few rows the 2-norm is that of few numbers
    near("o", f64(o)[own], ref, want["mag_o"][own], f + (U16 if bf else 0), U16 if bf else 2 * U32, 2 * U16 if bf else None)
    if rest is not None:
        full = f64(o)[own] + f64(rest)[own]
        near("o + rest", full, ref, want["mag_o"][own], f + U16, 2 * U16 ** 2)
        assert np.all(np.abs(f64(rest)[own]) <= U16 * np.abs(f64(o)[own]) * (1 + 2 * U16) + 1e-38)
    return want


def check_backward(c, grads, want):
    dq, dk, dv, dtable = grads
    _, f = c.rounding(want)
    bf = c.dtype is BF
    u, norm = (U16, 2 * U16) if bf else (2 * U32, None)
    near("dq", f64(dq), want["dq"], want["mag_dq"], f + (2 * U16 if bf else 0), u, norm)
    near("dk", f64(dk), want["dk"], want["mag_dk"], f + (2 * U16 if bf else 0), u, norm)
    near("dv", f64(dv), want["dv"], want["mag_dv"], f + (U16 if bf else 0), u, norm)
    if dtable is not None:
        near("dtable", f64(dtable), want["dtable"], want["mag_dtable"], f + (U16 ** 2 if bf else 0), u)


def check(c, grads=True):
    o, lse, rest = c.forward()
    want = check_forward(c, o, lse, rest, c.oracle(grads))
    if grads:
        check_backward(c, c.backward(o, lse, rest), want)
    return o, lse


REL = {"none": None, "both": api.RelBuckets(32, 128, True), "back": api.RelBuckets(32, 128, False),
       "short": api.RelBuckets(5, 9, False), "wide": api.RelBuckets(64, 700, True)}
RAGGED = [(3, 5), (0, 7), (130, 257), (1, 1), (64, 0), (0, 0), (129, 128), (200, 90), (17, 300)]


# ----------------------------------------------------------------- forward ---
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("rel", ["none", "back", "both"])
@pytest.mark.parametrize("nq", [1, 3, 6])
def test_few_queries(nq, rel, d):
    """The slice kernel in bf16: up to 16 and up to 32 packed rows."""
    c = Case([(nq, n) for n in (777, 1, 0, 64, 65, 300, 2049)], H=8, Hkv=2, d=d, rel=REL[rel], causal=rel == "back", max_q=nq)
    p, args = c.problem, (c.q, c.k, c.v, *c.dcu)
    o, lse = api.cross_attn_fwd(p, *args, **c.at)
    check_forward(c, o, lse)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H,Hkv", [(4, 4), (8, 2), (7, 1)])
def test_many_queries_over_other_lengths(H, Hkv, d):
    check(Case(RAGGED, H=H, Hkv=Hkv, d=d))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("nq,nk", [(1, 1), (127, 128), (128, 127), (129, 129), (256, 1), (1, 256), (300, 513)])
def test_one_sequence(nq, nk, dtype):
    check(Case([(nq, nk)], H=2, Hkv=1, d=64, dtype=dtype, causal=nq % 2 == 1))


def test_wide_groups():
    """More heads a kv-head than a tile of the pair kernel has rows: slices; the most that it has: pairs."""
    c = Case([(5, 300), (2, 7)], H=160, Hkv=1, d=64)
    o, lse, _ = c.forward()
    check_forward(c, o, lse)
    check(Case([(5, 300), (2, 7)], H=160, Hkv=1, d=64, causal=True, rel=REL["both"], dtype=F32))
    wide = Case([(5, 300), (2, 7)], H=160, Hkv=1, d=64, causal=True, rel=REL["both"])
    assert wide.forward()[2] is None       # the slices do not write it
    check(Case([(5, 300), (2, 7)], H=128, Hkv=1, d=64, causal=True))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("max_q", [0, 1, 5])
def test_the_hint_does_not_change_results(max_q, dtype):
    """max_q says less, or nothing, about the queries: every kernel computes any number."""
    c = Case(RAGGED, H=4, Hkv=2, d=64, dtype=dtype, rel=REL["both"], max_q=max_q)
    o, lse = api.cross_attn_fwd(c.problem, c.q, c.k, c.v, *c.dcu, **c.at)
    check_forward(c, o, lse)


def test_rows_that_see_few_keys():
    """A causal row's first keys: dP - D nearly cancels, and the rest keeps it (dS of a row with one key is 0)."""
    c = Case([(64, 64)], H=4, Hkv=4, d=128, causal=True)
    o, lse, rest = c.forward()
    with_rest, without = c.backward(o, lse, rest), c.backward(o, lse, None)
    assert float(with_rest[0][0].float().abs().max()) <= float(without[0][0].float().abs().max())
    # D to 2^-17, scores and P to f of |dO| |v|
    want = c.oracle()
    _, f = c.rounding(want)
    assert np.all(np.abs(f64(with_rest[0][0])) <= (f + 2 * U16 ** 2) * want["mag_dq"][0] + 1e-30)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("nk", [2, 3, 4])
def test_every_row_over_few_keys(nk, d):
    """Without a causal mask or a bias too: scores without a scale lie on one key nearly, where dP - D cancels."""
    check(Case([(9, nk)] * 40, H=8, Hkv=2, d=d, p=0.1, scale=1.0))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H,Hkv,nq", [(8, 2, 1), (8, 2, 4), (8, 2, 7), (16, 16, 2), (160, 1, 2)])
def test_rest_of_few_rows(H, Hkv, nq, d):
    """The slices leave rest too: whole tiles, cut ones (joined by the merge), rows of padding and more heads than a tile has."""
    c = Case([(nq, n) for n in (2, 777, 1, 0, 64, 3, 9000)], H=H, Hkv=Hkv, d=d, max_q=nq, scale=1.0, pad_q=1, tail=2)
    o, lse, rest = c.forward()
    assert rest is not None
    want = check_forward(c, o, lse, rest, c.oracle())
    check_backward(c, c.backward(o, lse, rest), want)
    own = torch.from_numpy(c.owned(False)).to(DEV)
    plain = api.cross_attn_fwd(c.problem, c.q, c.k, c.v, *c.dcu, **c.at)
    assert torch.equal(o[own], plain[0][own]) and torch.equal(lse[own], plain[1][own])


def test_table_gradient_without_the_rest():
    """Without what o lost to its rounding, D is off by u16 of the sum of |dO| |o|."""
    c = Case(RAGGED, rel=REL["both"], d=64)
    o, lse, _ = c.forward()
    want = c.oracle()
    _, f = c.rounding(want)
    got = c.backward(o, lse, None)
    near("dtable", f64(got[3]), want["dtable"], want["mag_dtable"], f + U16, U16)
    near("dq", f64(got[0]), want["dq"], want["mag_dq"], f + 2 * U16, U16, 2 * U16)


# ---------------------------------------------------- everything, each type ---
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("rel", list(REL))
@pytest.mark.parametrize("p", [0.0, 0.3])
@pytest.mark.parametrize("causal", [False, True])
def test_forward_and_backward(causal, p, rel, d, dtype):
    check(Case(RAGGED, d=d, dtype=dtype, causal=causal, rel=REL[rel], p=p, seed=3))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_scale_of_the_scores(dtype):
    """Scores without a scale: the largest weights of a row are nearly 1."""
    check(Case([(140, 200), (3, 150)], d=64, dtype=dtype, rel=REL["both"], p=0.1, scale=1.0))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_no_sequence_has_work(dtype):
    c = Case([(0, 0), (0, 5), (7, 0), (0, 140)], dtype=dtype, rel=REL["both"], p=0.1, tail=3, max_q=0)
    o, lse, rest = c.forward()
    own = torch.from_numpy(c.owned(False)).to(DEV)
    assert bool((o[own] == 0).all()) and bool(torch.isneginf(lse[own]).all())
    assert all(bool((g == 0).all()) for g in c.backward(o, lse, rest))
    few = Case([(0, 0), (0, 5), (2, 0)], dtype=dtype, rel=REL["both"], tail=3, max_q=2)
    o, lse = api.cross_attn_fwd(few.problem, few.q, few.k, few.v, *few.dcu, **few.at)
    assert bool((o[few.owned(False)] == 0).all())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("p", [0.0, 0.1])
def test_longer_self_attention(p, dtype):
    """Tiles on both sides of the bias's reach, several heads a group, several tiles each way."""
    check(Case([(700, 700), (300, 300)], H=4, Hkv=2, d=64, dtype=dtype, rel=REL["both"], p=p))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_few_queries_over_a_long_context(dtype):
    """What cut tiles leave is joined; the gradient of a table whose far bucket holds nearly all keys."""
    check(Case([(2, 6000), (3, 4001)], H=8, Hkv=4, d=64, dtype=dtype, rel=api.RelBuckets(16, 600, False), causal=True, p=0.1))


# buckets, their distance, directions; a row's keys outside the bucket that holds most of them
LONG = [(4, 16, False, 6), (16, 100, False, 73), (8, 40, True, 9), (32, 128, True, 91), (2, 1, False, 1)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("p", [0.0, 0.1])
@pytest.mark.parametrize("buckets,distance,both,w", LONG)
def test_table_gradient_where_one_bucket_holds_nearly_all_keys(buckets, distance, both, w, p, dtype):
    """A row's dS sums to 0, and the far bucket keeps what D = dO . o is off by: sqrt(n / w) of the gradient times that.

    float32: P is off by about 4 u32 (a score of d = 64 products 3, the exponent 2), in the forward's o and, by
    other sums, in the backward's: D by 6 u32, 2^-21.4; five deviations: 2^-19.  bf16: P, and o with rest, are kept in two
    parts of 8 bits, each off by u16^2 of the value at most: together 2^-15, half of which is more than their mean; and the
    rounding of the gradient itself, u16 at most."""
    rel, n = api.RelBuckets(buckets, distance, both), 30000
    c = Case([(8, n), (3, n // 2)], H=4, Hkv=2, d=64, dtype=dtype, rel=rel, p=p, causal=not both, seed=5)
    o, lse, rest = c.forward()
    want = check_forward(c, o, lse, rest, c.oracle())
    grads = c.backward(o, lse, rest)
    check_backward(c, grads, want)
    share = 2 ** -16 if dtype is BF else 2 ** -19
    far = np.linalg.norm(f64(grads[3]) - want["dtable"]) / np.linalg.norm(want["dtable"])
    assert far <= share * np.sqrt(n / w) + (U16 if dtype is BF else U32), far


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("p", [0.0, 0.3])
@pytest.mark.parametrize("rel", ["back", "both", "short"])
@pytest.mark.parametrize("seqs", [RAGGED, [(3, 9000), (1, 4000)], [(600, 700)]])
def test_output_and_rest_under_a_bias(seqs, rel, p, d):
    """P in two parts of 8 bits (u16^2 of P lost) and rest (u16^2 of o): whole tiles, cut ones, tiles far from the diagonal."""
    c = Case(seqs, H=4, Hkv=2, d=d, rel=REL[rel], p=p, causal=rel == "back", seed=6)
    o, lse, rest = c.forward()
    want = check_forward(c, o, lse, rest)
    own, (_, f) = c.owned(False), c.rounding(want)
    full = f64(o)[own] + f64(rest)[own]
    near("o + rest", full, want["o"][own], want["mag_o"][own], f + U16 ** 2, U16 ** 2, U16 ** 2)
    o, lse = api.cross_attn_fwd(c.problem, c.q, c.k, c.v, *c.dcu, **c.at)  # the copies without rest
    check_forward(c, o, lse, None, want)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("nq,nk", [(2, 60000), (20000, 70)])
def test_long_sums_in_float32(nq, nk, d):
    """dQ over many keys, dK and dV over many queries: tiles of 64 are summed apart, then n / 64 of them.

    A chain of t sums of mixed sign is off by sqrt(t / 2) roundings of 0.42 u32 (a half step's root mean square) of its end:
    9 u32 for 940 tiles; P and dS by 6 u32 in the mean (scores 3, exponents 2, D): 11 u32 together, doubled."""
    c = Case([(nq, nk)], H=2, Hkv=1, d=d, dtype=F32)
    o, lse, rest = c.forward()
    want = c.oracle()
    for got, name in zip(c.backward(o, lse, rest), ("dq", "dk", "dv")):
        assert np.linalg.norm(f64(got) - want[name]) <= 22 * U32 * np.linalg.norm(want[name]), name


def test_fused_and_padded_inputs():
    for dtype in (BF, F32):
        check(Case(RAGGED, dtype=dtype, fused=True, pad=37, pad_q=11, tail=5, rel=REL["both"], p=0.2))


# --------------------------------------------------- what is not to be seen ---
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("p,rel", [(0.0, "none"), (0.2, "both")])
@pytest.mark.parametrize("nq", [2, 150])
def test_rows_that_no_sequence_owns(nq, p, rel, dtype):
    """NaN there reaches nothing; outputs there stay, gradients are zeros."""
    c = Case([(nq, 130), (nq + 1, 60), (0, 3), (nq, 0), (nq - 1, 129)], dtype=dtype, pad=9, pad_q=7, tail=140, junk=float("nan"),
             p=p, rel=REL[rel])
    o, lse = torch.full_like(c.q, 7.0), torch.full(c.q.shape[:2], 7.0, device=DEV)
    _, _, rest = c.forward(out=o, lse=lse)
    own = torch.from_numpy(c.owned(False)).to(DEV)
    assert bool((o[~own] == 7).all()) and bool((lse[~own] == 7).all())
    seen = Case([s[1::2] for s in c.seqs], dtype=dtype, pad=9, pad_q=7, tail=140, junk=0.0, p=p, rel=REL[rel])
    want = seen.oracle()
    check_forward(seen, o, lse, None, want)
    grads = c.backward(o, lse, rest)
    check_backward(seen, grads, want)
    assert bool((grads[0][~own] == 0).all())
    own_k = torch.from_numpy(c.owned(True)).to(DEV)
    assert bool((grads[1][~own_k] == 0).all()) and bool((grads[2][~own_k] == 0).all())


@pytest.mark.parametrize("dtype", [BF, F32])
def test_one_sequence_that_is_not_finite(dtype):
    """Infinities and NaN of one sequence reach no other, forward or backward."""
    c = Case([(70, 100), (90, 77), (130, 140)], dtype=dtype, rel=REL["both"], p=0.1)
    clean = c.oracle()
    _, f = c.rounding(clean)
    q0, nq, k0, nk = c.seqs[1]
    for x, row, bad in ((c.k, k0 + 70, float("nan")), (c.v, k0 + 3, float("inf")), (c.q, q0 + 88, float("-inf")),
                        (c.do, q0 + 1, float("nan"))):
        x[row] = bad
    o, lse, rest = c.forward()
    dq, dk, dv, _ = c.backward(o, lse, rest)
    share = f + (2 * U16 if dtype is BF else 0)
    for i in (0, 2):
        a, n, b, m = c.seqs[i]
        for got, name, at in ((o, "o", slice(a, a + n)), (dq, "dq", slice(a, a + n)), (dk, "dk", slice(b, b + m)),
                              (dv, "dv", slice(b, b + m))):
            near(name, f64(got)[at], clean[name][at], clean["mag_" + name][at], share, U16)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("value", [float("-inf"), "lowest"])
def test_table_entries_that_mask(value, dtype):
    """-inf or the type's lowest number in the table: never; a head of only such sees nothing."""
    c = Case([(70, 200), (3, 40), (150, 150)], dtype=dtype, rel=REL["both"])
    low = torch.finfo(dtype).min if value == "lowest" else value
    c.table[3:9] = low       # near ones
    c.table[15, 1] = low     # a far one
    c.table[:, 2] = low      # a head that sees nothing
    o, lse = check(c)
    assert bool(torch.isneginf(lse[:, 2]).all()) and bool((o[:, 2] == 0).all())


# ----------------------------------------------------------------- dropout ---
def test_dropped_share_and_seeds():
    """V of ones gives the kept share of P; other seeds, offsets, heads and rows give other masks."""
    c = Case([(400, 1000)], H=2, Hkv=2, d=64, p=0.25)
    c.v.fill_(1.0)
    o, _, _ = c.forward()
    mean = float(o.float().mean())
    assert abs(mean - 1.0) < 0.01          # 800 rows of about 1000 keys: a deviation of 0.0007
    rows = o[:, :, 0].float()
    # a row's deviation is sqrt(1 / 3 sum P^2) = 0.03; six of them hold 0.18 / 2^-7 .. 2^-8 = 23 to 46 bf16 values
    assert rows.unique().numel() > 20 and not torch.equal(rows[:, 0], rows[:, 1])
    c.rng[1] += 1
    assert not torch.equal(o, c.forward()[0])
    c.rng[1] -= 1
    c.rng[0] += 2 ** 40
    assert not torch.equal(o, c.forward()[0])
    c.rng[0] -= 2 ** 40
    assert torch.equal(o, c.forward()[0])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("k", [3276, 9831])
@pytest.mark.parametrize("side", [-1, 0, 1])
def test_dropout_next_to_a_border(side, k, dtype):
    """p at (k + 1/2) / 2^15 and the doubles beside it: which pairs are kept, counted row by row."""
    p = np.nextafter((k + 0.5) / 32768, (0, 1)[side > 0]) if side else (k + 0.5) / 32768
    c = Case([(1500, 64)], H=16, Hkv=16, d=64, dtype=dtype, p=p)  # 1.5 million pairs: 47 for each threshold
    c.q.zero_()
    c.v.fill_(1.0)                                                # o: the kept of 64 keys / (64 (1 - p))
    counts = np.stack([X.keep(1500, 64, h, p, c.seed, c.offset)[0].sum(1) for h in range(16)], 1)
    pe = round(p * 32768) / 32768
    rows = lambda o: np.rint(f64(o[:, :, 0]) * 64 * (1 - pe))     # noqa: E731  (a step of 64 is 4 u16 and more)
    assert np.array_equal(rows(c.forward()[0]), counts)
    c.problem._desc.dropout = (k + 0.5) / 32768                   # a float's half, past the binding
    cut = round(k + 0.5)
    counts = np.stack([X.keep(1500, 64, h, cut / 32768, c.seed, c.offset)[0].sum(1) for h in range(16)], 1)
    assert np.array_equal(rows(c.forward()[0]), counts)


def test_dropout_of_nearly_nothing_and_nearly_all():
    for p in (1e-6, 0.999):
        for dtype in (BF, F32):
            check(Case([(130, 300), (2, 3)], dtype=dtype, p=p))


# ----------------------------------------------------------------- streams ---
def test_same_call_same_bits():
    c = Case([(300, 700), (129, 64)], rel=REL["both"], p=0.1, d=64)
    first = c.forward()
    grads = c.backward(*first)
    for _ in range(3):
        again = c.forward()
        assert all(torch.equal(x, y) for x, y in zip(first, again))
        for x, y in zip(grads[1:], c.backward(*again)[1:]):
            assert torch.equal(x, y)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_captured_and_replayed_on_new_values(dtype):
    """One graph of a forward and a backward, replayed on other lengths, biases, numbers and inputs."""
    c = Case([(200, 300), (100, 77)], dtype=dtype, rel=REL["both"], p=0.2, pad=8, pad_q=8)
    n = len(c.seqs)
    ws = api.cross_workspace(c.problem, n, c.q.shape[0], c.k.shape[0], True)
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        out = c.forward(ws=ws)
        c.backward(*out, ws=ws)
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            out = c.forward(ws=ws)
            grads = c.backward(*out, ws=ws)
    other = Case([(150, 308), (108, 20)], dtype=dtype, rel=REL["both"], p=0.2, seed=9)
    for old, new in ((c.at["len_q"], [150, 108]), (c.at["len_k"], [308, 20])):
        old.copy_(i32(new))
    c.seqs = [(s[0], a, s[2], b) for s, (a, b) in zip(c.seqs, [(150, 308), (108, 20)])]
    c.table.copy_(other.table)
    c.seed, c.offset = other.seed, other.offset
    c.rng.copy_(other.rng)
    c.q.normal_()
    c.do.normal_()
    graph.replay()
    torch.cuda.synchronize()
    want = check_forward(c, *out, c.oracle())
    check_backward(c, grads, want)


def test_two_streams_at_once():
    cs = [Case([(300, 700), (129, 64)], rel=REL["both"], p=0.1, d=64, seed=s) for s in (1, 2)]
    want = [c.forward() for c in cs]
    grads = [c.backward(*w) for c, w in zip(cs, want)]
    streams = [torch.cuda.Stream() for _ in cs]
    ws = [api.cross_workspace(c.problem, 2, c.q.shape[0], c.k.shape[0], True) for c in cs]
    torch.cuda.synchronize()
    got = [None, None]
    for _ in range(3):
        for i, c in enumerate(cs):
            with torch.cuda.stream(streams[i]):
                o = c.forward(ws=ws[i])
                got[i] = (o, c.backward(*o, ws=ws[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(x, y) for x, y in zip(got[i][0], want[i]))
        assert all(torch.equal(x, y) for x, y in zip(got[i][1][1:], grads[i][1:]))


# ------------------------------------------------------------------ sizes ---
def test_calls_without_rows():
    p = api.CrossProblem(4, 2, 64, rel=REL["both"])
    table = torch.ones((32, 4), dtype=BF, device=DEV)
    for rq, rk, n in ((0, 10, 1), (10, 0, 1), (0, 0, 1), (5, 5, 0), (0, 0, 0)):
        q, k = torch.ones((rq, 4, 64), dtype=BF, device=DEV), torch.ones((rk, 2, 64), dtype=BF, device=DEV)
        cu_q, cu_k = i32([0] + [rq] * n), i32([0] + [rk] * n)
        o, lse, rest = api.cross_attn_fwd(p, q, k, k, cu_q, cu_k, bias=table, for_backward=True)
        if n and rq:
            assert bool((o == 0).all()) and bool(torch.isneginf(lse).all())
        else:
            o, lse, rest = torch.zeros_like(o), torch.zeros_like(lse), torch.zeros_like(o)
        g = api.cross_attn_bwd(p, q, k, k, o, lse, q, cu_q, cu_k, bias=table, rest=rest)
        assert all(bool((x == 0).all()) for x in g)


def test_lengths_that_leave_the_tensors():
    """What cu_q, cu_k and the lengths say beyond the rows is left out."""
    c = Case([(60, 100), (70, 90)], d=64, rel=REL["back"], causal=True)
    want = c.oracle()
    c.dcu = (i32([0, 60, 1000]), i32([0, 100, 2 ** 31 - 1]))
    c.at.update(len_q=i32([900, 900]), len_k=i32([2 ** 30, 2 ** 31 - 1]))
    o, lse, rest = c.forward()
    check_forward(c, o, lse, rest, want)
    check_backward(c, c.backward(o, lse, rest), want)
    c.at.update(len_q=i32([-5, 70]), len_k=i32([100, -1]))
    c.seqs = [(0, 0, 0, 100), (60, 70, 100, 0)]
    o, lse, rest = c.forward()
    want = check_forward(c, o, lse, rest, c.oracle())
    check_backward(c, c.backward(o, lse, rest), want)


def test_many_sequences():
    rng = np.random.default_rng(5)
    seqs = [(int(a), int(b)) for a, b in zip(rng.integers(0, 6, 700), rng.integers(0, 9, 700))]
    for dtype in (BF, F32):
        check(Case(seqs, H=2, Hkv=2, d=64, dtype=dtype, causal=True, p=0.1, rel=REL["short"]))


def test_offsets_beyond_32_bits():
    """Rows whose elements lie beyond 2^32: the last sequence of a tensor of that size."""
    rows, H, d = 2 ** 32 // (8 * 128) + 300, 8, 128
    big = torch.zeros((rows, H, d), dtype=BF, device=DEV)
    small = Case([(200, 250)], H=H, Hkv=H, d=d)
    big[rows - 250:] = small.k
    cu_k, cu_q = i32([0, rows - 250, rows]), i32([0, 0, 200])
    o, lse = api.cross_attn_fwd(small.problem, small.q, big, big, cu_q, cu_k)
    w, wl = api.cross_attn_fwd(small.problem, small.q, small.k, small.k, *small.dcu)
    check_forward(Case([(200, 250)], H=H, Hkv=H, d=d), o, lse, None, X.attention(f64(small.q), f64(small.k), f64(small.k), small.seqs))
    assert torch.allclose(lse, wl, atol=1e-5)


# ----------------------------------------------------------- differences ---
def test_gradients_against_differences():
    """float32: the loss along a random step of each input, by the kernel's own forward."""
    c = Case([(40, 70), (33, 20)], H=4, Hkv=2, d=64, dtype=F32, rel=REL["both"], p=0.2)
    o, lse, rest = c.forward()
    grads = c.backward(o, lse, rest)
    for x, g in zip((c.q, c.k, c.v, c.table), grads):
        gen = torch.Generator(device=DEV).manual_seed(1)
        step = torch.randn(x.shape, generator=gen, device=DEV)
        keep, h, ends = x.clone(), 1e-2, []
        for sign in (1, -1):
            x.copy_(keep + sign * h * step)
            ends.append(float((c.forward()[0].double() * c.do.double()).sum()))
        x.copy_(keep)
        diff, want = (ends[0] - ends[1]) / (2 * h), float((g.double() * step.double()).sum())
        # the loss's third derivative along the step times h^2 / 6, and its rounding / h
        scale = float((g.double() * step.double()).norm())
        assert abs(diff - want) <= 0.02 * scale + 1e-3, (diff, want, scale)


# ---------------------------------------------------------------- together ---
def test_encoder_and_decoder_together():
    """An encoder layer's attention, a decoder's causal one and the attention between them,
    forward and backward, as a training step chains them (float32, against the oracle's chain)."""
    H, d = 4, 64
    src, tgt = [70, 130, 9], [33, 64, 12]
    enc = Case([(n, n) for n in src], H=H, Hkv=H, d=d, dtype=F32, rel=REL["both"], p=0.1, seed=1)
    dec = Case([(n, n) for n in tgt], H=H, Hkv=H, d=d, dtype=F32, rel=REL["back"], causal=True, p=0.1, seed=2)
    mid = Case(list(zip(tgt, src)), H=H, Hkv=H, d=d, dtype=F32, p=0.1, seed=3)
    e, d_ = enc.forward(), dec.forward()
    mid.q, mid.k = d_[0], e[0]            # queries from the decoder, keys from the encoder
    m = mid.forward()
    dq, dk, dv, _ = mid.backward(*m)
    enc.do, dec.do = dk, dq
    ge, gd = enc.backward(*e), dec.backward(*d_)
    # the same in float64
    we, wd = enc.oracle(False), dec.oracle(False)

    def chain(q, k, v, do, c, table=None):
        rel = None if c.rel is None else (c.rel.buckets, c.rel.max_distance, c.rel.both)
        return X.attention(q, k, v, c.seqs, do=do, causal=c.causal, table=table, rel=rel, p=c.p, rng=(c.seed, c.offset))
    wm = chain(wd["o"], we["o"], f64(mid.v), f64(mid.do), mid)
    wge = chain(f64(enc.q), f64(enc.k), f64(enc.v), wm["dk"], enc, f64(enc.table))
    wgd = chain(f64(dec.q), f64(dec.k), f64(dec.v), wm["dq"], dec, f64(dec.table))
    for got, want in ((m[0], wm["o"]), (dv, wm["dv"]), *zip(ge, (wge[x] for x in ("dq", "dk", "dv", "dtable"))),
                      *zip(gd, (wgd[x] for x in ("dq", "dk", "dv", "dtable")))):
        # three calls of about f each, on magnitudes a few times the values
        assert np.linalg.norm(f64(got) - want) <= 1e-4 * np.linalg.norm(want)


def test_token_by_token_equals_the_whole_pass():
    """A decoder answering: each new token over its own growing keys and over its source, against the
    pass over all tokens at once."""
    H, d, n, rel = 4, 64, 40, REL["back"]
    whole = Case([(n, n)], H=H, Hkv=2, d=d, rel=rel, causal=True)
    ws = api.cross_workspace(whole.problem, 1, n, n, True)
    want = check_forward(whole, *whole.forward())
    one = api.CrossProblem(H, 2, d, causal=True, rel=rel, max_q=1)
    rows = []
    for t in range(n):
        o, lse = api.cross_attn_fwd(one, whole.q[t:t + 1], whole.k, whole.v, i32([0, 1]), i32([0, n]), len_k=i32([t + 1]),
                                    bias=whole.table, ws=ws)
        rows.append((o, lse))
    check_forward(whole, torch.cat([r[0] for r in rows]), torch.cat([r[1] for r in rows]), None, want)


def test_states_merge_with_other_partial_states():
    """Two halves of a source, attended apart, merge to the whole (cp_merge_partials)."""
    c = Case([(100, 300)], dtype=F32, H=4, Hkv=2)
    parts = [api.cross_attn_fwd(c.problem, c.q, c.k[lo:hi], c.v[lo:hi], i32([0, 100]), i32([0, hi - lo]))
             for lo, hi in ((0, 130), (130, 300))]
    o, lse = api.merge_partials(torch.stack([p[0] for p in parts]), torch.stack([p[1] for p in parts]))
    check_forward(c, o, lse)


def test_counted_launches():
    api.profile_read()
    c = Case([(130, 200)], rel=REL["both"])
    c.backward(*c.forward())
    n = {k: v[1] for k, v in api.profile_read().items()}
    assert (n["cross"], n["cross_merge"], n["cross_prep"], n["cross_bwd"], n["cross_post"]) == (1, 1, 3, 1, 1)
