"""Failure detection on the GPU without a fault: the tcgen05 kernels' bounded
waits.

cp_debug_set_wait_limit shortens the cycle budget of every main-loop wait of
the tensor-core forward and backward.  With a budget of one cycle every wait
that is not already complete runs out: the block raises its abort flag,
drains its own copies and MMAs (with the default budget), frees TMEM and
returns, and the host reads CP_ERR_TIMEOUT.  The context must stay usable: the
next call with the default budget is checked against the float64 oracle.
"""

import numpy as np
import pytest
import torch

from oracle import attention as A
from tile_attention_lse_gb300 import api

from helpers import TOL_F32, TOL_GRAD_REL, TOL_LSE_BF16, TOL_O_BF16, f64, make_inputs, max_abs

pytestmark = pytest.mark.gpu
DEV = "cuda"
CP_ERR_TIMEOUT = -6


def _case():
    b, s, H, d, cp = 1, 2048, 2, 128, 4
    q, k, v, do = make_inputs(b, s, H, H, d, seed=17, dtype=torch.bfloat16, with_do=True)
    p = api.Problem(batch=b, heads_q=H, heads_kv=H, head_dim=d, cp=cp, seqlen=s)
    return p, q, k, v, do


def test_wait_limit_runs_out_then_recovers():
    p, q, k, v, do = _case()
    qd, kd, vd, dod = (x.to(DEV) for x in (q, k, v, do))
    assert api.device_error() == 0
    try:
        api.set_wait_limit(1)
        api.ring_attn_fwd(p, qd, kd, vd)                 # host status: launched
        assert api.device_error() == CP_ERR_TIMEOUT       # a forward wait ran out
        api.set_wait_limit(0)
        o_ok, l_ok = api.ring_attn_fwd(p, qd, kd, vd)    # backward input from a clean forward
        assert api.device_error() == 0
        api.set_wait_limit(1)
        api.ring_attn_bwd(p, qd, kd, vd, o_ok, l_ok, dod)
        assert api.device_error() == CP_ERR_TIMEOUT       # a backward wait ran out
    finally:
        api.set_wait_limit(0)
    # the word was read and cleared; the default budget gives correct results again
    assert api.device_error() == 0
    o, l = api.ring_attn_fwd(p, qd, kd, vd)
    dq, dk, dv = api.ring_attn_bwd(p, qd, kd, vd, o, l, dod)
    assert api.device_error() == 0
    ro, rl = A.attention_forward_bshd(f64(q), f64(k), f64(v))
    assert max_abs(f64(o[0]), ro[0]) <= TOL_O_BF16
    assert max_abs(f64(l[0]), rl[0]) <= TOL_LSE_BF16
    rq, rk, rv = A.attention_backward_bshd(f64(q), f64(k), f64(v), f64(do))
    for got, ref in ((dq, rq), (dk, rk), (dv, rv)):
        assert max_abs(f64(got[0]), ref[0]) <= TOL_GRAD_REL * float(np.max(np.abs(ref)))


def test_wait_limit_argument_checks():
    with pytest.raises(api.CpError) as e:
        api.set_wait_limit(10 ** 12)                     # above the default budget
    assert e.value.code == -1
    api.set_wait_limit(-5)                               # <= 0: the default
    api.set_wait_limit(0)


def test_wait_limit_of_the_paged_kernel():
    b, s, H, d, page = 1, 512, 4, 128, 64
    q, k, v, _ = make_inputs(b, s, H, H, d, seed=18, dtype=torch.bfloat16, with_do=True)
    kv = api.PagedKV(k[0].view(-1, page, H, d).to(DEV), v[0].view(-1, page, H, d).to(DEV))
    table = torch.arange(s // page, dtype=torch.int32, device=DEV)[None]
    cu, lens = (torch.tensor(x, dtype=torch.int32, device=DEV) for x in ([0, s], [s]))
    p = api.PagedProblem(kv, H, max_new=s)
    qd = q[0].to(DEV)
    try:
        api.set_wait_limit(1)
        api.paged_attn_fwd(p, qd, table, cu, lens)
        assert api.device_error() == CP_ERR_TIMEOUT
    finally:
        api.set_wait_limit(0)
    assert api.device_error() == 0
    o, l = api.paged_attn_fwd(p, qd, table, cu, lens)
    assert api.device_error() == 0
    ro, rl = A.attention_forward_bshd(f64(q), f64(k), f64(v))
    assert max_abs(f64(o), ro[0]) <= TOL_O_BF16
    assert max_abs(f64(l), rl[0]) <= TOL_LSE_BF16


# The kernels of few rows: single tokens, a few, float32 of both, and a call
# with a launch of either kind.  Cut tiles and whole ones, the last stages of
# a block's share partly filled.
PAGED = {
    "bf16_single": (torch.bfloat16, 128, [1] * 5, [3, 700, 64, 1, 9000], 8, 2, 1),
    "bf16_d64_few": (torch.bfloat16, 64, [8, 5, 1], [4000, 77, 300], 8, 2, 8),
    "f32_single": (torch.float32, 64, [1, 1], [1500, 20], 4, 2, 1),
    "f32_chunk": (torch.float32, 128, [40, 7], [900, 7], 4, 2, 40),
    "mixed": (torch.bfloat16, 128, [1, 90, 1, 200], [5000, 900, 64, 3000], 8, 2, 200),
    "bf16_d64_single": (torch.bfloat16, 64, [1, 1], [700, 20], 8, 2, 1),
    "bf16_few": (torch.bfloat16, 128, [8, 3], [900, 40], 8, 2, 8),
    "f32_d128_single": (torch.float32, 128, [1, 1], [700, 20], 4, 2, 1),
    "f32_d64_chunk": (torch.float32, 64, [30, 7], [900, 7], 4, 2, 40),
    "bf16_d64_mixed": (torch.bfloat16, 64, [1, 90], [700, 900], 8, 2, 90),
}


@pytest.mark.parametrize("name", PAGED)
def test_wait_limit_of_every_paged_kernel(name):
    from oracle import paged as P
    dtype, d, new, lens, hq, hkv, max_new = PAGED[name]
    page, g = 32, torch.Generator().manual_seed(19)
    used = -(-np.asarray(lens) // page)
    width, pages = int(used.max()), int(used.sum())
    kv = api.PagedKV(*(torch.randn((pages, page, hkv, d), generator=g).to(DEV, dtype) for _ in range(2)))
    table = np.full((len(lens), width), -1, dtype=np.int32)
    for r, n in enumerate(used):
        table[r, :n] = used[:r].sum() + np.arange(n)
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    q = torch.randn((int(cu[-1]), hq, d), generator=g).to(DEV, dtype)
    p = api.PagedProblem(kv, hq, max_new=max_new)
    args = (p, q, *(torch.from_numpy(np.asarray(x, dtype=np.int32)).to(DEV) for x in (table, cu, lens)))
    before = api.paged_attn_fwd(*args)
    assert api.device_error() == 0
    try:
        api.set_wait_limit(1)
        api.paged_attn_fwd(*args)
        assert api.device_error() == CP_ERR_TIMEOUT
    finally:
        api.set_wait_limit(0)
    assert api.device_error() == 0
    o, l = api.paged_attn_fwd(*args)
    assert api.device_error() == 0
    assert torch.equal(o, before[0]) and torch.equal(l, before[1])
    ro, rl = P.attention(f64(q), f64(kv.k_cache), f64(kv.v_cache), table, cu, lens)
    if dtype == torch.bfloat16:  # the weights' and the output's roundings, half a step (2^-8) each
        vmax = float(kv.v_cache.abs().max())
        assert (np.abs(f64(o) - ro) <= 2.0 ** -8 * (vmax + np.abs(ro)) + 1e-4).all()
        assert max_abs(f64(l), rl) <= TOL_LSE_BF16
    else:
        assert max_abs(f64(o), ro) <= TOL_F32 and max_abs(f64(l), rl) <= TOL_F32
