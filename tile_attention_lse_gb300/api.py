"""ctypes binding of libcpattn.so (argument marshalling only).

Every function here passes device pointers, sizes and the current CUDA stream
of PyTorch to the C ABI declared in ``include/cpattn.h``; all arithmetic runs
in the library's kernels.  PyTorch only provides device memory and streams.
If the library is missing the import of any entry point raises: there is no
fallback.
"""

from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass, field

import numpy as np
import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libcpattn.so")

CP_F32, CP_BF16 = 0, 1
CP_ORDER_ORIGINAL, CP_ORDER_RANK_LOCAL = 0, 1
CP_PARTITION_ZIGZAG, CP_PARTITION_STRIPED = 0, 1
STATUS = {0: "CP_OK", -1: "CP_ERR_INVALID_ARG", -2: "CP_ERR_ALIGNMENT", -3: "CP_ERR_UNSUPPORTED",
          -4: "CP_ERR_WORKSPACE", -5: "CP_ERR_CUDA", -6: "CP_ERR_TIMEOUT"}

# Every symbol the header declares (checked by the CPU test suite).
EXPORTS = ("cp_status_string", "cp_validate_desc", "cp_partition_indices", "cp_permute_tokens",
           "cp_tile_attn_fwd", "cp_merge_partials", "cp_ring_attn_workspace_bytes",
           "cp_ring_attn_fwd", "cp_ring_attn_bwd", "cp_get_device_error", "cp_ring_plan_stats",
           "cp_profile_enable", "cp_profile_read", "cp_ring_attn_fwd_static_ws",
           "cp_static_ws_capacity", "cp_ring_bwd_schedule", "cp_permute_rope", "cp_hybrid_schedule",
           "cp_ring_plan_tables", "cp_token_seq_pos", "cp_debug_set_wait_limit",
           "cp_kv_extend", "cp_kv_release", "cp_rope_axes", "cp_kv_append", "cp_validate_paged_desc",
           "cp_paged_attn_workspace_bytes", "cp_paged_attn_fwd", "cp_paged_schedule",
           "cp_validate_cross_desc", "cp_cross_attn_workspace_bytes", "cp_cross_attn_fwd", "cp_cross_attn_bwd")
KERNEL_CLASSES = ("partition", "permute", "tile_fwd", "merge", "delta", "tile_bwd", "convert", "tables", "rope",
                  "kv_tables", "head_rows", "paged", "paged_merge", "cross", "cross_merge", "cross_prep", "cross_bwd",
                  "cross_post")


class CpError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {STATUS.get(code, code)}")


class CpAttnDesc(ctypes.Structure):
    _fields_ = [
        ("batch", ctypes.c_int32),
        ("heads_q", ctypes.c_int32),
        ("heads_kv", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
        ("cp", ctypes.c_int32),
        ("causal", ctypes.c_int32),
        ("seqlen", ctypes.c_int64),
        ("cu_seqlens_host", ctypes.c_void_p),
        ("cu_seqlens_dev", ctypes.c_void_p),
        ("n_seqs", ctypes.c_int32),
        ("dtype", ctypes.c_int32),
        ("order", ctypes.c_int32),
        ("softmax_scale", ctypes.c_float),
        ("partition", ctypes.c_int32),
        ("window", ctypes.c_int32),
        ("seq_cp_host", ctypes.c_void_p),
        ("seq_rank0_host", ctypes.c_void_p),
        ("seq_cp_dev", ctypes.c_void_p),
        ("seq_rank0_dev", ctypes.c_void_p),
    ]


class CpRope(ctypes.Structure):
    _fields_ = [
        ("n_axes", ctypes.c_int32),
        ("section", ctypes.c_int32 * 4),
        ("interleaved", ctypes.c_int32),
        ("restart", ctypes.c_int32),
        ("adjacent", ctypes.c_int32),
        ("base", ctypes.c_float),
    ]


class CpKvCache(ctypes.Structure):
    _fields_ = [
        ("k", ctypes.c_void_p),
        ("v", ctypes.c_void_p),
        ("n_pages", ctypes.c_int32),
        ("page_size", ctypes.c_int32),
        ("heads_kv", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
        ("page_stride", ctypes.c_int64),
        ("token_stride", ctypes.c_int64),
        ("head_stride", ctypes.c_int64),
        ("dtype", ctypes.c_int32),
    ]


class CpPagedDesc(ctypes.Structure):
    _fields_ = [
        ("kv", CpKvCache),
        ("heads_q", ctypes.c_int32),
        ("max_new", ctypes.c_int32),
        ("causal", ctypes.c_int32),
        ("window", ctypes.c_int32),
        ("softmax_scale", ctypes.c_float),
    ]


class CpCrossDesc(ctypes.Structure):
    _fields_ = [
        ("heads_q", ctypes.c_int32),
        ("heads_kv", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
        ("dtype", ctypes.c_int32),
        ("causal", ctypes.c_int32),
        ("max_q", ctypes.c_int32),
        ("rel_buckets", ctypes.c_int32),
        ("rel_max_distance", ctypes.c_int32),
        ("rel_both", ctypes.c_int32),
        ("dropout", ctypes.c_float),
        ("softmax_scale", ctypes.c_float),
    ]


_lib = None


def lib():
    """Loads the library once; raises if it was not built."""
    global _lib
    if _lib is None:
        if not os.path.exists(_LIB_PATH):
            raise ImportError(f"libcpattn.so not built ({_LIB_PATH}); run "
                              "python -m tile_attention_lse_gb300.build")
        L = ctypes.CDLL(_LIB_PATH)
        P, I32, I64, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
        D = ctypes.POINTER(CpAttnDesc)
        sig = {
            "cp_status_string": ([I32], ctypes.c_char_p),
            "cp_validate_desc": ([D], I32),
            "cp_partition_indices": ([D, P, P, P], I32),
            "cp_permute_tokens": ([D, P, I32, P, P, I32, P], I32),
            "cp_permute_rope": ([D, P, I32, ctypes.c_float, P, P, I32, P], I32),
            "cp_tile_attn_fwd": ([D, P, P, P, I64, I64, I64, I64, I64, I64, P, P, P], I32),
            "cp_merge_partials": ([I32, I64, I32, I32, P, P, P, I32, P, P], I32),
            "cp_ring_attn_workspace_bytes": ([D, I32], SZ),
            "cp_ring_attn_fwd": ([D, P, P, P, P, P, P, SZ, P], I32),
            "cp_ring_attn_bwd": ([D, P, P, P, P, P, P, P, P, P, P, SZ, P], I32),
            "cp_get_device_error": ([P], I32),
            "cp_ring_plan_stats": ([D, P], I32),
            "cp_ring_bwd_schedule": ([D, P, P, P, P, P], I32),
            "cp_profile_enable": ([I32], I32),
            "cp_profile_read": ([P, P], I32),
            "cp_ring_attn_fwd_static_ws": ([D, P, P, P, P, P, P], I32),
            "cp_static_ws_capacity": ([], SZ),
            "cp_hybrid_schedule": ([P, I32, I32, I64, P, P, P, P], I32),
            "cp_ring_plan_tables": ([D, I32, P, P, P, P], I32),
            "cp_token_seq_pos": ([D, P, P, P], I32),
            "cp_debug_set_wait_limit": ([I64], I32),
            "cp_kv_extend": ([I32, I32, I32, I64, I32] + [P] * 11, I32),
            "cp_kv_release": ([I32, I32, I32, I32] + [P] * 8, I32),
            "cp_rope_axes": ([ctypes.POINTER(CpRope), P, I64, I32, I32, I32, P, I64, P, I32, P, I64, P, I32, P], I32),
            "cp_kv_append": ([ctypes.POINTER(CpKvCache), P, I64, P, I64, P, I64, ctypes.POINTER(CpRope), P, I32, P, I64,
                              P, P], I32),
            "cp_validate_paged_desc": ([ctypes.POINTER(CpPagedDesc)], I32),
            "cp_paged_schedule": ([ctypes.POINTER(CpPagedDesc), I32, I64, I32, P, P, P, P, P], I32),
            "cp_paged_attn_workspace_bytes": ([ctypes.POINTER(CpPagedDesc)], SZ),
            "cp_paged_attn_fwd": ([ctypes.POINTER(CpPagedDesc), I32, I64, I32, P, I64, P, P, P, P, P, P, SZ, P], I32),
            "cp_validate_cross_desc": ([ctypes.POINTER(CpCrossDesc)], I32),
            "cp_cross_attn_workspace_bytes": ([ctypes.POINTER(CpCrossDesc), I32, I64, I64, I32], SZ),
            "cp_cross_attn_fwd": ([ctypes.POINTER(CpCrossDesc), I32, I64, I64, P, I64, P, I64, P, I64] + [P] * 10 + [SZ, P],
                                  I32),
            "cp_cross_attn_bwd": ([ctypes.POINTER(CpCrossDesc), I32, I64, I64, P, I64, P, I64, P, I64, P, P, P, P, I64]
                                  + [P] * 11 + [SZ, P], I32),
        }
        for name, (args, res) in sig.items():
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = res
        _lib = L
    return _lib


def _check(code: int, where: str):
    if code != 0:
        raise CpError(code, where)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _dtype_code(dt):
    if dt == torch.bfloat16:
        return CP_BF16
    if dt == torch.float32:
        return CP_F32
    raise ValueError(f"unsupported dtype {dt}")


@dataclass
class Problem:
    """A descriptor plus the arrays it points to (kept alive here)."""
    batch: int
    heads_q: int
    heads_kv: int
    head_dim: int
    cp: int
    seqlen: int
    dtype: torch.dtype = torch.bfloat16
    cu_seqlens: object = None          # host sequence of int (THD) or None (BSHD)
    order: int = CP_ORDER_ORIGINAL
    causal: bool = True
    softmax_scale: float = 0.0
    device: str = "cuda"
    partition: int = CP_PARTITION_ZIGZAG
    window: int = 0                    # sliding-window width (0: none)
    seq_cp: object = None              # hybrid CP: per sub-sequence CP size (host ints) or None
    seq_rank0: object = None           # hybrid CP: first rank of each sub-sequence's group
    _cu_host: np.ndarray = field(default=None, repr=False)
    _cu_dev: torch.Tensor = field(default=None, repr=False)
    _grp_host: list = field(default=None, repr=False)   # hybrid CP arrays kept alive (host)
    _grp_dev: list = field(default=None, repr=False)    # and their device copies
    _desc: CpAttnDesc = field(default=None, repr=False)

    def __post_init__(self):
        d = CpAttnDesc()
        d.batch, d.heads_q, d.heads_kv, d.head_dim = self.batch, self.heads_q, self.heads_kv, self.head_dim
        d.cp, d.causal, d.seqlen = self.cp, int(bool(self.causal)), self.seqlen
        d.dtype, d.order, d.softmax_scale = _dtype_code(self.dtype), self.order, float(self.softmax_scale)
        d.partition = int(self.partition)
        d.window = int(self.window)
        if self.seq_cp is not None:
            self._grp_host = [np.ascontiguousarray(np.asarray(x, dtype=np.int32)) for x in (self.seq_cp, self.seq_rank0)]
            d.seq_cp_host, d.seq_rank0_host = (a.ctypes.data for a in self._grp_host)
            if self.device != "cpu" and torch.cuda.is_available():
                self._grp_dev = [torch.from_numpy(a).to(self.device) for a in self._grp_host]
                d.seq_cp_dev, d.seq_rank0_dev = (t.data_ptr() for t in self._grp_dev)
        if self.cu_seqlens is not None:
            self._cu_host = np.ascontiguousarray(np.asarray(self.cu_seqlens, dtype=np.int32))
            d.cu_seqlens_host = self._cu_host.ctypes.data
            d.n_seqs = len(self._cu_host) - 1
            if self.device != "cpu" and torch.cuda.is_available():
                self._cu_dev = torch.from_numpy(self._cu_host).to(self.device)
                d.cu_seqlens_dev = self._cu_dev.data_ptr()
        self._desc = d

    @property
    def desc(self):
        return ctypes.byref(self._desc)

    @property
    def thd(self) -> bool:
        return self.cu_seqlens is not None


def status_string(code: int) -> str:
    return lib().cp_status_string(code).decode()


def validate(p: Problem) -> int:
    return int(lib().cp_validate_desc(p.desc))


def plan_stats(p: Problem) -> dict:
    out = (ctypes.c_int64 * 6)()
    _check(lib().cp_ring_plan_stats(p.desc, ctypes.cast(out, ctypes.c_void_p)), "cp_ring_plan_stats")
    keys = ("fwd_items", "partial_rows", "merge_segments", "bwd_items", "pairs", "fwd_key_tiles")
    return dict(zip(keys, list(out)))


PLAN_TABLES = {"fwd": 0, "fwd_wide": 1, "bwd": 2, "dq": 3, "merge": 4}


def plan_tables(p: Problem, which: str):
    """The planner's items [n, 8] and segments [m, 4] (int32 numpy, host only)."""
    import numpy as np
    n, m = ctypes.c_int64(0), ctypes.c_int64(0)
    w = PLAN_TABLES[which]
    _check(lib().cp_ring_plan_tables(p.desc, w, ctypes.byref(n), ctypes.byref(m), None, None),
           "cp_ring_plan_tables")
    items = np.zeros((n.value, 8), dtype=np.int32)
    segs = np.zeros((m.value, 4), dtype=np.int32)
    _check(lib().cp_ring_plan_tables(p.desc, w, None, None, items.ctypes.data if n.value else None,
                                     segs.ctypes.data if m.value else None), "cp_ring_plan_tables")
    return items, segs


def bwd_schedule(p: Problem) -> dict:
    """The tensor-core backward's per-CTA work lists (host only): grid, cta
    offsets [grid + 1], work indices and per-CTA planned loads (numpy)."""
    import numpy as np
    grid, n = ctypes.c_int32(0), ctypes.c_int64(0)
    _check(lib().cp_ring_bwd_schedule(p.desc, ctypes.byref(grid), ctypes.byref(n), None, None, None),
           "cp_ring_bwd_schedule")
    cta = np.zeros(grid.value + 1, dtype=np.int32)
    work = np.zeros(n.value, dtype=np.int32)
    load = np.zeros(grid.value, dtype=np.int64)
    _check(lib().cp_ring_bwd_schedule(p.desc, None, None, cta.ctypes.data, work.ctypes.data, load.ctypes.data),
           "cp_ring_bwd_schedule")
    return {"grid": grid.value, "cta": cta, "work": work, "load": load}


def workspace_bytes(p: Problem, backward: bool = False) -> int:
    return int(lib().cp_ring_attn_workspace_bytes(p.desc, int(backward)))


def workspace(p: Problem, backward: bool = False) -> torch.Tensor:
    n = workspace_bytes(p, backward)
    if n == 0:
        raise CpError(-1, "cp_ring_attn_workspace_bytes")
    return torch.empty(n, dtype=torch.uint8, device=p.device)


def partition_indices(p: Problem, out: torch.Tensor | None = None):
    """idx [cp, seqlen/cp] int32 (device) and, for THD, local cu_seqlens.

    Hybrid CP: idx [seqlen] (ranks of different lengths) and local_cu
    [cp, n_seqs + 1], the slot where each rank's slice of each sub-sequence
    starts."""
    if p.seq_cp is not None:
        idx = torch.empty(p.seqlen, dtype=torch.int32, device=p.device) if out is None else out
        local_cu = torch.empty((p.cp, len(p._cu_host)), dtype=torch.int32, device=p.device)
    else:
        idx = torch.empty((p.cp, p.seqlen // p.cp), dtype=torch.int32, device=p.device) if out is None else out
        local_cu = (torch.empty(len(p._cu_host), dtype=torch.int32, device=p.device) if p.thd else None)
    _check(lib().cp_partition_indices(p.desc, _ptr(idx), _ptr(local_cu), _stream()),
           "cp_partition_indices")
    return idx, local_cu


def hybrid_schedule(lens, world: int, capacity: int):
    """Hybrid CP schedule (host only): per sequence (round, cp, rank0) and the round count."""
    L = np.ascontiguousarray(np.asarray(lens, dtype=np.int32))
    n = len(L)
    rnd, cp, r0 = (np.zeros(n, dtype=np.int32) for _ in range(3))
    nr = ctypes.c_int32(0)
    _check(lib().cp_hybrid_schedule(L.ctypes.data if n else None, n, int(world), int(capacity),
                                    rnd.ctypes.data if n else None, cp.ctypes.data if n else None,
                                    r0.ctypes.data if n else None, ctypes.byref(nr)), "cp_hybrid_schedule")
    return rnd, cp, r0, nr.value


def token_seq_pos(p: Problem, idx: torch.Tensor) -> torch.Tensor:
    """[seqlen, 2] int32: sub-sequence index and in-sequence position of every rank-local slot."""
    out = torch.empty((p.seqlen, 2), dtype=torch.int32, device=p.device)
    _check(lib().cp_token_seq_pos(p.desc, _ptr(idx), _ptr(out), _stream()), "cp_token_seq_pos")
    return out


def permute_tokens(p: Problem, idx: torch.Tensor, x: torch.Tensor, inverse: bool = False,
                   out: torch.Tensor | None = None) -> torch.Tensor:
    assert x.is_contiguous() and x.dtype == p.dtype
    heads = x.shape[-2]
    out = torch.empty_like(x) if out is None else out
    _check(lib().cp_permute_tokens(p.desc, _ptr(idx), heads, _ptr(x), _ptr(out), int(inverse),
                                   _stream()), "cp_permute_tokens")
    return out


def permute_rope(p: Problem, idx: torch.Tensor, x: torch.Tensor, rope_base: float = 10000.0,
                 inverse: bool = False, out: torch.Tensor | None = None) -> torch.Tensor:
    """Token gather with the rotary position embedding fused in (cp_permute_rope)."""
    assert x.is_contiguous() and x.dtype == p.dtype
    heads = x.shape[-2]
    out = torch.empty_like(x) if out is None else out
    _check(lib().cp_permute_rope(p.desc, _ptr(idx), heads, float(rope_base), _ptr(x), _ptr(out), int(inverse),
                                 _stream()), "cp_permute_rope")
    return out


def tile_attn_fwd(p: Problem, q, k, v, q_row0, q_pos0, q_len, kv_row0, kv_pos0, kv_len):
    """One TileAttention edge -> (o_part [b, q_len, H, d] f32, lse_part [b, q_len, H] f32)."""
    o = torch.empty((p.batch, q_len, p.heads_q, p.head_dim), dtype=torch.float32, device=q.device)
    l = torch.empty((p.batch, q_len, p.heads_q), dtype=torch.float32, device=q.device)
    _check(lib().cp_tile_attn_fwd(p.desc, _ptr(q), _ptr(k), _ptr(v), q_row0, q_pos0, q_len,
                                  kv_row0, kv_pos0, kv_len, _ptr(o), _ptr(l), _stream()),
           "cp_tile_attn_fwd")
    return o, l


def merge_partials(o_parts: torch.Tensor, lse_parts: torch.Tensor, out_dtype=torch.float32):
    """o_parts [P, rows, H, d] f32, lse_parts [P, rows, H] f32 -> (o, lse)."""
    n, rows, H, d = o_parts.shape
    o = torch.empty((rows, H, d), dtype=out_dtype, device=o_parts.device)
    l = torch.empty((rows, H), dtype=torch.float32, device=o_parts.device)
    _check(lib().cp_merge_partials(n, rows, H, d, _ptr(o_parts), _ptr(lse_parts), _ptr(o),
                                   _dtype_code(out_dtype), _ptr(l), _stream()), "cp_merge_partials")
    return o, l


def ring_attn_fwd(p: Problem, q, k, v, ws: torch.Tensor | None = None, out=None, lse=None):
    ws = workspace(p, False) if ws is None else ws
    o = torch.empty_like(q) if out is None else out
    l = (torch.empty(q.shape[:-1], dtype=torch.float32, device=q.device) if lse is None else lse)
    _check(lib().cp_ring_attn_fwd(p.desc, _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(l), _ptr(ws),
                                  ws.numel(), _stream()), "cp_ring_attn_fwd")
    return o, l


def ring_attn_bwd(p: Problem, q, k, v, o, lse, dout, ws: torch.Tensor | None = None,
                  dq=None, dk=None, dv=None):
    ws = workspace(p, True) if ws is None else ws
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    _check(lib().cp_ring_attn_bwd(p.desc, _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dout),
                                  _ptr(dq), _ptr(dk), _ptr(dv), _ptr(ws), ws.numel(), _stream()),
           "cp_ring_attn_bwd")
    return dq, dk, dv


# ---------------------------------------------------------------- serving ---
class PagedKV:
    """The pages of a K/V cache: two [n_pages, page_size, heads_kv, head_dim]
    views of the same strides (any order of pages, tokens and heads in memory,
    head_dim contiguous), kept alive here."""

    def __init__(self, k_cache: torch.Tensor, v_cache: torch.Tensor):
        if k_cache.dim() != 4 or k_cache.shape != v_cache.shape or k_cache.stride() != v_cache.stride():
            raise ValueError("k_cache and v_cache are [n_pages, page_size, heads_kv, head_dim] views of the same strides")
        if k_cache.dtype != v_cache.dtype or k_cache.device != v_cache.device or k_cache.stride(3) != 1:
            raise ValueError("k_cache and v_cache share their type and device, head_dim contiguous")
        self.k_cache, self.v_cache = k_cache, v_cache
        self.n_pages, self.page_size, self.heads_kv, self.head_dim = k_cache.shape
        self.dtype, self.device, self._index = k_cache.dtype, k_cache.device, k_cache.get_device()
        s = k_cache.stride()
        self._desc = CpKvCache(k_cache.data_ptr(), v_cache.data_ptr(), *k_cache.shape, s[0], s[1], s[2],
                               _dtype_code(k_cache.dtype))
        self._ref = ctypes.byref(self._desc)


class Rope:
    """Rotary positions with several axes (cp_rope): pairs of each axis."""

    def __init__(self, sections, base: float = 10000.0, interleaved: bool = False, restart: bool = False,
                 adjacent: bool = False):
        self.sections = [int(x) for x in sections]
        if not 1 <= len(self.sections) <= 4:
            raise ValueError("one to four axes")
        self._desc = CpRope(len(self.sections), (ctypes.c_int32 * 4)(*self.sections), int(interleaved), int(restart),
                            int(adjacent), float(base))
        self._ref = ctypes.byref(self._desc)


class PagedProblem:
    """Attention over a paged cache (cp_paged_desc)."""

    def __init__(self, kv: PagedKV, heads_q: int, max_new: int = 0, causal: bool = True, window: int = 0,
                 softmax_scale: float = 0.0):
        self.kv, self.heads_q = kv, int(heads_q)
        self._desc = CpPagedDesc(kv._desc, self.heads_q, int(max_new), int(bool(causal)), int(window),
                                 float(softmax_scale))
        self._ref = ctypes.byref(self._desc)


# A call's checks, marshalling and output tensors cost more host time than its
# launch (a few microseconds, which a step of small calls feels).  So the
# checks compare singletons and device indices, the raw stream is looked up
# directly, and new tensors are made below PyTorch's dispatcher where it offers
# that (a table call's five outputs: 12 us through it, 4 us below).
_I32, _F32 = torch.int32, torch.float32
try:
    _raw_stream = torch._C._cuda_getCurrentRawStream
except AttributeError:  # a PyTorch without CUDA: the host-only calls still work
    def _raw_stream(device):
        return torch.cuda.current_stream(device).cuda_stream
try:
    from torch._C._dynamo.guards import _empty_strided_cuda, _reinterpret_tensor
except ImportError:  # the same by the public functions
    def _empty_strided_cuda(size, stride, dtype):
        return torch.empty_strided(size, stride, dtype=dtype, device="cuda")

    def _reinterpret_tensor(x, size, stride, offset):
        return x.as_strided(size, stride, offset)


def _rows(x: torch.Tensor, what: str, heads: int, d: int, dtype, device: int):
    """Row stride (elements) of a [rows, heads, d] tensor whose rows are contiguous."""
    shape = x.shape
    if len(shape) != 3 or shape[1] != heads or shape[2] != d or x.dtype is not dtype or x.get_device() != device:
        raise ValueError(f"{what} is a [rows, {heads}, {d}] {dtype} tensor on cuda:{device}")
    s = x.stride()
    if s[2] != 1 or (s[1] != d and heads > 1):
        raise ValueError(f"{what}: the heads of a row are contiguous")
    return s[0] if shape[0] > 1 else heads * d


def _ints(x: torch.Tensor, what: str, shape, device: int):
    if x.dtype is not _I32 or x.shape != shape or x.get_device() != device or not x.is_contiguous():
        raise ValueError(f"{what} is a contiguous {list(shape)} int32 tensor on cuda:{device}")
    return x.data_ptr()


def _new(out, what, shape, dtype, device: int):
    """The caller's output tensor (contiguous, of that shape and type), or a
    new one on the current device."""
    if out is None:
        return _empty_strided_cuda(shape, (shape[1] * shape[2], shape[2], 1) if len(shape) == 3 else (shape[1], 1), dtype)
    if out.shape != shape or out.dtype is not dtype or out.get_device() != device or not out.is_contiguous():
        raise ValueError(f"{what} is a contiguous {list(shape)} {dtype} tensor on cuda:{device}")
    return out


def _stream_of(device: int) -> int:
    """The current stream of the device that holds the tensors (it has to be the current device)."""
    if device < 0 or device != torch.cuda.current_device():
        raise ValueError("the tensors are not on the current CUDA device")
    return _raw_stream(device)


def _tables(block_table, free_pages, n_free, **per_request):
    """Sizes, device index and pointers of a call on the request tables."""
    if block_table.dim() != 2:
        raise ValueError("block_table is [n_reqs, max_blocks]")
    n, width = block_table.shape
    dev = block_table.get_device()
    pool = free_pages.numel()
    args = [_ints(x, name, (n,), dev) for name, x in per_request.items()]
    args += [_ints(free_pages, "free_pages", (pool,), dev), _ints(n_free, "n_free", (1,), dev),
             _ints(block_table, "block_table", (n, width), dev)]
    return n, width, pool, args, _stream_of(dev)


def kv_extend(page_size: int, block_table, lens, add, free_pages, n_free, max_rows: int):
    """Pages, slots and positions for `add` new tokens of every request (cp_kv_extend).

    block_table [n_reqs, max_blocks] changes in place; returns (lens, cu_new,
    slots, pos, n_free), views of one new allocation that lives as long as any
    of them (clone what is kept for long)."""
    n, width, pool, args, s = _tables(block_table, free_pages, n_free, lens=lens, add=add)
    out = _empty_strided_cuda((2 * n + 2 + 2 * max_rows,), (1,), _I32)
    at = out.data_ptr()
    rows_at = at + 4 * (2 * n + 2)
    _check(lib().cp_kv_extend(n, width, page_size, max_rows, pool, *args, at, at + 4 * n, rows_at,
                              rows_at + 4 * max_rows, rows_at - 4, s), "cp_kv_extend")
    one, view = (1,), _reinterpret_tensor
    return (view(out, (n,), one, 0), view(out, (n + 1,), one, n), view(out, (max_rows,), one, 2 * n + 2),
            view(out, (max_rows,), one, 2 * n + 2 + max_rows), view(out, one, one, 2 * n + 1))


def kv_release(page_size: int, block_table, lens, done, free_pages, n_free):
    """Gives the pages of the requests with done != 0 back (cp_kv_release);
    block_table and free_pages change in place; returns (lens, n_free).  Entries
    below zero (pages given back before) are passed over."""
    n, width, pool, args, s = _tables(block_table, free_pages, n_free, lens=lens, done=done)
    lens_out, n_free_out = torch.empty_like(lens), torch.empty_like(n_free)
    _check(lib().cp_kv_release(n, width, page_size, pool, *args, lens_out.data_ptr(), n_free_out.data_ptr(), s),
           "cp_kv_release")
    return lens_out, n_free_out


def _positions(rope: Rope, pos: torch.Tensor, rows: int, device: int):
    axes = len(rope.sections)
    return _ints(pos, "pos", (rows,) if axes == 1 and pos.dim() == 1 else (axes, rows), device)


def rope_axes(rope: Rope, pos, q, k=None, inverse: bool = False, q_out=None, k_out=None):
    """Rotates q [rows, heads, head_dim] (and k) by pos [axes, rows] (cp_rope_axes);
    inverse: the transpose, which is the gradient."""
    if q.dim() != 3 or (k is not None and k.dim() != 3):
        raise ValueError("q and k are [rows, heads, head_dim]")
    dev, dt = q.get_device(), q.dtype
    rows, hq, d = q.shape
    qs, hk, ks, kp, ko = _rows(q, "q", hq, d, dt, dev), 0, 0, None, None
    p, s = _positions(rope, pos, rows, dev), _stream_of(dev)
    q_out = _new(q_out, "q_out", (rows, hq, d), dt, dev)
    if k is not None:
        hk = k.shape[1]
        ks = _rows(k, "k", hk, d, dt, dev)
        if k.shape[0] != rows:
            raise ValueError("q and k have the same rows")
        k_out = _new(k_out, "k_out", (rows, hk, d), dt, dev)
        kp, ko = k.data_ptr(), k_out.data_ptr()
    _check(lib().cp_rope_axes(rope._ref, p, rows, d, _dtype_code(dt), hq, q.data_ptr(), qs, q_out.data_ptr(), hk, kp, ks,
                              ko, int(inverse), s), "cp_rope_axes")
    return q_out if k is None else (q_out, k_out)


def kv_append(kv: PagedKV, slots, k, v, rope: Rope | None = None, pos=None, q=None, q_out=None):
    """Writes k and v [rows, heads_kv, head_dim] into the slots of the cache
    (cp_kv_append); with rope, k is rotated by pos on the way and q into the
    returned q_out.  Rows whose slot is outside the cache (a padded batch's) are
    left out: their q_out rows stay as they were, unset in a new q_out."""
    dev, dt, heads, d = kv._index, kv.dtype, kv.heads_kv, kv.head_dim
    rows = k.shape[0]
    ks, vs = _rows(k, "k", heads, d, dt, dev), _rows(v, "v", heads, d, dt, dev)
    if v.shape[0] != rows:
        raise ValueError("k and v have the same rows")
    if (rope is None) != (pos is None) or (q is not None and rope is None):
        raise ValueError("rope, pos and q: positions come with a rotation, q is rotated")
    hq, qs, qp, qo, r, p = 0, 0, None, None, None, None
    if rope is not None:
        r, p = rope._ref, _positions(rope, pos, rows, dev)
    at, s = _ints(slots, "slots", (rows,), dev), _stream_of(dev)
    if q is not None:
        if q.dim() != 3 or q.shape[0] != rows:
            raise ValueError("q is [rows, heads_q, head_dim]")
        hq = q.shape[1]
        qs = _rows(q, "q", hq, d, dt, dev)
        q_out = _new(q_out, "q_out", (rows, hq, d), dt, dev)
        qp, qo = q.data_ptr(), q_out.data_ptr()
    _check(lib().cp_kv_append(kv._ref, at, rows, k.data_ptr(), ks, v.data_ptr(), vs, r, p, hq, qp, qs, qo, s),
           "cp_kv_append")
    return None if q is None else q_out


def validate_paged(p: PagedProblem) -> int:
    return int(lib().cp_validate_paged_desc(p._ref))


def paged_workspace_bytes(p: PagedProblem) -> int:
    return int(lib().cp_paged_attn_workspace_bytes(p._ref))


def paged_workspace(p: PagedProblem) -> torch.Tensor:
    n = paged_workspace_bytes(p)
    if n == 0:
        raise CpError(validate_paged(p), "cp_paged_attn_workspace_bytes")
    return torch.empty(n, dtype=torch.uint8, device=p.kv.device)


def paged_schedule(p: PagedProblem, cu_new, kv_lens, rows: int, max_blocks: int):
    """The pieces [n, 8] of a call with these lengths (host only): block, request,
    kv-head, first packed row, packed rows, first key, end of its keys, slot
    (-1: the outputs); and the number of blocks."""
    cu, lens = (np.ascontiguousarray(np.asarray(x, dtype=np.int32)) for x in (cu_new, kv_lens))
    n, grid = ctypes.c_int64(0), ctypes.c_int32(0)
    args = (p._ref, len(lens), rows, max_blocks, cu.ctypes.data, lens.ctypes.data)
    _check(lib().cp_paged_schedule(*args, ctypes.byref(grid), ctypes.byref(n), None), "cp_paged_schedule")
    out = np.zeros((n.value, 8), dtype=np.int32)
    _check(lib().cp_paged_schedule(*args, None, None, out.ctypes.data), "cp_paged_schedule")
    return out, grid.value


def paged_attn_fwd(p: PagedProblem, q, block_table, cu_new, kv_lens, ws: torch.Tensor | None = None, out=None,
                   lse=None):
    """Attention of the new tokens q [rows, heads_q, head_dim] over the pages of
    their requests (cp_paged_attn_fwd) -> (o, lse).  Rows behind the last
    request's are left as they were (unset in a new o and lse)."""
    kv, heads = p.kv, p.heads_q
    dev, d = kv._index, kv.head_dim
    qs = _rows(q, "q", heads, d, kv.dtype, dev)
    if block_table.dim() != 2:
        raise ValueError("block_table is [n_reqs, max_blocks]")
    n, width = block_table.shape
    table, cu, lens = (_ints(block_table, "block_table", (n, width), dev), _ints(cu_new, "cu_new", (n + 1,), dev),
                       _ints(kv_lens, "kv_lens", (n,), dev))
    s = _stream_of(dev)
    if ws is None:
        ws = paged_workspace(p)
    elif ws.get_device() != dev or not ws.is_contiguous():
        raise ValueError(f"ws is a contiguous tensor on cuda:{dev}")
    rows = q.shape[0]
    out = _new(out, "out", (rows, heads, d), kv.dtype, dev)
    lse = _new(lse, "lse", (rows, heads), _F32, dev)
    _check(lib().cp_paged_attn_fwd(p._ref, n, rows, width, q.data_ptr(), qs, table, cu, lens, out.data_ptr(),
                                   lse.data_ptr(), ws.data_ptr(), ws.nbytes, s), "cp_paged_attn_fwd")
    return out, lse


# -------------------------------------------------------- cross attention ---
class RelBuckets:
    """Buckets of the relative position (cp_cross_desc): `buckets` of them, the
    last one from at most `max_distance` on; both: keys behind the query have
    half of them for themselves."""

    def __init__(self, buckets: int, max_distance: int = 128, both: bool = True):
        self.buckets, self.max_distance, self.both = int(buckets), int(max_distance), bool(both)


class CrossProblem:
    """Attention of packed query sequences over packed key sequences (cp_cross_desc).

    max_q: about how many queries a sequence has at most (chooses the forward's
    kernel; 0: many); rel: a bias by buckets of the relative position; dropout: of the probabilities, to the
    nearest multiple of 2^-15 (halves to even)."""

    def __init__(self, heads_q: int, heads_kv: int, head_dim: int, dtype: torch.dtype = torch.bfloat16,
                 causal: bool = False, max_q: int = 0, rel: RelBuckets | None = None, dropout: float = 0.0,
                 softmax_scale: float = 0.0):
        self.heads_q, self.heads_kv, self.head_dim, self.dtype = int(heads_q), int(heads_kv), int(head_dim), dtype
        self.rel, self.dropout, self.causal = rel, float(dropout), bool(causal)
        if 0.0 < self.dropout < 1.0:  # here, in 64 bits: a float next to a border rounds to the other side
            self.dropout = round(self.dropout * 32768) / 32768
        r = (rel.buckets, rel.max_distance, int(rel.both)) if rel is not None else (0, 0, 0)
        self._desc = CpCrossDesc(self.heads_q, self.heads_kv, self.head_dim, _dtype_code(dtype), int(bool(causal)),
                                 int(max_q), *r, self.dropout, float(softmax_scale))
        self._ref = ctypes.byref(self._desc)


def validate_cross(p: CrossProblem) -> int:
    return int(lib().cp_validate_cross_desc(p._ref))


def cross_workspace_bytes(p: CrossProblem, n_seqs: int, rows_q: int, rows_k: int, backward: bool = False) -> int:
    return int(lib().cp_cross_attn_workspace_bytes(p._ref, n_seqs, rows_q, rows_k, int(backward)))


def cross_workspace(p: CrossProblem, n_seqs: int, rows_q: int, rows_k: int, backward: bool = False,
                    device="cuda") -> torch.Tensor:
    """A workspace for cross_attn_fwd, and with backward for cross_attn_bwd too."""
    n = cross_workspace_bytes(p, n_seqs, rows_q, rows_k, backward)
    if n == 0:
        raise CpError(validate_cross(p) or -1, "cp_cross_attn_workspace_bytes")
    return torch.empty(n, dtype=torch.uint8, device=device)


def _cross_inputs(p: CrossProblem, q, k, v, cu_q, cu_k, len_q, len_k, bias, rng):
    """Device index, sizes and leading arguments of both directions (checks included)."""
    dev, d, dt = q.get_device(), p.head_dim, p.dtype
    qs = _rows(q, "q", p.heads_q, d, dt, dev)
    ks, vs = _rows(k, "k", p.heads_kv, d, dt, dev), _rows(v, "v", p.heads_kv, d, dt, dev)
    rows_q, rows_k = q.shape[0], k.shape[0]
    if v.shape[0] != rows_k:
        raise ValueError("k and v have the same rows")
    n = cu_q.numel() - 1
    if n < 0:
        raise ValueError("cu_q is [n_seqs + 1]")
    cu = (_ints(cu_q, "cu_q", (n + 1,), dev), _ints(cu_k, "cu_k", (n + 1,), dev))
    lens = tuple(None if x is None else _ints(x, what, (n,), dev) for x, what in ((len_q, "len_q"), (len_k, "len_k")))
    if (p.rel is None) != (bias is None):
        raise ValueError("a bias table comes with the problem's rel, and the other way round")
    if bias is not None:
        shape = (p.rel.buckets, p.heads_q)
        if bias.shape != shape or bias.dtype is not dt or bias.get_device() != dev or not bias.is_contiguous():
            raise ValueError(f"bias is a contiguous {list(shape)} {dt} tensor on cuda:{dev}")
        bias = bias.data_ptr()
    if p.dropout > 0.0:
        if rng is None or rng.dtype is not torch.int64 or rng.shape != (2,) or rng.get_device() != dev \
                or not rng.is_contiguous():
            raise ValueError(f"dropout takes rng, a contiguous [2] int64 tensor (seed, offset) on cuda:{dev}")
        rng = rng.data_ptr()
    else:
        rng = None
    return dev, n, rows_q, rows_k, (q.data_ptr(), qs, k.data_ptr(), ks, v.data_ptr(), vs), cu + lens, bias, rng


def _cross_ws(p, ws, n, rows_q, rows_k, backward, dev):
    if ws is None:
        return cross_workspace(p, n, rows_q, rows_k, backward, torch.device("cuda", dev))
    if ws.get_device() != dev or not ws.is_contiguous():
        raise ValueError(f"ws is a contiguous tensor on cuda:{dev}")
    return ws


def cross_attn_fwd(p: CrossProblem, q, k, v, cu_q, cu_k, len_q=None, len_k=None, bias=None, rng=None,
                   for_backward: bool = False, ws: torch.Tensor | None = None, out=None, lse=None):
    """Attention of q [rows_q, heads_q, head_dim] over k and v [rows_k, heads_kv, head_dim],
    sequence by sequence (cp_cross_attn_fwd) -> (o, lse).  Rows that no sequence owns are
    left as they were (unset in a new o and lse).  for_backward: -> (o, lse, rest), rest what o lost
    to rounding, which cross_attn_bwd takes (the gradients of rows whose weight lies on few keys, and a bias table's; None
    in float32, and with a bias for more than 128 q-heads a kv-head)."""
    dev, n, rows_q, rows_k, qkv, cu, bias, rng = _cross_inputs(p, q, k, v, cu_q, cu_k, len_q, len_k, bias, rng)
    s = _stream_of(dev)
    ws = _cross_ws(p, ws, n, rows_q, rows_k, False, dev)
    heads, d = p.heads_q, p.head_dim
    out = _new(out, "out", (rows_q, heads, d), p.dtype, dev)
    lse = _new(lse, "lse", (rows_q, heads), _F32, dev)
    rest = None
    if for_backward and p.dtype is torch.bfloat16 and (bias is None or heads <= 128 * p.heads_kv):
        rest = _new(None, "rest", (rows_q, heads, d), p.dtype, dev)
    _check(lib().cp_cross_attn_fwd(p._ref, n, rows_q, rows_k, *qkv, *cu, bias, rng, out.data_ptr(),
                                   None if rest is None else rest.data_ptr(), lse.data_ptr(), ws.data_ptr(), ws.nbytes, s),
           "cp_cross_attn_fwd")
    return (out, lse, rest) if for_backward else (out, lse)


def cross_attn_bwd(p: CrossProblem, q, k, v, o, lse, dout, cu_q, cu_k, len_q=None, len_k=None, bias=None, rng=None,
                   rest=None, ws: torch.Tensor | None = None, dq=None, dk=None, dv=None, dbias=None):
    """Gradients (cp_cross_attn_bwd) -> (dq, dk, dv, dbias); dbias is None without a bias.
    o, lse and rest are cross_attn_fwd's for the same inputs and rng (in bf16 without rest the gradients of rows whose weight
    lies on few keys lose digits, and so does dbias over many).  Rows that no sequence owns get zeros."""
    dev, n, rows_q, rows_k, qkv, cu, bias, rng = _cross_inputs(p, q, k, v, cu_q, cu_k, len_q, len_k, bias, rng)
    s = _stream_of(dev)
    ws = _cross_ws(p, ws, n, rows_q, rows_k, True, dev)
    heads, d, dt = p.heads_q, p.head_dim, p.dtype
    ds = _rows(dout, "dout", heads, d, dt, dev)
    if dout.shape[0] != rows_q:
        raise ValueError("dout has q's rows")
    for x, what, shape, t in ((o, "o", (rows_q, heads, d), dt), (lse, "lse", (rows_q, heads), _F32)) \
            + (() if rest is None else ((rest, "rest", (rows_q, heads, d), dt),)):
        if x.shape != shape or x.dtype is not t or x.get_device() != dev or not x.is_contiguous():
            raise ValueError(f"{what} is a contiguous {list(shape)} {t} tensor on cuda:{dev}")
    dq = _new(dq, "dq", (rows_q, heads, d), dt, dev)
    dk, dv = (_new(x, what, (rows_k, p.heads_kv, d), dt, dev) for x, what in ((dk, "dk"), (dv, "dv")))
    if bias is not None:
        dbias = _new(dbias, "dbias", (p.rel.buckets, heads), dt, dev)
    elif dbias is not None:
        raise ValueError("dbias comes with a bias")
    _check(lib().cp_cross_attn_bwd(p._ref, n, rows_q, rows_k, *qkv, o.data_ptr(), None if rest is None else rest.data_ptr(),
                                   lse.data_ptr(), dout.data_ptr(), ds, *cu, bias, rng, dq.data_ptr(), dk.data_ptr(),
                                   dv.data_ptr(), None if dbias is None else dbias.data_ptr(), ws.data_ptr(), ws.nbytes, s),
           "cp_cross_attn_bwd")
    return dq, dk, dv, dbias


def device_error() -> int:
    """Synchronises the current stream and returns the library's device status."""
    return int(lib().cp_get_device_error(_stream()))


def set_wait_limit(cycles: int) -> None:
    """Cycle budget of the tcgen05 kernels' main-loop waits (0: the default)."""
    _check(lib().cp_debug_set_wait_limit(int(cycles)), "cp_debug_set_wait_limit")


def profile_enable(on: bool = True) -> None:
    _check(lib().cp_profile_enable(int(on)), "cp_profile_enable")


def profile_read() -> dict:
    """{class: (total_ms, launches)} since the last read (waits for the events)."""
    ms = (ctypes.c_double * len(KERNEL_CLASSES))()
    n = (ctypes.c_int64 * len(KERNEL_CLASSES))()
    _check(lib().cp_profile_read(ctypes.cast(ms, ctypes.c_void_p), ctypes.cast(n, ctypes.c_void_p)),
           "cp_profile_read")
    return {name: (ms[i], n[i]) for i, name in enumerate(KERNEL_CLASSES)}
