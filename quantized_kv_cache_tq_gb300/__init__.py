"""Attention over a TurboQuant-compressed KV cache on GB300 (sm_103a).

The compute lives in libtq.so (C ABI, include/tq.h); ``_lib`` binds it with
ctypes under the same names.  The helpers below only hold PyTorch tensors for
device memory and pass their pointers and the current CUDA stream through.
"""
from __future__ import annotations

import ctypes as C
import math

from . import _lib
from ._lib import (TQ_BF16, TQ_DECODE_AUTO, TQ_DECODE_LUT, TQ_DECODE_MMA, TQ_F16, TQ_F32,
                   TQ_TURBO2, TQ_TURBO3, TQ_TURBO4, TQError, tq_cache, tq_codebook, tq_paged4)

QS_BYTES = {2: 32, 3: 32, 4: 64}


def _torch():
    import torch
    return torch


def _stream(stream=None):
    torch = _torch()
    s = torch.cuda.current_stream() if stream is None else stream
    return s.cuda_stream


class TqCache:
    """Device planes of one compressed cache (K or V), allocated with PyTorch."""

    def __init__(self, tq_type: int, n_kv_heads: int, head_dim: int, n_cells: int, device="cuda"):
        torch = _torch()
        nb = (head_dim + 127) // 128
        self.tq_type, self.n_kv_heads, self.head_dim, self.n_cells, self.n_blocks = (
            tq_type, n_kv_heads, head_dim, n_cells, nb)
        self.norms = torch.zeros((n_kv_heads, n_cells, nb), dtype=torch.int16, device=device)
        self.qs = torch.zeros((n_kv_heads, n_cells, nb, QS_BYTES[tq_type]), dtype=torch.uint8, device=device)
        self.signs = (torch.zeros((n_kv_heads, n_cells, nb, 16), dtype=torch.uint8, device=device)
                      if tq_type == 3 else None)
        self.c = tq_cache(tq_type, n_kv_heads, head_dim, nb, n_cells, self.norms.data_ptr(),
                          self.qs.data_ptr(), 0 if self.signs is None else self.signs.data_ptr())

    def planes(self):
        return self.norms, self.qs, self.signs


def codebook(tq_type: int, sign_bits) -> tq_codebook:
    return _lib.tq_codebook_init(tq_type, sign_bits)


def workspace(nbytes: int, device="cuda"):
    """Zero-filled, 256-byte aligned workspace (PyTorch allocations are)."""
    torch = _torch()
    return torch.zeros(max(int(nbytes), 256), dtype=torch.uint8, device=device)


def set_rows(cache: TqCache, cb: tq_codebook, src, cell_ids, dev_status=None, stream=None):
    torch = _torch()
    src_type = {torch.float32: TQ_F32, torch.float16: TQ_F16, torch.bfloat16: TQ_BF16}[src.dtype]
    assert src.is_contiguous() and cell_ids.dtype == torch.int64 and cell_ids.is_contiguous()
    st = _lib.tq_set_rows(cache.c, cb, src.data_ptr(), src_type, cell_ids.data_ptr(),
                          cell_ids.numel(), None if dev_status is None else dev_status.data_ptr(),
                          _stream(stream))
    _lib.check("tq_set_rows", st)


def fattn_decode(kc: TqCache, vc: TqCache, cbk, cbv, q, kv_len: int, scale: float | None = None,
                 algo: int = TQ_DECODE_AUTO, out=None, ws=None, stream=None, sparse_v: float = 0.0):
    """Decode over cells 0..kv_len-1; ``sparse_v`` > 0 leaves out of the V sum the
    keys whose weights relative to the running maximum are below it."""
    torch = _torch()
    n_q = q.shape[0]
    scale = 1.0 / math.sqrt(kc.head_dim) if scale is None else scale
    if out is None:
        out = torch.empty((n_q, vc.head_dim), dtype=torch.float32, device=q.device)
    if ws is None:
        ws = workspace(_lib.tq_fattn_decode_workspace(kc.c, vc.c, n_q, kv_len), q.device)
    if sparse_v:
        st = _lib.tq_fattn_decode_sparse_v(kc.c, vc.c, cbk, cbv, q.data_ptr(), n_q, kv_len, scale, sparse_v,
                                           algo, out.data_ptr(), ws.data_ptr(), ws.numel(), _stream(stream))
        _lib.check("tq_fattn_decode_sparse_v", st)
    else:
        st = _lib.tq_fattn_decode(kc.c, vc.c, cbk, cbv, q.data_ptr(), n_q, kv_len, scale, algo,
                                  out.data_ptr(), ws.data_ptr(), ws.numel(), _stream(stream))
        _lib.check("tq_fattn_decode", st)
    return out


def fattn_decode_append(kc: TqCache, vc: TqCache, cbk, cbv, k_row, v_row, cell_id, q, kv_len: int,
                        scale: float | None = None, algo: int = TQ_DECODE_AUTO, out=None, ws=None, stream=None):
    """SET_ROWS of one token's K/V rows ([n_kv_heads][head_dim]) into cell ``cell_id``
    (a device int64 tensor of one element), then decode over cells 0..kv_len-1."""
    torch = _torch()
    n_q = q.shape[0]
    src_type = {torch.float32: TQ_F32, torch.float16: TQ_F16, torch.bfloat16: TQ_BF16}[k_row.dtype]
    assert v_row.dtype == k_row.dtype and k_row.is_contiguous() and v_row.is_contiguous()
    assert cell_id.dtype == torch.int64 and cell_id.numel() == 1
    scale = 1.0 / math.sqrt(kc.head_dim) if scale is None else scale
    if out is None:
        out = torch.empty((n_q, vc.head_dim), dtype=torch.float32, device=q.device)
    if ws is None:
        ws = workspace(_lib.tq_fattn_decode_workspace(kc.c, vc.c, n_q, kv_len), q.device)
    st = _lib.tq_fattn_decode_append(kc.c, vc.c, cbk, cbv, k_row.data_ptr(), v_row.data_ptr(), src_type,
                                     cell_id.data_ptr(), q.data_ptr(), n_q, kv_len, scale, algo,
                                     out.data_ptr(), ws.data_ptr(), ws.numel(), _stream(stream))
    _lib.check("tq_fattn_decode_append", st)
    return out


def fattn_decode_batch(kc: TqCache, vc: TqCache, cbk, cbv, q, seq_cell0, seq_len, scale: float | None = None,
                       algo: int = TQ_DECODE_AUTO, out=None, ws=None, stream=None):
    """Decode of several sequences in one launch: q [n_seq][n_q_heads][Dk];
    sequence s attends cells seq_cell0[s] .. + seq_len[s] - 1 (host integers)."""
    torch = _torch()
    n_seq, n_q, _ = q.shape
    scale = 1.0 / math.sqrt(kc.head_dim) if scale is None else scale
    if out is None:
        out = torch.empty((n_seq, n_q, vc.head_dim), dtype=torch.float32, device=q.device)
    if ws is None:
        ws = workspace(_lib.tq_fattn_decode_batch_workspace(kc.c, vc.c, n_q, n_seq, max(seq_len)), q.device)
    st = _lib.tq_fattn_decode_batch(kc.c, vc.c, cbk, cbv, q.data_ptr(), n_q, list(seq_cell0), list(seq_len), scale,
                                    algo, out.data_ptr(), ws.data_ptr(), ws.numel(), _stream(stream))
    _lib.check("tq_fattn_decode_batch", st)
    return out


def fattn_prefill(kc: TqCache, vc: TqCache, cbk, cbv, q, kv_len: int, scale: float | None = None,
                  causal: bool = True, out=None, ws=None, stream=None):
    torch = _torch()
    nq, n_q, _ = q.shape
    q_type = {torch.float32: TQ_F32, torch.float16: TQ_F16, torch.bfloat16: TQ_BF16}[q.dtype]
    scale = 1.0 / math.sqrt(kc.head_dim) if scale is None else scale
    if out is None:
        out = torch.empty((nq, n_q, vc.head_dim), dtype=torch.float32, device=q.device)
    if ws is None:
        ws = workspace(_lib.tq_fattn_prefill_workspace(kc.c, vc.c, nq, n_q, kv_len), q.device)
    st = _lib.tq_fattn_prefill(kc.c, vc.c, cbk, cbv, q.data_ptr(), q_type, nq, n_q, kv_len, scale,
                               int(causal), out.data_ptr(), ws.data_ptr(), ws.numel(), _stream(stream))
    _lib.check("tq_fattn_prefill", st)
    return out


def int8_prompt_attn(k, k_scale, v, v_scale, cell_of_pos, ctx: int, q, scale: float | None = None,
                     causal: bool = True, out=None, ws=None, stream=None):
    torch = _torch()
    n_cells, n_kv, d = k.shape
    nq, n_q, _ = q.shape
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    if out is None:
        out = torch.empty((nq, n_q, d), dtype=torch.float32, device=q.device)
    if ws is None:
        ws = workspace(_lib.tq_int8_prompt_attn_workspace(nq, n_q, n_kv, d, ctx), q.device)
    st = _lib.tq_int8_prompt_attn(k.data_ptr(), k_scale.data_ptr(), v.data_ptr(), v_scale.data_ptr(),
                                  n_cells, cell_of_pos.data_ptr(), ctx, q.data_ptr(), nq, n_q, n_kv, d,
                                  scale, int(causal), out.data_ptr(), ws.data_ptr(), ws.numel(),
                                  _stream(stream))
    _lib.check("tq_int8_prompt_attn", st)
    return out


def f16_prompt_attn(k, v, cell_of_pos, ctx: int, q, scale: float | None = None, causal: bool = True, out=None,
                    ws=None, stream=None):
    """Prompt attention over binary16 K/V rows [n_cells][n_kv_heads][128] gathered
    through cell_of_pos (the int8 path's other cache mode, no scales)."""
    torch = _torch()
    assert k.dtype == torch.float16 and v.dtype == torch.float16
    n_cells, n_kv, d = k.shape
    nq, n_q, _ = q.shape
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    if out is None:
        out = torch.empty((nq, n_q, d), dtype=torch.float32, device=q.device)
    if ws is None:
        ws = workspace(_lib.tq_int8_prompt_attn_workspace(nq, n_q, n_kv, d, ctx), q.device)
    st = _lib.tq_f16_prompt_attn(k.data_ptr(), v.data_ptr(), n_cells, cell_of_pos.data_ptr(), ctx, q.data_ptr(),
                                 nq, n_q, n_kv, d, scale, int(causal), out.data_ptr(), ws.data_ptr(), ws.numel(),
                                 _stream(stream))
    _lib.check("tq_f16_prompt_attn", st)
    return out


def checksum(t) -> str:
    """FNV-1a 64 of a tensor's bytes (copied to the host), as 16 hex digits."""
    import numpy as np
    a = np.ascontiguousarray(t.detach().cpu().numpy())
    return f"{_lib.tq_checksum_fnv1a64(a.ctypes.data, a.nbytes):016x}"


# ---- paged 4-bit cache (include/tq.h, "Paged 4-bit cache")

# These calls also serve single decode steps, where the host's share counts: checks are plain comparisons.

_T = None                        # torch's names used on every call, bound on the first one


class _Torch:
    def __init__(self):
        torch = _torch()
        self.int32, self.int64, self.float32, self.uint8 = torch.int32, torch.int64, torch.float32, torch.uint8
        self.float16, self.empty, self.zeros = torch.float16, torch.empty, torch.zeros
        self.row_types = {torch.float32: TQ_F32, torch.float16: TQ_F16, torch.bfloat16: TQ_BF16}
        self.raw_stream = torch._C._cuda_getCurrentRawStream
        self.current = torch.cuda.current_device


def _t() -> _Torch:
    global _T
    if _T is None:
        _T = _Torch()
    return _T


def _need(ok, what: str):
    if not ok:
        raise ValueError(what)


def _row_type(t, what: str, f32: bool = True) -> int:
    """TQ_* type of a tensor of rows."""
    code = _t().row_types.get(t.dtype, -1)
    if code < 0 or (code == TQ_F32 and not f32):
        raise ValueError(f"{what}: rows of {t.dtype} are not taken")
    return code


def _stream_here(stream, device: int, *tensors) -> int:
    """The stream's handle.  The call runs on the current device, where every tensor has to be."""
    if device < 0 or device != _t().current():
        raise ValueError("the cache is not on the current CUDA device")
    for t in tensors:
        if t is not None and t.get_device() != device:
            raise ValueError("tensors are on different devices")
    return _T.raw_stream(device) if stream is None else stream.cuda_stream


def _made_on(stream, make):
    """What a call allocates for itself is filled and reused in the order of the call's stream."""
    if stream is None:
        return make()
    with _torch().cuda.stream(stream):
        return make()


def _ints(t, dtype, shape, what: str):
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{what}: a contiguous {dtype} tensor of shape {tuple(shape)} is expected")


def _row_stride(t, shape, what: str) -> int:
    """Elements between rows of t [n][heads][dim] whose rows are contiguous."""
    if t.shape != shape:
        raise ValueError(f"{what}: shape {tuple(shape)} is expected, not {tuple(t.shape)}")
    if t.is_contiguous():
        return shape[1] * shape[2]
    s0, s1, s2 = t.stride()
    if (s2 != 1 and shape[2] > 1) or (s1 != shape[2] and shape[1] > 1):
        raise ValueError(f"{what}: a row's heads have to be contiguous")
    return s0 if shape[0] > 1 else shape[1] * shape[2]


def _row_width(head_dim: int) -> int:
    return 64 if head_dim <= 64 else 128 if head_dim <= 128 else 256


class Paged4Cache:
    """Planes of one paged 4-bit cache (K or V): codes [n_pages][n_kv_heads][page_size][D / 2] and
    scales (scale, offset) [n_pages][n_kv_heads][page_size][2], D = head_dim rounded up to 64, 128 or 256."""

    def __init__(self, n_kv_heads: int, head_dim: int, page_size: int, n_pages: int, device="cuda", _planes=None):
        torch = _torch()
        _lib.tq_paged4_plane_bytes(n_kv_heads, head_dim, page_size, n_pages)      # refuses what the library does
        self.n_kv_heads, self.head_dim, self.page_size, self.n_pages = n_kv_heads, head_dim, page_size, n_pages
        shape = (n_pages, n_kv_heads, page_size)
        if _planes is None:
            self.codes = torch.zeros((*shape, _row_width(head_dim) // 2), dtype=torch.uint8, device=device)
            self.scales = torch.zeros((*shape, 2), dtype=torch.float16, device=device)
        else:
            self.codes, self.scales = _planes
            _ints(self.codes, torch.uint8, (*shape, _row_width(head_dim) // 2), "codes")
            _ints(self.scales, torch.float16, (*shape, 2), "scales")
            _need(self.codes.device == self.scales.device, "tensors are on different devices")
        self.device = self.codes.device
        self.index = self.codes.get_device()
        self.c = tq_paged4(n_kv_heads, head_dim, page_size, n_pages, self.codes.data_ptr(), self.scales.data_ptr())
        self.ref = C.byref(self.c)

    @classmethod
    def from_planes(cls, codes, scales, head_dim: int):
        """A cache over planes that exist already."""
        n_pages, heads, page = codes.shape[:3]
        return cls(heads, head_dim, page, n_pages, _planes=(codes, scales))


class PagePlan:
    """What page_plan fills: ``seq_len``, ``free_count``, ``q_start``, ``page_start``, ``slots``, ``positions``
    (tq_page_plan in include/tq.h) for n_seq sequences and at most n_rows new cells."""

    def __init__(self, n_seq: int, n_rows: int, device="cuda"):
        torch = _torch()
        i32 = lambda n: torch.zeros((n,), dtype=torch.int32, device=device)  # noqa: E731
        self.n_seq, self.n_rows = n_seq, n_rows
        self.seq_len, self.free_count = i32(n_seq), i32(1)
        self.q_start, self.page_start = i32(n_seq + 1), i32(n_seq + 1)
        self.slots = torch.full((n_rows,), -1, dtype=torch.int64, device=device)
        self.positions = i32(n_rows)
        self.index = self.slots.get_device()
        self._len, self._count = self.seq_len.data_ptr(), self.free_count.data_ptr()
        self._out = (self.q_start.data_ptr(), self.page_start.data_ptr(), self.slots.data_ptr(),
                     self.positions.data_ptr())


def page_plan(seq_len, n_new, page_size: int, block_table, free_pages, free_count, plan: PagePlan | None = None,
              n_rows: int | None = None, in_place: bool = False, dev_status=None, stream=None) -> PagePlan:
    """Pages, slots and positions of a step's new cells (tq_page_plan).  The block table and the free list are
    updated; lengths and the free count go to ``plan``, or with ``in_place`` to seq_len and free_count themselves."""
    n_seq, i32 = seq_len.shape[0], _t().int32
    if plan is None:
        _need(n_rows is not None, "page_plan needs a plan or n_rows")
        plan = _made_on(stream, lambda: PagePlan(n_seq, n_rows, seq_len.device))
    _need(plan.n_seq == n_seq, "the plan is for another number of sequences")
    _need(block_table.dim() == 2 and free_pages.dim() == 1, "block_table: [n_seq][max_pages], free_pages: [capacity]")
    width, capacity = block_table.shape[1], free_pages.shape[0]
    _ints(seq_len, i32, (n_seq,), "seq_len")
    _ints(n_new, i32, (n_seq,), "n_new")
    _ints(block_table, i32, (n_seq, width), "block_table")
    _ints(free_pages, i32, (capacity,), "free_pages")
    _ints(free_count, i32, (1,), "free_count")
    status = None
    if dev_status is not None:
        _ints(dev_status, i32, (1,), "dev_status")
        status = dev_status.data_ptr()
    stream = _stream_here(stream, plan.index, seq_len, n_new, block_table, free_pages, free_count, dev_status)
    len_p, count_p = seq_len.data_ptr(), free_count.data_ptr()
    st = _lib.tq_page_plan(len_p, n_new.data_ptr(), n_seq, page_size, block_table.data_ptr(), width,
                           free_pages.data_ptr(), capacity, count_p, len_p if in_place else plan._len,
                           count_p if in_place else plan._count, *plan._out, plan.n_rows, status, stream)
    if st:
        _lib.check("tq_page_plan", st)
    return plan


def paged4_set_rows(kc: Paged4Cache, vc: Paged4Cache, k_src, v_src, slots, dev_status=None, stream=None):
    """Quantise rows k_src, v_src [n][n_kv_heads][head_dim] (rows may be strided) into cells ``slots``
    (device int64 [n]; -1: not stored)."""
    n = slots.shape[0]
    t = _row_type(k_src, "k_src")
    _need(v_src.dtype is k_src.dtype, "k_src and v_src have different types")
    status = _rows_status(slots, n, dev_status)
    ks = _row_stride(k_src, (n, kc.n_kv_heads, kc.head_dim), "k_src")
    vs = _row_stride(v_src, (n, vc.n_kv_heads, vc.head_dim), "v_src")
    stream = _stream_here(stream, kc.index, vc.codes, k_src, v_src, slots, dev_status)
    st = _lib.tq_paged4_set_rows(kc.ref, vc.ref, k_src.data_ptr(), ks, v_src.data_ptr(), vs, t, slots.data_ptr(), n,
                                 status, stream)
    if st:
        _lib.check("tq_paged4_set_rows", st)


def _rows_status(slots, n, dev_status):
    _ints(slots, _T.int64, (n,), "slots")
    if dev_status is None:
        return None
    _ints(dev_status, _T.int32, (1,), "dev_status")
    return dev_status.data_ptr()


def paged4_get_rows(kc: Paged4Cache, vc: Paged4Cache, slots, dtype=None, k_out=None, v_out=None, dev_status=None,
                    stream=None):
    """The values that cells ``slots`` stand for: (k, v) [n][n_kv_heads][head_dim] of ``dtype`` (default float16),
    or in k_out and v_out (rows may be strided).  Rows whose slot is -1 stay as they were (new outputs: zeros)."""
    n = slots.shape[0]
    if k_out is None or v_out is None:
        dtype = dtype or (k_out if k_out is not None else v_out if v_out is not None else None) or _t().float16
        dtype = getattr(dtype, "dtype", dtype)
        if k_out is None:
            k_out = _made_on(stream, lambda: _t().zeros((n, kc.n_kv_heads, kc.head_dim), dtype=dtype,
                                                        device=slots.device))
        if v_out is None:
            v_out = _made_on(stream, lambda: _t().zeros((n, vc.n_kv_heads, vc.head_dim), dtype=dtype,
                                                        device=slots.device))
    t = _row_type(k_out, "k_out")
    _need(v_out.dtype is k_out.dtype and (dtype is None or dtype is k_out.dtype), "k_out, v_out and dtype differ")
    status = _rows_status(slots, n, dev_status)
    ks = _row_stride(k_out, (n, kc.n_kv_heads, kc.head_dim), "k_out")
    vs = _row_stride(v_out, (n, vc.n_kv_heads, vc.head_dim), "v_out")
    stream = _stream_here(stream, kc.index, vc.codes, k_out, v_out, slots, dev_status)
    st = _lib.tq_paged4_get_rows(kc.ref, vc.ref, k_out.data_ptr(), ks, v_out.data_ptr(), vs, t, slots.data_ptr(), n,
                                 status, stream)
    if st:
        _lib.check("tq_paged4_get_rows", st)
    return k_out, v_out


def paged4_decode_workspace(kc: Paged4Cache, vc: Paged4Cache, n_heads: int, n_seq: int) -> int:
    """Bytes of workspace of paged4_decode and, where K has two heads per V head, paged4_diff_decode."""
    return _lib.tq_paged4_decode_workspace(kc.ref, vc.ref, n_heads, n_seq)


def paged4_prefill_workspace(kc: Paged4Cache, vc: Paged4Cache, n_heads: int, n_seq: int, n_rows: int,
                             max_len: int) -> int:
    """Bytes of workspace of paged4_prefill and, where K has two heads per V head, paged4_diff_prefill: it serves every
    call of at most n_rows rows."""
    return _lib.tq_paged4_prefill_workspace(kc.ref, vc.ref, n_heads, n_seq, n_rows, max_len)


def _paged4_ws(nbytes: int, device):
    """A workspace for one call: what has to be zero is, the partial results' room is left as it comes."""
    ws = _T.empty(max(nbytes, _lib.PAGED4_WORKSPACE_HEAD), dtype=_T.uint8, device=device)
    ws[:_lib.PAGED4_WORKSPACE_HEAD].zero_()
    return ws


def _paged4_args(kc, vc, block_table, seq_len, q, maps, out, ws, stream, *extra):
    """Checks shared by the attention calls -> (n_seq, max_pages, q type, q stride, output heads, out, stream)."""
    t = _row_type(q, "q", f32=False)
    if ws is not None and (ws.element_size() != 1 or not ws.is_contiguous()):
        raise ValueError("ws: a contiguous tensor of bytes is expected")
    if block_table.dim() != 2 or q.dim() != 3 or q.shape[1] % maps:
        raise ValueError("block_table: [n_seq][max_pages], q: [rows][heads][head_dim]")
    n_seq, max_pages = block_table.shape
    rows, heads, _ = q.shape
    _ints(block_table, _T.int32, (n_seq, max_pages), "block_table")
    _ints(seq_len, _T.int32, (n_seq,), "seq_len")
    stride = _row_stride(q, (rows, heads, kc.head_dim), "q")
    heads //= maps
    if out is None:
        out = _made_on(stream, lambda: _T.empty((rows, heads, vc.head_dim), dtype=q.dtype, device=q.device))
    else:
        _ints(out, q.dtype, (rows, heads, vc.head_dim), "out")
    return n_seq, max_pages, t, stride, heads, out, _stream_here(stream, kc.index, vc.codes, block_table, seq_len, q,
                                                                 out, ws, *extra)


def _diff_args(vc, heads, lam, norm_weight):
    _ints(lam, _T.float32, (heads,), "lam")
    if norm_weight is None:
        return lam.data_ptr(), None
    _ints(norm_weight, _T.float32, (vc.head_dim,), "norm_weight")
    return lam.data_ptr(), norm_weight.data_ptr()


def paged4_decode(kc: Paged4Cache, vc: Paged4Cache, block_table, seq_len, q, scale: float | None = None, out=None,
                  ws=None, stream=None):
    """One query row per sequence: q [n_seq][n_q_heads][Dk] (float16 or bfloat16, rows may be strided) over the
    seq_len[s] cells (device int32) of block_table[s] -> [n_seq][n_q_heads][Dv] of q's type."""
    n_seq, max_pages, t, stride, heads, out, handle = _paged4_args(kc, vc, block_table, seq_len, q, 1, out, ws, stream)
    _need(q.shape[0] == n_seq, "q: one row per sequence")
    scale = 1.0 / math.sqrt(kc.head_dim) if scale is None else scale
    if ws is None:
        ws = _made_on(stream, lambda: _paged4_ws(paged4_decode_workspace(kc, vc, heads, n_seq), q.device))
    st = _lib.tq_paged4_decode(kc.ref, vc.ref, block_table.data_ptr(), max_pages, seq_len.data_ptr(), n_seq,
                               q.data_ptr(), t, stride, heads, scale, out.data_ptr(), ws.data_ptr(), ws.numel(),
                               handle)
    if st:
        _lib.check("tq_paged4_decode", st)
    return out


def paged4_prefill(kc: Paged4Cache, vc: Paged4Cache, block_table, seq_len, q, q_start, scale: float | None = None,
                   causal: bool = True, max_rows: int = 0, max_len: int | None = None, out=None, ws=None,
                   stream=None):
    """Several query rows per sequence: rows q_start[s] .. q_start[s + 1] - 1 (device int32 [n_seq + 1]) of q
    [n_rows][n_q_heads][Dk] are the last cells of sequence s.  max_rows and max_len (host): the most rows and cells
    of one sequence, where known; they only choose the kernel.  A workspace for the call is what
    paged4_prefill_workspace gives for at least as many rows."""
    n_seq, max_pages, t, stride, heads, out, handle = _paged4_args(kc, vc, block_table, seq_len, q, 1, out, ws, stream,
                                                                   q_start)
    _ints(q_start, _T.int32, (n_seq + 1,), "q_start")
    scale = 1.0 / math.sqrt(kc.head_dim) if scale is None else scale
    n_rows, max_len = q.shape[0], max_len or max_pages * kc.page_size
    if ws is None:
        ws = _made_on(stream, lambda: _paged4_ws(paged4_prefill_workspace(kc, vc, heads, n_seq, n_rows, max_len), q.device))
    st = _lib.tq_paged4_prefill(kc.ref, vc.ref, block_table.data_ptr(), max_pages, seq_len.data_ptr(),
                                q_start.data_ptr(), n_seq, q.data_ptr(), t, stride, n_rows, heads, max_rows, max_len,
                                scale, int(causal), out.data_ptr(), ws.data_ptr(), ws.numel(), handle)
    if st:
        _lib.check("tq_paged4_prefill", st)
    return out


def paged4_diff_decode(kc: Paged4Cache, vc: Paged4Cache, block_table, seq_len, q, lam, scale: float | None = None,
                       norm_weight=None, eps: float = 1e-5, out_scale: float = 1.0, out=None, ws=None, stream=None):
    """Differential attention, one query row per sequence: q [n_seq][2 n_heads][Dk], K with two heads per V head,
    lam (device float32 [n_heads]) the weights of the second map; optional RMS norm over each head's output."""
    n_seq, max_pages, t, stride, heads, out, handle = _paged4_args(kc, vc, block_table, seq_len, q, 2, out, ws, stream,
                                                                   lam, norm_weight)
    _need(q.shape[0] == n_seq, "q: one row per sequence")
    lam_p, norm_p = _diff_args(vc, heads, lam, norm_weight)
    scale = 1.0 / math.sqrt(kc.head_dim) if scale is None else scale
    if ws is None:
        ws = _made_on(stream, lambda: _paged4_ws(paged4_decode_workspace(kc, vc, heads, n_seq), q.device))
    st = _lib.tq_paged4_diff_decode(kc.ref, vc.ref, block_table.data_ptr(), max_pages, seq_len.data_ptr(), n_seq,
                                    q.data_ptr(), t, stride, heads, lam_p, norm_p, eps, out_scale, scale,
                                    out.data_ptr(), ws.data_ptr(), ws.numel(), handle)
    if st:
        _lib.check("tq_paged4_diff_decode", st)
    return out


def paged4_diff_prefill(kc: Paged4Cache, vc: Paged4Cache, block_table, seq_len, q, q_start, lam,
                        scale: float | None = None, norm_weight=None, eps: float = 1e-5, out_scale: float = 1.0,
                        causal: bool = True, max_rows: int = 0, max_len: int | None = None, out=None, ws=None,
                        stream=None):
    """Differential attention of several query rows per sequence: rows as paged4_prefill, heads as
    paged4_diff_decode."""
    n_seq, max_pages, t, stride, heads, out, handle = _paged4_args(kc, vc, block_table, seq_len, q, 2, out, ws, stream,
                                                                   q_start, lam, norm_weight)
    _ints(q_start, _T.int32, (n_seq + 1,), "q_start")
    lam_p, norm_p = _diff_args(vc, heads, lam, norm_weight)
    scale = 1.0 / math.sqrt(kc.head_dim) if scale is None else scale
    n_rows, max_len = q.shape[0], max_len or max_pages * kc.page_size
    if ws is None:
        ws = _made_on(stream, lambda: _paged4_ws(paged4_prefill_workspace(kc, vc, heads, n_seq, n_rows, max_len), q.device))
    st = _lib.tq_paged4_diff_prefill(kc.ref, vc.ref, block_table.data_ptr(), max_pages, seq_len.data_ptr(),
                                     q_start.data_ptr(), n_seq, q.data_ptr(), t, stride, n_rows, heads, max_rows,
                                     max_len, lam_p, norm_p, eps, out_scale, scale, int(causal), out.data_ptr(),
                                     ws.data_ptr(), ws.numel(), handle)
    if st:
        _lib.check("tq_paged4_diff_prefill", st)
    return out
