"""Full-attention layers: a step's pages planned on the GPU, the attention of packed
prompts, K/V stored in 8-bit pages and the decode attention that reads them.

Argument marshalling for the ``rkv_page_*`` and ``rkv_prompt_attention`` entry points of
``include/rkv.h``, which give each operator's formulas and limits.  The functions take plain
CUDA tensors; ``PageTable`` and ``PagedCache`` hold the ones that a serving loop keeps:

    table = PageTable(batch, max_blocks, num_blocks, block_tokens)
    caches = [PagedCache(n_kv_heads, head_dim, num_blocks, block_tokens) for _ in layers]
    plan = table.plan(new_tokens, max_rows)          # once a step
    for cache in caches:                             # in each layer
        o = prompt_attention(q, k, v, plan.cu_rows)  # prompts, from their raw K/V
        cache.append(k, v, table, plan)
        o = cache.attend(q, table)                   # decode: one query a sequence
    table.release(finished)

Every tensor of a call must lie on one device, which need not be the current one.  Work goes
to ``stream`` (a ``torch.cuda.Stream`` of that device), or to the device's current stream;
tensors made on another stream must be ready there, as for any torch operation.
"""
from __future__ import annotations

import ctypes
import math
from dataclasses import dataclass

import torch

import residual_kv_cache_gb300 as _rkv

__all__ = ["PagedCache", "PagePlan", "PageTable", "page_append", "page_attention", "page_plan",
           "page_release", "prompt_attention"]

_I32, _I64, _P = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p
_Strides = _I64 * 2


class _Pages(ctypes.Structure):
    _fields_ = [("k", _P), ("v", _P), ("k_scale", _P), ("v_scale", _P), ("n_kv_heads", _I32),
                ("head_dim", _I32), ("block_tokens", _I32), ("num_blocks", _I32)]


class _Table(ctypes.Structure):
    _fields_ = [("block_table", _P), ("seq_len", _P), ("batch", _I32), ("max_blocks", _I32)]


class _Prompt(ctypes.Structure):
    _fields_ = [("q", _P), ("k", _P), ("v", _P), ("out", _P), ("lse", _P),
                ("q_strides", _Strides), ("k_strides", _Strides), ("v_strides", _Strides),
                ("out_strides", _Strides), ("cu_q", _P), ("cu_k", _P), ("batch", _I32),
                ("total_q", _I32), ("total_k", _I32), ("n_q_heads", _I32), ("n_kv_heads", _I32),
                ("head_dim", _I32), ("scale", ctypes.c_double)]


# ------------------------------------------------------------------------------ checks
def _array(t, what: str, shape, device, dtype=torch.int32):
    """A contiguous CUDA tensor of this shape (None: any size of that dimension) and type."""
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or t.dim() != len(shape) \
            or any(w is not None and s != w for s, w in zip(t.shape, shape)) \
            or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous CUDA tensor of {dtype}, shape {tuple(shape)}")
    if device is not None and t.device != device:
        raise ValueError(f"{what} is on {t.device}, the call's other tensors on {device}")
    return t.data_ptr()


def _rows(t, what: str, shape, device, dtypes):
    """A [rows, heads, D] CUDA tensor whose rows of D lie 16-byte aligned: its strides."""
    if not isinstance(t, torch.Tensor) or t.dtype not in dtypes or t.dim() != 3 \
            or any(w is not None and s != w for s, w in zip(t.shape, shape)) or not t.is_cuda:
        raise ValueError(f"{what} must be a CUDA tensor of {' or '.join(map(str, dtypes))}, "
                         f"shape {tuple(shape)}")
    if device is not None and t.device != device:
        raise ValueError(f"{what} is on {t.device}, the call's other tensors on {device}")
    if t.numel() == 0:
        return _Strides(0, 0)
    row, head, one = t.stride()
    # the stride of a single row or head is never used: torch may give any
    row, head = row if t.shape[0] > 1 else 0, head if t.shape[1] > 1 else 0
    if (one != 1 and t.shape[2] > 1) or row * t.element_size() % 16 or head * t.element_size() % 16:
        raise ValueError(f"{what} needs unit element stride and strides of whole 16 bytes")
    return _Strides(row, head)


def _flags(flags, device):
    return None if flags is None else _array(flags, "flags", (1,), device)


class _On:
    """Makes `device` current for the call (the library launches on the current device) and
    gives the raw stream to launch on."""
    __slots__ = ("guard", "stream")

    def __init__(self, device, stream):
        if stream is not None and stream.device != device:
            raise ValueError(f"stream is on {stream.device}, the call's tensors on {device}")
        self.guard = None if _cur_device() == device.index else torch.cuda.device(device)
        self.stream = stream

    def __enter__(self):
        if self.guard is not None:
            self.guard.__enter__()
        return _rkv._stream_ptr(self.stream)

    def __exit__(self, *exc):
        if self.guard is not None:
            self.guard.__exit__(*exc)


def _cur_device() -> int:
    return _rkv._cur_device() if _rkv._cur_device is not None else torch.cuda.current_device()


def _new(shape, dtype, device, stream):
    """A tensor for work on `stream`: from the memory of that stream, so that it is not handed
    on while the work runs."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _scale(scale, d: int) -> float:
    s = 1.0 / math.sqrt(d) if scale is None else float(scale)
    if not (math.isfinite(s) and s > 0):
        raise ValueError("scale must be finite and > 0")
    return s


def _table_struct(block_table, seq_len, device):
    bt = _array(block_table, "block_table", (None, None), device)
    B, M = block_table.shape
    return _Table(bt, _array(seq_len, "seq_len", (B,), block_table.device), B, M)


def _pages_struct(k8, v8, k_scale, v_scale):
    kp = _array(k8, "k8", (None, None, None, None), None, torch.uint8)
    nb, N, P, D = k8.shape
    dev = k8.device
    return _Pages(kp, _array(v8, "v8", (nb, N, P, D), dev, torch.uint8),
                  _array(k_scale, "k_scale", (nb, N), dev, torch.float32),
                  _array(v_scale, "v_scale", (nb, N), dev, torch.float32), N, D, P, nb)


# ---------------------------------------------------------------------------- operators
@dataclass
class PagePlan:
    """Where a step's packed rows go: sequence b's are cu_rows[b] .. cu_rows[b + 1] - 1; of
    each row its sequence, position and slot (page * block_tokens + row in the page), -1 past
    the total."""
    cu_rows: torch.Tensor
    row_seq: torch.Tensor
    row_pos: torch.Tensor
    row_slot: torch.Tensor


def page_plan(new_tokens, seq_len, block_table, free_blocks, n_free, block_tokens: int, max_rows: int,
              seq_len_out=None, n_free_out=None, flags=None, stream=None) -> PagePlan:
    """Take the pages that a step's new positions need and map its packed rows to them.

    All int32: new_tokens, seq_len [batch], block_table [batch, max_blocks] (receives the new
    pages), free_blocks [num_blocks], n_free [1].  The lengths and the free count after the
    step go to seq_len_out and n_free_out, by default to seq_len and n_free themselves.
    A step that does not fit changes nothing and has no rows (FLAG_NO_SPACE in `flags`)."""
    dev = getattr(block_table, "device", None)
    if max_rows < 0:
        raise ValueError("max_rows must be >= 0")
    table = _table_struct(block_table, seq_len, None)
    B = table.batch
    new_p = _array(new_tokens, "new_tokens", (B,), dev)
    free_p = _array(free_blocks, "free_blocks", (None,), dev)
    nf_p = _array(n_free, "n_free", (1,), dev)
    lo_p = table.seq_len if seq_len_out is None else _array(seq_len_out, "seq_len_out", (B,), dev)
    no_p = nf_p if n_free_out is None else _array(n_free_out, "n_free_out", (1,), dev)
    f_p = _flags(flags, dev)
    with _On(dev, stream) as s:
        # one allocation: the offsets, then the three row maps
        buf = _new(B + 1 + 3 * max_rows, torch.int32, dev, stream)
        cu, seq, pos, slot = buf.split_with_sizes((B + 1, max_rows, max_rows, max_rows))
        p = buf.data_ptr()
        r0 = p + 4 * (B + 1)
        _rkv._check(_rkv.lib().rkv_page_plan(
            ctypes.byref(table), new_p, free_p, nf_p, free_blocks.shape[0], block_tokens, max_rows,
            lo_p, no_p, p, r0, r0 + 4 * max_rows, r0 + 8 * max_rows, f_p, s))
    return PagePlan(cu, seq, pos, slot)


def page_release(finished, seq_len, block_table, free_blocks, n_free, block_tokens: int, flags=None,
                 stream=None):
    """Put the pages of the sequences b with finished[b] != 0 (int32 [batch]) back on the free
    list; their lengths become 0."""
    table = _table_struct(block_table, seq_len, None)
    dev = block_table.device
    fin_p = _array(finished, "finished", (table.batch,), dev)
    free_p = _array(free_blocks, "free_blocks", (None,), dev)
    nf_p = _array(n_free, "n_free", (1,), dev)
    f_p = _flags(flags, dev)
    with _On(dev, stream) as s:
        _rkv._check(_rkv.lib().rkv_page_release(ctypes.byref(table), fin_p, free_p, nf_p,
                                                free_blocks.shape[0], block_tokens, f_p, s))


def page_append(k, v, k8, v8, k_scale, v_scale, block_table, seq_len, cu_rows, flags=None, stream=None):
    """Store packed rows k, v ([rows, N, D], both bf16 or both fp32, strided rows allowed) in
    their pages: rows cu_rows[b] .. cu_rows[b + 1] - 1 are the last positions of sequence b,
    seq_len the lengths with them.  k8, v8 [num_blocks, N, block_tokens, D] uint8 (E4M3 codes)
    and k_scale, v_scale [num_blocks, N] fp32 are updated."""
    pages = _pages_struct(k8, v8, k_scale, v_scale)
    dev = k8.device
    ks = _rows(k, "k", (None, pages.n_kv_heads, pages.head_dim), dev, (torch.bfloat16, torch.float32))
    vs = _rows(v, "v", tuple(k.shape), dev, (k.dtype,))
    table = _table_struct(block_table, seq_len, dev)
    cu_p = _array(cu_rows, "cu_rows", (table.batch + 1,), dev)
    f_p = _flags(flags, dev)
    with _On(dev, stream) as s:
        _rkv._check(_rkv.lib().rkv_page_append(
            ctypes.byref(pages), ctypes.byref(table), k.data_ptr(), ks, v.data_ptr(), vs,
            _rkv._dtype_code(k.dtype), k.shape[0], cu_p, f_p, s))


def page_attention(q, k8, v8, k_scale, v_scale, block_table, seq_len, scale=None, out=None, lse=None,
                   flags=None, stream=None):
    """One query row a sequence, q [batch, n_q_heads, D] bf16, against its stored positions:
    softmax(scale q K^T) V as [batch, n_q_heads, D] bf16 (`out`, if given).  scale defaults to
    1 / sqrt(D); lse, an fp32 [batch, n_q_heads], receives the log-sum-exp."""
    pages = _pages_struct(k8, v8, k_scale, v_scale)
    dev = k8.device
    table = _table_struct(block_table, seq_len, dev)
    qs = _rows(q, "q", (table.batch, None, pages.head_dim), dev, (torch.bfloat16,))
    B, Hq, D = q.shape
    lse_p = None if lse is None else _array(lse, "lse", (B, Hq), dev, torch.float32)
    f_p = _flags(flags, dev)
    sc = _scale(scale, D)
    lib, nbytes = _rkv.lib(), ctypes.c_size_t()
    _rkv._check(lib.rkv_page_attention_workspace(ctypes.byref(pages), ctypes.byref(table), Hq,
                                                 ctypes.byref(nbytes)))
    with _On(dev, stream) as s:
        if out is None:
            out = _new((B, Hq, D), torch.bfloat16, dev, stream)
        out_p = _array(out, "out", (B, Hq, D), dev, torch.bfloat16)
        ws = _new(nbytes.value, torch.uint8, dev, stream)
        _rkv._check(lib.rkv_page_attention(
            ctypes.byref(pages), ctypes.byref(table), q.data_ptr(), qs, Hq, sc, out_p, lse_p,
            ws.data_ptr(), nbytes.value, f_p, s))
    return out


def prompt_attention(q, k, v, cu_q, cu_k=None, scale=None, out=None, lse=None, flags=None, stream=None):
    """Causal attention of packed prompts: q [total_q, n_q_heads, D], k and v [total_k, N, D]
    bf16 (strided rows allowed), sequence b's rows cu_q[b] .. cu_q[b + 1] - 1 of q and
    cu_k[b] .. cu_k[b + 1] - 1 of k and v (cu_k defaults to cu_q); its queries are its last
    positions.  Returns [total_q, n_q_heads, D] bf16 (`out`, if given; rows past cu_q[-1] are
    not written).  lse, an fp32 [total_q, n_q_heads], receives the log-sum-exp."""
    qs = _rows(q, "q", (None, None, None), None, (torch.bfloat16,))
    dev = q.device
    Tq, Hq, D = q.shape
    ks = _rows(k, "k", (None, None, D), dev, (torch.bfloat16,))
    vs = _rows(v, "v", tuple(k.shape), dev, (torch.bfloat16,))
    cq = _array(cu_q, "cu_q", (None,), dev)
    ck = cq if cu_k is None else _array(cu_k, "cu_k", (cu_q.shape[0],), dev)
    lse_p = None if lse is None else _array(lse, "lse", (Tq, Hq), dev, torch.float32)
    f_p = _flags(flags, dev)
    sc = _scale(scale, D)
    with _On(dev, stream) as s:
        if out is None:
            out = _new((Tq, Hq, D), torch.bfloat16, dev, stream)
        os_ = _rows(out, "out", (Tq, Hq, D), dev, (torch.bfloat16,))
        a = _Prompt(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse_p, qs, ks, vs, os_,
                    cq, ck, cu_q.shape[0] - 1, Tq, k.shape[0], Hq, k.shape[1], D, sc)
        _rkv._check(_rkv.lib().rkv_prompt_attention(ctypes.byref(a), f_p, s))
    return out


class PageTable:
    """The pages of `batch` sequence slots, shared by all layers: block table, lengths, free
    list and a flags word (FLAG_*, ORed by the calls made through this table)."""

    def __init__(self, batch: int, max_blocks: int, num_blocks: int, block_tokens: int = 64, device=None):
        dev = torch.device(device or "cuda")
        self.block_tokens = block_tokens
        self.block_table = torch.full((batch, max_blocks), -1, dtype=torch.int32, device=dev)
        self.seq_len = torch.zeros(batch, dtype=torch.int32, device=dev)
        self.free_blocks = torch.arange(num_blocks - 1, -1, -1, dtype=torch.int32, device=dev)
        self.n_free = torch.full((1,), num_blocks, dtype=torch.int32, device=dev)
        self.flags = torch.zeros(1, dtype=torch.int32, device=dev)

    def plan(self, new_tokens, max_rows: int, stream=None) -> PagePlan:
        """Append new_tokens[b] positions to each sequence (see page_plan)."""
        return page_plan(new_tokens, self.seq_len, self.block_table, self.free_blocks, self.n_free,
                         self.block_tokens, max_rows, flags=self.flags, stream=stream)

    def release(self, finished, stream=None):
        """Give back the pages of the sequences marked in `finished` (int32 [batch])."""
        page_release(finished, self.seq_len, self.block_table, self.free_blocks, self.n_free,
                     self.block_tokens, flags=self.flags, stream=stream)


class PagedCache:
    """One layer's K/V rows in 8-bit pages."""

    def __init__(self, n_kv_heads: int, head_dim: int, num_blocks: int, block_tokens: int = 64, device=None):
        dev = torch.device(device or "cuda")
        shape = (num_blocks, n_kv_heads, block_tokens, head_dim)
        self.k8 = torch.empty(shape, dtype=torch.uint8, device=dev)
        self.v8 = torch.empty(shape, dtype=torch.uint8, device=dev)
        self.k_scale = torch.empty(shape[:2], dtype=torch.float32, device=dev)
        self.v_scale = torch.empty(shape[:2], dtype=torch.float32, device=dev)

    def append(self, k, v, table: PageTable, plan: PagePlan, stream=None):
        """Store the planned step's rows (see page_append)."""
        page_append(k, v, self.k8, self.v8, self.k_scale, self.v_scale, table.block_table,
                    table.seq_len, plan.cu_rows, flags=table.flags, stream=stream)

    def attend(self, q, table: PageTable, scale=None, out=None, lse=None, stream=None):
        """Decode attention, one query a sequence (see page_attention)."""
        return page_attention(q, self.k8, self.v8, self.k_scale, self.v_scale, table.block_table,
                              table.seq_len, scale=scale, out=out, lse=lse, flags=table.flags,
                              stream=stream)
