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
                ("head_dim", _I32), ("scale", ctypes.c_double), ("workspace", _P),
                ("workspace_bytes", ctypes.c_size_t)]


# ------------------------------------------------------------------------------ checks
# These calls are a few microseconds on the GPU at their smallest, so their checks read each
# tensor's properties once and format messages only when one fails.
_INT, _BF16, _FP32, _U8 = torch.int32, torch.bfloat16, torch.float32, torch.uint8


def _device(t, what: str) -> int:
    """Index of the CUDA device of a call's first tensor."""
    dev = t.get_device() if isinstance(t, torch.Tensor) else -1
    if dev < 0:
        raise ValueError(f"{what} must be a CUDA tensor")
    return dev


def _array(t, what: str, shape, dev: int, dtype=_INT) -> int:
    """Address of a contiguous tensor of this type and shape on CUDA device `dev`."""
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.shape != shape \
            or t.get_device() != dev or not t.is_contiguous():
        got = f"{t.dtype}, shape {tuple(t.shape)} on {t.device}" if isinstance(t, torch.Tensor) else type(t)
        raise ValueError(f"{what} must be a contiguous tensor of {dtype}, shape {tuple(shape)} on cuda:{dev}, "
                         f"not {got}")
    return t.data_ptr()


def _rows(t, what: str, shape, dev: int, dtype):
    """Strides (row, head) of a [rows, heads, D] tensor of this type and shape on CUDA device
    `dev`, whose rows of D must start on 16 bytes."""
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.shape != shape or t.get_device() != dev:
        got = f"{t.dtype}, shape {tuple(t.shape)} on {t.device}" if isinstance(t, torch.Tensor) else type(t)
        raise ValueError(f"{what} must be a tensor of {dtype}, shape {tuple(shape)} on cuda:{dev}, not {got}")
    rows, heads, _ = shape
    row, head, one = t.stride()
    # the stride of a single row or head is never used: torch may give any
    if rows <= 1:
        row = 0
    if heads <= 1:
        head = 0
    whole = 8 if dtype is _BF16 else 4
    if one != 1 or row % whole or head % whole:
        if t.numel() == 0:
            return _Strides(0, 0)
        raise ValueError(f"{what} needs unit element stride and strides of whole 16 bytes")
    return _Strides(row, head)


def _shape(t, what: str, dims: int):
    if not isinstance(t, torch.Tensor) or t.dim() != dims:
        raise ValueError(f"{what} must be a tensor of {dims} dimensions")
    return t.shape


def _flags(flags, dev: int):
    return None if flags is None else _array(flags, "flags", (1,), dev)


def _call(fn, dev: int, stream, *args):
    """fn(*args, stream) with CUDA device `dev` current."""
    if stream is None:
        sp = _rkv._raw_stream(dev) if _rkv._raw_stream is not None else torch.cuda.current_stream(dev).cuda_stream
    else:
        if stream.device.index != dev:
            raise ValueError(f"stream is on {stream.device}, the call's tensors on cuda:{dev}")
        sp = stream.cuda_stream
    if (_rkv._cur_device() if _rkv._cur_device is not None else torch.cuda.current_device()) == dev:
        status = fn(*args, sp)
    else:
        with torch.cuda.device(dev):
            status = fn(*args, sp)
    if status != 0:
        _rkv._check(status)


def _new(shape, dtype, dev: int, stream):
    """A tensor for work on `stream`: from the memory of that stream, so that it is not handed
    on while the work runs."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=dev)


def _scale(scale, d: int) -> float:
    if scale is None:
        return d ** -0.5
    s = float(scale)
    if not (math.isfinite(s) and s > 0):
        raise ValueError("scale must be finite and > 0")
    return s


def _table(block_table, seq_len, dev: int):
    B, M = _shape(block_table, "block_table", 2)
    return _Table(_array(block_table, "block_table", (B, M), dev), _array(seq_len, "seq_len", (B,), dev), B, M)


def _pages(k8, v8, k_scale, v_scale, dev: int):
    shape = _shape(k8, "k8", 4)
    nb, N, P, D = shape
    return _Pages(_array(k8, "k8", shape, dev, _U8), _array(v8, "v8", shape, dev, _U8),
                  _array(k_scale, "k_scale", (nb, N), dev, _FP32),
                  _array(v_scale, "v_scale", (nb, N), dev, _FP32), N, D, P, nb)


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
    if max_rows < 0:
        raise ValueError("max_rows must be >= 0")
    dev = _device(block_table, "block_table")
    table = _table(block_table, seq_len, dev)
    B = table.batch
    num = _shape(free_blocks, "free_blocks", 1)[0]
    new_p = _array(new_tokens, "new_tokens", (B,), dev)
    free_p = _array(free_blocks, "free_blocks", (num,), dev)
    nf_p = _array(n_free, "n_free", (1,), dev)
    lo_p = table.seq_len if seq_len_out is None else _array(seq_len_out, "seq_len_out", (B,), dev)
    no_p = nf_p if n_free_out is None else _array(n_free_out, "n_free_out", (1,), dev)
    f_p = _flags(flags, dev)
    # one allocation: the offsets, then the three row maps
    buf = _new(B + 1 + 3 * max_rows, _INT, dev, stream)
    p = buf.data_ptr()
    r0 = p + 4 * (B + 1)
    _call(_rkv.lib().rkv_page_plan, dev, stream, ctypes.byref(table), new_p, free_p, nf_p, num, block_tokens,
          max_rows, lo_p, no_p, p, r0, r0 + 4 * max_rows, r0 + 8 * max_rows, f_p)
    return PagePlan(*buf.split_with_sizes((B + 1, max_rows, max_rows, max_rows)))


def page_release(finished, seq_len, block_table, free_blocks, n_free, block_tokens: int, flags=None,
                 stream=None):
    """Put the pages of the sequences b with finished[b] != 0 (int32 [batch]) back on the free
    list; their lengths become 0."""
    dev = _device(block_table, "block_table")
    table = _table(block_table, seq_len, dev)
    num = _shape(free_blocks, "free_blocks", 1)[0]
    _call(_rkv.lib().rkv_page_release, dev, stream, ctypes.byref(table),
          _array(finished, "finished", (table.batch,), dev), _array(free_blocks, "free_blocks", (num,), dev),
          _array(n_free, "n_free", (1,), dev), num, block_tokens, _flags(flags, dev))


def page_append(k, v, k8, v8, k_scale, v_scale, block_table, seq_len, cu_rows, flags=None, stream=None):
    """Store packed rows k, v ([rows, N, D], both bf16 or both fp32, strided rows allowed) in
    their pages: rows cu_rows[b] .. cu_rows[b + 1] - 1 are the last positions of sequence b,
    seq_len the lengths with them.  k8, v8 [num_blocks, N, block_tokens, D] uint8 (E4M3 codes)
    and k_scale, v_scale [num_blocks, N] fp32 are updated."""
    dev = _device(k8, "k8")
    pages = _pages(k8, v8, k_scale, v_scale, dev)
    n = _shape(k, "k", 3)[0]
    dtype = _FP32 if k.dtype is _FP32 else _BF16
    shape = (n, pages.n_kv_heads, pages.head_dim)
    ks, vs = _rows(k, "k", shape, dev, dtype), _rows(v, "v", shape, dev, dtype)
    table = _table(block_table, seq_len, dev)
    _call(_rkv.lib().rkv_page_append, dev, stream, ctypes.byref(pages), ctypes.byref(table), k.data_ptr(), ks,
          v.data_ptr(), vs, _rkv.RKV_F32 if dtype is _FP32 else _rkv.RKV_BF16, n,
          _array(cu_rows, "cu_rows", (table.batch + 1,), dev), _flags(flags, dev))


_workspace_bytes: dict = {}          # (query heads per key/value head, head_dim) -> bytes


def page_attention(q, k8, v8, k_scale, v_scale, block_table, seq_len, scale=None, out=None, lse=None,
                   flags=None, stream=None):
    """One query row a sequence, q [batch, n_q_heads, D] bf16, against its stored positions:
    softmax(scale q K^T) V as [batch, n_q_heads, D] bf16 (`out`, if given).  scale defaults to
    1 / sqrt(D); lse, an fp32 [batch, n_q_heads], receives the log-sum-exp."""
    dev = _device(k8, "k8")
    pages = _pages(k8, v8, k_scale, v_scale, dev)
    table = _table(block_table, seq_len, dev)
    B, Hq, D = shape = _shape(q, "q", 3)
    if B != table.batch or D != pages.head_dim:
        raise ValueError(f"q must be [{table.batch}, n_q_heads, {pages.head_dim}]")
    qs = _rows(q, "q", shape, dev, _BF16)
    lse_p = None if lse is None else _array(lse, "lse", (B, Hq), dev, _FP32)
    sc = _scale(scale, D)
    lib = _rkv.lib()
    key = (Hq / pages.n_kv_heads if pages.n_kv_heads else 0, D)
    nbytes = _workspace_bytes.get(key)
    if nbytes is None:
        got = ctypes.c_size_t()
        _rkv._check(lib.rkv_page_attention_workspace(ctypes.byref(pages), ctypes.byref(table), Hq,
                                                     ctypes.byref(got)))
        nbytes = _workspace_bytes[key] = got.value
    if out is None:
        out = _new(shape, _BF16, dev, stream)
        out_p = out.data_ptr()
    else:
        out_p = _array(out, "out", shape, dev, _BF16)
    ws = _new(nbytes, _U8, dev, stream)
    _call(lib.rkv_page_attention, dev, stream, ctypes.byref(pages), ctypes.byref(table), q.data_ptr(), qs, Hq, sc,
          out_p, lse_p, ws.data_ptr(), nbytes, _flags(flags, dev))
    return out


def prompt_attention(q, k, v, cu_q, cu_k=None, scale=None, out=None, lse=None, flags=None, stream=None):
    """Causal attention of packed prompts: q [total_q, n_q_heads, D], k and v [total_k, N, D]
    bf16 (strided rows allowed), sequence b's rows cu_q[b] .. cu_q[b + 1] - 1 of q and
    cu_k[b] .. cu_k[b + 1] - 1 of k and v (cu_k defaults to cu_q); its queries are its last
    positions.  Returns [total_q, n_q_heads, D] bf16 (`out`, if given; rows past cu_q[-1] are
    not written).  lse, an fp32 [total_q, n_q_heads], receives the log-sum-exp."""
    dev = _device(q, "q")
    Tq, Hq, D = q_shape = _shape(q, "q", 3)
    Tk, N, _ = _shape(k, "k", 3)
    qs = _rows(q, "q", q_shape, dev, _BF16)
    ks, vs = _rows(k, "k", (Tk, N, D), dev, _BF16), _rows(v, "v", (Tk, N, D), dev, _BF16)
    n_cu = _shape(cu_q, "cu_q", 1)
    cq = _array(cu_q, "cu_q", n_cu, dev)
    ck = cq if cu_k is None else _array(cu_k, "cu_k", n_cu, dev)
    lse_p = None if lse is None else _array(lse, "lse", (Tq, Hq), dev, _FP32)
    sc = _scale(scale, D)
    if out is None:
        out = _new(q_shape, _BF16, dev, stream)
        os_ = _Strides(Hq * D, D)
    else:
        os_ = _rows(out, "out", q_shape, dev, _BF16)
    a = _Prompt(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse_p, qs, ks, vs, os_, cq, ck,
                n_cu[0] - 1, Tq, Tk, Hq, N, D, sc, None, 0)
    lib, nbytes = _rkv.lib(), ctypes.c_size_t()
    _rkv._check(lib.rkv_prompt_attention_workspace(ctypes.byref(a), ctypes.byref(nbytes)))
    ws = None
    if nbytes.value:
        ws = _new(nbytes.value, _U8, dev, stream)
        a.workspace, a.workspace_bytes = ws.data_ptr(), nbytes.value
    _call(lib.rkv_prompt_attention, dev, stream, ctypes.byref(a), _flags(flags, dev))
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
