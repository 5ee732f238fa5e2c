"""Full-attention layers: a step's pages planned on the GPU, queries' and keys' norm and
rotation, the attention of packed prompts, K/V stored in 8-bit pages, the decode attention
that reads them, and pages that several sequences hold.

Argument marshalling for the ``rkv_page_*``, ``rkv_head_norm_rotate`` and
``rkv_prompt_attention`` entry points of ``include/rkv.h``, which give each operator's formulas and limits.  The functions take plain
CUDA tensors; ``PageTable`` and ``PagedCache`` hold the ones that a serving loop keeps:

    table = PageTable(batch, max_blocks, num_blocks, block_tokens)
    caches = [PagedCache(n_kv_heads, head_dim, num_blocks, block_tokens) for _ in layers]
    plan = table.plan(new_tokens, max_rows)          # once a step
    for cache in caches:                             # in each layer
        q, k = head_norm_rotate(q, k, plan.row_pos, freq)
        o = prompt_attention(q, k, v, plan.cu_rows, flags=table.flags)   # prompts, from their raw K/V
        cache.append(k, v, table, plan)
        o = cache.attend(q, table)                   # decode: one query a sequence
    table.release(finished)

Requests that begin alike share the pages of what they have in common:

    table = PageTable(batch, max_blocks, num_blocks, block_tokens, sharing=True)
    copies = table.fork(source, length)              # rows become (prefixes of) other rows
    page_copy(caches, *copies, flags=table.flags)    # the pages that two of them have begun
    k, v, cu_k = cache.gather(table, max_rows, length)     # a prompt's keys with its prefix's
    page_copy(caches, *table.compact(), flags=table.flags)     # all pages to the pool's low end

What a call finds out of range, or has no space for, it leaves out or refuses on the GPU and
notes in ``table.flags`` (FLAG_*), which a program reads where it waits for the GPU anyway: a
copy without ``flags`` leaves no trace of it.

Every tensor of a call must lie on one device, which need not be the current one.  Work goes
to ``stream`` (a ``torch.cuda.Stream`` of that device), or to the device's current stream;
tensors made on another stream must be ready there, as for any torch operation.  Nothing is
differentiable: results carry no gradient.
"""
from __future__ import annotations

import importlib
import math
import os
from typing import NamedTuple

import torch

import residual_kv_cache_gb300 as _rkv

__all__ = ["PageCopies", "PagedCache", "PagePlan", "PageTable", "head_norm_rotate", "page_append",
           "page_attention", "page_compact", "page_copy", "page_fork", "page_gather", "page_plan",
           "page_release", "prompt_attention", "rotation_freq"]

_module = None


def _ext():
    """The compiled binding (csrc/pages_torch.cpp): checks, outputs, workspaces, the calls."""
    global _module
    if _module is None:
        if not os.path.exists(os.path.join(os.path.dirname(os.path.abspath(__file__)), "_pages.so")):
            raise _rkv.RkvLibraryMissing(
                "_pages.so is missing: build it with `python -m residual_kv_cache_gb300.build`")
        _rkv.lib()
        _module = importlib.import_module("residual_kv_cache_gb300._pages")
        _module.set_error(_rkv.RkvError)
    return _module


# ---------------------------------------------------------------------------- operators
class PagePlan(NamedTuple):
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
    return PagePlan(*_ext().page_plan(new_tokens, seq_len, block_table, free_blocks, n_free, block_tokens,
                                      max_rows, seq_len_out, n_free_out, flags, stream))


def page_release(finished, seq_len, block_table, free_blocks, n_free, block_tokens: int, flags=None,
                 stream=None):
    """Put the pages of the sequences b with finished[b] != 0 (int32 [batch]) back on the free
    list; their lengths become 0."""
    _ext().page_release(finished, seq_len, block_table, free_blocks, n_free, block_tokens, flags, stream)


def page_append(k, v, k8, v8, k_scale, v_scale, block_table, seq_len, cu_rows, flags=None, stream=None):
    """Store packed rows k, v ([rows, N, D], both bf16 or both fp32, strided rows allowed) in
    their pages: rows cu_rows[b] .. cu_rows[b + 1] - 1 are the last positions of sequence b,
    seq_len the lengths with them.  k8, v8 [num_blocks, N, block_tokens, D] uint8 (E4M3 codes)
    and k_scale, v_scale [num_blocks, N] fp32 are updated."""
    _ext().page_append(k, v, k8, v8, k_scale, v_scale, block_table, seq_len, cu_rows, flags, stream)


def page_attention(q, k8, v8, k_scale, v_scale, block_table, seq_len, scale=None, out=None, lse=None,
                   flags=None, stream=None):
    """One query row a sequence, q [batch, n_q_heads, D] bf16, against its stored positions:
    softmax(scale q K^T) V as [batch, n_q_heads, D] bf16 (`out`, if given).  scale defaults to
    1 / sqrt(D); lse, an fp32 [batch, n_q_heads], receives the log-sum-exp."""
    return _ext().page_attention(q, k8, v8, k_scale, v_scale, block_table, seq_len, scale, out, lse, flags,
                                 stream)


def prompt_attention(q, k, v, cu_q, cu_k=None, scale=None, out=None, lse=None, flags=None, stream=None):
    """Causal attention of packed prompts: q [total_q, n_q_heads, D], k and v [total_k, N, D]
    bf16 (strided rows allowed), sequence b's rows cu_q[b] .. cu_q[b + 1] - 1 of q and
    cu_k[b] .. cu_k[b + 1] - 1 of k and v (cu_k defaults to cu_q); its queries are its last
    positions.  Returns [total_q, n_q_heads, D] bf16 (`out`, if given; rows past cu_q[-1] are
    not written).  lse, an fp32 [total_q, n_q_heads], receives the log-sum-exp."""
    return _ext().prompt_attention(q, k, v, cu_q, cu_k, scale, out, lse, flags, stream)


def rotation_freq(rotary_dim: int, base: float = 10000.0, device=None):
    """base^(-2 j / rotary_dim) radians a position, j < rotary_dim / 2, as head_norm_rotate takes
    them (float64; the codec's restore rotates K by the same angles)."""
    if rotary_dim < 0 or rotary_dim % 2:
        raise ValueError("rotary_dim must be even and >= 0")
    if not 0 < base < math.inf:
        raise ValueError("base must be finite and > 0")
    j = torch.arange(0, rotary_dim, 2, dtype=torch.float64)
    return torch.pow(torch.tensor(base, dtype=torch.float64), -j / max(1, rotary_dim)).to("cuda" if device is None else device)


def head_norm_rotate(q, k, positions, freq, q_weight=None, k_weight=None, eps=None, adjacent: bool = False,
                     q_out=None, k_out=None, stream=None):
    """Root-mean-square norm of each head of q [rows, n_q_heads, D] and k [rows, N, D] (both bf16
    or both fp32, strided rows allowed; either may be None), times q_weight and k_weight [D] of
    the same type (that start on 4 bytes: a bf16 slice from an even element on), then its
    rotation: pair j of the first 2 len(freq) values turns by positions[r] * freq[j] (int32
    [rows]; float64 radians, finite, see rotation_freq).  Pairs are values j and j + len(freq),
    or 2 j and 2 j + 1 where `adjacent`.  eps None leaves the norm out.
    Returns (q, k) of the same type; q_out and k_out may be given (q_out may be q itself, k_out
    k, else they are apart from both inputs and from each other; bf16 for fp32 rows), and rows
    at negative positions are not written."""
    return _ext().head_norm_rotate(q, k, positions, freq, q_weight, k_weight, eps, adjacent, q_out, k_out, stream)


class PageCopies(NamedTuple):
    """Pages to copy in every layer, int32: the first rows[i] rows (None: all) of page src[i] to
    page dst[i]; -1 is none, and so is everything from count[0] on (None: the whole list)."""
    src: torch.Tensor
    dst: torch.Tensor
    rows: torch.Tensor | None
    count: torch.Tensor | None


def page_fork(source, seq_len, block_table, free_blocks, n_free, block_tokens: int, length=None, finished=None,
              block_table_out=None, seq_len_out=None, n_free_out=None, flags=None, stream=None) -> PageCopies:
    """Row b of the table becomes the first length[b] positions (None or negative: all) of row
    source[b] as it was (None: its own; negative: nothing); rows marked in `finished` become
    empty.  Pages that no row holds any more go to the free list.  Rows of one call may share
    pages; a last page that two rows have begun is replaced by one of its own for all but one of
    them: the copies that are returned (page_copy) must be made before rows are appended.

    All int32, as in page_plan; source, length, finished [batch].  The table, lengths and free
    count after the call go to the _out tensors, by default to the inputs themselves.  A call
    that does not fit changes nothing (FLAG_NO_SPACE or FLAG_BAD_INDEX in `flags`)."""
    return PageCopies(*_ext().page_fork(source, seq_len, block_table, free_blocks, n_free, block_tokens, length,
                                        finished, block_table_out, seq_len_out, n_free_out, flags, stream), None)


def page_compact(seq_len, block_table, free_blocks, n_free, block_tokens: int, block_table_out=None, flags=None,
                 stream=None) -> PageCopies:
    """Move the pages that rows hold to the lowest numbers, so that the pool's end is free; the
    free list becomes all others.  The returned copies must be made (page_copy) before the pages
    are read."""
    src, dst, count = _ext().page_compact(seq_len, block_table, free_blocks, n_free, block_tokens,
                                          block_table_out, flags, stream)
    return PageCopies(src, dst, None, count)


def page_copy(caches, src, dst, rows=None, count=None, flags=None, stream=None):
    """Make the copies of a PageCopies in `caches`, a list of up to 128 layers of one shape:
    PagedCache objects or (k8, v8, k_scale, v_scale) tuples."""
    _ext().page_copy(caches, src, dst, rows, count, flags, stream)


def page_gather(k8, v8, k_scale, v_scale, block_table, seq_len, max_rows=None, length=None, k_out=None, v_out=None,
                flags=None, stream=None):
    """The first length[b] (int32 [batch]; None: all) stored positions of each sequence as packed
    rows: (k, v, cu_rows) with k, v [max_rows, N, D] bf16 (k_out and v_out, if given, which must
    not overlap and whose rows max_rows is by default) and int32 cu_rows [batch + 1].  Rows past cu_rows[-1] are not
    written.  More than max_rows rows: none, cu_rows all 0 and FLAG_NO_SPACE in `flags`."""
    return _ext().page_gather(k8, v8, k_scale, v_scale, block_table, seq_len, max_rows, length, k_out, v_out, flags,
                              stream)


class PageTable:
    """The pages of `batch` sequence slots, shared by all layers: block table, lengths, free
    list and a flags word (FLAG_*, ORed by the calls made through this table).  With `sharing`,
    rows may be forked: a release then frees pages that no other row holds."""

    def __init__(self, batch: int, max_blocks: int, num_blocks: int, block_tokens: int = 64, device=None,
                 sharing: bool = False):
        dev = torch.device("cuda" if device is None else device)
        self.block_tokens = block_tokens
        self.sharing = sharing
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
        """Give back the pages of the sequences marked in `finished` (int32 [batch]).  With `sharing`
        all or nothing, as page_fork: a length out of range in any row, finished or not, leaves the
        table as it is (FLAG_BAD_INDEX), since the pages which that row holds are not known."""
        if self.sharing:                             # (a release shortens no row: there are no copies)
            page_fork(None, self.seq_len, self.block_table, self.free_blocks, self.n_free, self.block_tokens,
                      finished=finished, flags=self.flags, stream=stream)
            return
        page_release(finished, self.seq_len, self.block_table, self.free_blocks, self.n_free,
                     self.block_tokens, flags=self.flags, stream=stream)

    def fork(self, source, length=None, finished=None, stream=None) -> PageCopies:
        """Rows become (the first length[b] positions of) rows source[b]; see page_fork.  The
        copies must be made in every layer's cache before the next append."""
        if not self.sharing:
            raise ValueError("the table was made without sharing")
        return page_fork(source, self.seq_len, self.block_table, self.free_blocks, self.n_free, self.block_tokens,
                         length=length, finished=finished, flags=self.flags, stream=stream)

    def compact(self, stream=None) -> PageCopies:
        """Move all pages to the pool's low end (see page_compact); the copies must be made in
        every layer's cache before the pages are read."""
        return page_compact(self.seq_len, self.block_table, self.free_blocks, self.n_free, self.block_tokens,
                            flags=self.flags, stream=stream)


class PagedCache:
    """One layer's K/V rows in 8-bit pages."""

    def __init__(self, n_kv_heads: int, head_dim: int, num_blocks: int, block_tokens: int = 64, device=None):
        dev = torch.device("cuda" if device is None else device)
        shape = (num_blocks, n_kv_heads, block_tokens, head_dim)
        self.k8 = torch.empty(shape, dtype=torch.uint8, device=dev)
        self.v8 = torch.empty(shape, dtype=torch.uint8, device=dev)
        self.k_scale = torch.empty(shape[:2], dtype=torch.float32, device=dev)
        self.v_scale = torch.empty(shape[:2], dtype=torch.float32, device=dev)

    def arrays(self):
        return self.k8, self.v8, self.k_scale, self.v_scale

    def append(self, k, v, table: PageTable, plan: PagePlan, stream=None):
        """Store the planned step's rows (see page_append)."""
        page_append(k, v, self.k8, self.v8, self.k_scale, self.v_scale, table.block_table,
                    table.seq_len, plan.cu_rows, flags=table.flags, stream=stream)

    def attend(self, q, table: PageTable, scale=None, out=None, lse=None, stream=None):
        """Decode attention, one query a sequence (see page_attention)."""
        return page_attention(q, self.k8, self.v8, self.k_scale, self.v_scale, table.block_table,
                              table.seq_len, scale=scale, out=out, lse=lse, flags=table.flags,
                              stream=stream)

    def gather(self, table: PageTable, max_rows=None, length=None, k_out=None, v_out=None, stream=None):
        """Stored rows as packed bf16 rows: (k, v, cu_rows), see page_gather."""
        return page_gather(self.k8, self.v8, self.k_scale, self.v_scale, table.block_table, table.seq_len, max_rows,
                           length=length, k_out=k_out, v_out=v_out, flags=table.flags, stream=stream)
