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
tensors made on another stream must be ready there, as for any torch operation.  Nothing is
differentiable: results carry no gradient.
"""
from __future__ import annotations

import importlib
import os
from typing import NamedTuple

import torch

import residual_kv_cache_gb300 as _rkv

__all__ = ["PagedCache", "PagePlan", "PageTable", "page_append", "page_attention", "page_plan",
           "page_release", "prompt_attention"]

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
