"""What the calls around the paged cache refuse because of what their buffers share, without a GPU."""
import ctypes
import math

import pytest
import torch

import residual_kv_cache_gb300 as rkv

from test_share_cpu import A, Rows, S, pages, table


@pytest.fixture(scope="module")
def lib():
    from residual_kv_cache_gb300 import build
    build.build()
    return rkv.lib()


def refused(lib, status, text):
    assert status == -1 and text in lib.rkv_last_error().decode(), (status, lib.rkv_last_error())


def test_head_rows_that_overlap(lib):
    """Outputs on each other or on an input that is not their own.  (1000 rows of 4 and of 2 heads
    of 64 bf16 values, at addresses that are only looked at.)"""
    far = 1 << 24

    def call(**kw):
        d = dict(q=A, k=A + far, q_out=A + 2 * far, k_out=A + 3 * far, q_strides=S(256, 64), k_strides=S(128, 64),
                 q_out_strides=S(256, 64), k_out_strides=S(128, 64), q_weight=None, k_weight=None, positions=A, freq=A,
                 n_rows=1000, n_q_heads=4, n_k_heads=2, head_dim=64, rotary_dim=64, adjacent=0, norm=0, dtype=1,
                 out_dtype=1, eps=0.0)
        return lib.rkv_head_norm_rotate(ctypes.byref(Rows(**{**d, **kw})), None)
    both = "q_out and k_out overlap"
    wide = dict(q_out_strides=S(512, 64), k_out_strides=S(512, 64))            # parts of rows of 512 values
    apart = dict(q_out_strides=S(512, 128), k_out_strides=S(512, 128))         # heads with room between them
    heads = dict(q_out_strides=S(64, 64000), k_out_strides=S(64, 64000))       # heads outermost
    for bad in (dict(k_out=A + 2 * far), dict(k_out=A + 2 * far + 1000 * 512 - 16), dict(k_out=A + 2 * far - 256000 + 16),
                dict(k_out=A + 2 * far + 3 * 128, **wide), dict(k_out=A + 2 * far - 2 * 128 + 16, **wide),
                dict(k_out=A + 2 * far + 64, **apart), dict(k_out=A + 2 * far + 3 * 256 + 112, **apart),
                dict(k_out=A + 2 * far + 999 * 128, **heads), dict(k_out=A + 2 * far, q_out_strides=S(64, 64000)),
                dict(k_out=A + 2 * far + 16, n_rows=1)):
        refused(lib, call(**bad), both)
    own = "overlaps an input"
    for bad in (dict(q_out=A + 512), dict(q_out=A, q_out_strides=S(512, 64)), dict(q_out=A + far),
                dict(k_out=A + far + 128), dict(k_out=A + 512 * 999),
                dict(q_out=A, k=A),                                                        # in place, and read as k
                dict(q=A, q_out=A, dtype=0, q_strides=S(256, 64)),                         # bf16 over fp32
                dict(q=A, q_out=A, q_strides=S(0, 64)),                                    # one row for all, and in place
                dict(q=A + 128, q_out=A, q_strides=S(512, 64), q_out_strides=S(512, 64))):
        refused(lib, call(**bad), own)
    refused(lib, call(q_strides=S(1 << 60, 64)), "address space")


def test_gathered_rows_that_overlap(lib):
    """(1000 rows of 8 heads of 128, at addresses that are only looked at.)"""
    far = 1 << 24

    def call(k=A, ks=S(1024, 128), v=A + far, vs=S(1024, 128), rows=1000):
        return lib.rkv_page_gather(ctypes.byref(pages()), table(), None, k, ks, v, vs, rows, A, None, None)
    for bad in (dict(v=A), dict(v=A + 1000 * 2048 - 16), dict(v=A - 1000 * 2048 + 16), dict(v=A + 2032, rows=1),
                dict(ks=S(2048, 128), v=A + 7 * 256, vs=S(2048, 128)), dict(ks=S(128, 128000), v=A + 999 * 256, vs=S(128, 128000)),
                dict(ks=S(2048, 256), v=A + 128, vs=S(2048, 256)), dict(ks=S(128, 128000))):
        refused(lib, call(**{**dict(v=A), **bad}), "k and v overlap")
    refused(lib, call(ks=S(1 << 60, 128)), "address space")


def test_tables_that_overlap_without_being_one(lib):
    """Entries would be read after others were written over them: 4 rows of 50, at A."""
    n, m, more = ctypes.c_size_t(), ctypes.c_size_t(), 1 << 16
    lib.rkv_page_fork_workspace(table(), 100, 64, ctypes.byref(n))
    lib.rkv_page_compact_workspace(100, ctypes.byref(m))
    t = table(seq_len=A + more)
    for out, lens in ((A + 4, A + more), (A - 4, A + more), (A + 199 * 4, A + more), (A, A + more + 4), (A, A + more - 12)):
        refused(lib, lib.rkv_page_fork(t, None, None, None, A, A, 100, 64, out, lens, A, A, A, A, A, n.value, None, None),
                "overlaps the table's")
    for out in (A + 4, A - 4, A + 199 * 4, A - 199 * 4):
        refused(lib, lib.rkv_page_compact(t, A, A, 100, 64, out, A, A, A, A, m.value, None, None), "overlaps the table's")


def test_gathered_offsets_on_the_lengths(lib):
    far = 1 << 24
    for lens, length, cu in ((A, None, A), (A, None, A - 16), (A, None, A + 12), (A, A + far, A + far), (A, A + far, A + far - 4)):
        refused(lib, lib.rkv_page_gather(ctypes.byref(pages()), table(seq_len=lens), length, A + 2 * far, S(1024, 128),
                                         A + 3 * far, S(1024, 128), 9, cu, None, None), "cu_rows overlaps")


def test_rotation_freq_refusals():
    """15 values are no pairs (they made the frequencies of 8), and powers of these are not."""
    for dim in (15, 1, -2):
        with pytest.raises(ValueError, match="rotary_dim"):
            rkv.rotation_freq(dim, device="cpu")
    for base in (0.0, -1e4, math.inf, math.nan):
        with pytest.raises(ValueError, match="base"):
            rkv.rotation_freq(16, base, device="cpu")
    assert rkv.rotation_freq(2, 5e5, device="cpu").tolist() == [1.0]


def test_device_zero_is_not_the_current_one(monkeypatch):
    seen = []
    for name in ("full", "zeros", "empty", "arange"):
        make = getattr(torch, name)
        monkeypatch.setattr(torch, name, lambda *a, _make=make, device=None, **kw: seen.append(device) or _make(*a, **kw))
    monkeypatch.setattr(torch.Tensor, "to", lambda t, where: seen.append(torch.device(where)) or t)
    rkv.PageTable(2, 3, 4, 16, device=0)
    rkv.PagedCache(2, 64, 4, 16, device=0)
    rkv.rotation_freq(16, device=0)
    assert len(seen) > 9 and {x for x in seen if x is not None} == {torch.device("cuda", 0)}
