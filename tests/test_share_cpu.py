"""Norm and rotation of head rows, and pages that several sequences hold, without a GPU: what the
library and the binding refuse, and the float64 definitions pinned against independent facts."""
import ctypes
import math

import numpy as np
import pytest
import torch

import residual_kv_cache_gb300 as rkv
from oracle import codec as C
from oracle import pages as OP

S = ctypes.c_int64 * 2
A = 1 << 20          # an aligned address that is only looked at, never read


class Pages(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("k", "v", "k_scale", "v_scale")] + \
        [(n, ctypes.c_int32) for n in ("n_kv_heads", "head_dim", "block_tokens", "num_blocks")]


class Table(ctypes.Structure):
    _fields_ = [("block_table", ctypes.c_void_p), ("seq_len", ctypes.c_void_p), ("batch", ctypes.c_int32),
                ("max_blocks", ctypes.c_int32)]


class Rows(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("q", "k", "q_out", "k_out")] + \
        [(n, S) for n in ("q_strides", "k_strides", "q_out_strides", "k_out_strides")] + \
        [(n, ctypes.c_void_p) for n in ("q_weight", "k_weight", "positions", "freq")] + \
        [(n, ctypes.c_int32) for n in ("n_rows", "n_q_heads", "n_k_heads", "head_dim", "rotary_dim", "adjacent",
                                       "norm", "dtype", "out_dtype")] + [("eps", ctypes.c_double)]


@pytest.fixture(scope="module")
def lib():
    from residual_kv_cache_gb300 import build
    build.build()
    return rkv.lib()


def pages(**kw):
    d = dict(k=A, v=A, k_scale=A, v_scale=A, n_kv_heads=8, head_dim=128, block_tokens=64, num_blocks=100)
    return Pages(**{**d, **kw})


def table(**kw):
    return ctypes.byref(Table(**{**dict(block_table=A, seq_len=A, batch=4, max_blocks=50), **kw}))


BAD_PAGES = [(dict(k=None), -1), (dict(v_scale=None), -1), (dict(k=A + 8), -2), (dict(n_kv_heads=0), -1),
             (dict(head_dim=96), -1), (dict(block_tokens=48), -1), (dict(num_blocks=0), -1)]
BAD_TABLE = [(dict(block_table=None), -1), (dict(seq_len=None), -1), (dict(batch=0), -1), (dict(batch=8193), -1),
             (dict(max_blocks=0), -1), (dict(max_blocks=1 << 26), -1)]


def changed(good, at):
    args = list(good)
    for i, x in at.items():
        args[i] = x
    return args


def test_head_rows_refusals(lib):
    def call(**kw):
        d = dict(q=A, k=A, q_out=A, k_out=A, q_strides=S(4096, 128), k_strides=S(1024, 128),
                 q_out_strides=S(4096, 128), k_out_strides=S(1024, 128), q_weight=A, k_weight=None, positions=A,
                 freq=A, n_rows=5, n_q_heads=32, n_k_heads=8, head_dim=128, rotary_dim=128, adjacent=0, norm=1,
                 dtype=1, out_dtype=1, eps=1e-6)
        return lib.rkv_head_norm_rotate(ctypes.byref(Rows(**{**d, **kw})), None)
    assert lib.rkv_head_norm_rotate(None, None) == -1
    for bad in (dict(q=None), dict(k=None), dict(q_out=None), dict(k_out=None), dict(positions=None), dict(freq=None),
                dict(n_rows=-1), dict(n_rows=2 ** 30 + 1), dict(n_q_heads=-1), dict(n_k_heads=65536),
                dict(head_dim=96), dict(rotary_dim=24), dict(rotary_dim=144), dict(rotary_dim=-16), dict(dtype=2),
                dict(out_dtype=0), dict(eps=0.0), dict(eps=math.nan), dict(eps=math.inf), dict(eps=-1e-6),
                dict(norm=0), dict(q_out_strides=S(4096, 120)), dict(q_out_strides=S(0, 128)),
                dict(k_out_strides=S(1024, 0)), dict(k_out_strides=S(128, 512))):
        assert call(**bad) == -1, bad
    for bad in (dict(q=A + 8), dict(k_out=A + 2), dict(q_weight=A + 2), dict(freq=A + 4),
                dict(q_strides=S(4100, 128)), dict(k_strides=S(-1024, 128)), dict(q_out_strides=S(4096, 132))):
        assert call(**bad) == -2, bad
    assert call(n_rows=0, positions=None) == 0 and call(n_q_heads=0, n_k_heads=0) == 0
    assert call(dtype=0, out_dtype=0, q_strides=S(4098, 128)) == -2


def test_fork_and_compact_refusals(lib):
    n = ctypes.c_size_t()
    assert lib.rkv_page_fork_workspace(table(), 100, 64, ctypes.byref(n)) == 0 and n.value >= 4 * (2 * 100 + 200)
    fork = [table(), A, A, A, A, A, 100, 64, A, A, A, A, A, A, A, n.value, None, None]
    call = lambda at: lib.rkv_page_fork(*changed(fork, at))  # noqa: E731
    for bad, st in BAD_TABLE:
        assert call({0: table(**bad)}) == st, bad
        assert lib.rkv_page_fork_workspace(table(**bad), 100, 64, ctypes.byref(n)) == st
    assert call({0: None}) == -1 and call({0: table(batch=8192, max_blocks=1 << 18)}) == -1
    for i in (4, 5, 8, 9, 10, 11, 12, 13):
        assert call({i: None}) == -1, i
    for i, x in ((6, 0), (6, 1 << 26), (7, 24)):
        assert call({i: x}) == -1, (i, x)
    assert call({14: None}) == -3 and call({15: fork[15] - 1}) == -3 and call({14: A + 4}) == -2
    assert lib.rkv_page_fork_workspace(table(), 100, 64, None) == -1
    m = ctypes.c_size_t()
    assert lib.rkv_page_compact_workspace(100, ctypes.byref(m)) == 0 and m.value > 0
    assert lib.rkv_page_compact_workspace(0, ctypes.byref(m)) == -1 and lib.rkv_page_compact_workspace(9, None) == -1
    lib.rkv_page_compact_workspace(100, ctypes.byref(m))
    comp = [table(), A, A, 100, 64, A, A, A, A, A, m.value, None, None]
    call = lambda at: lib.rkv_page_compact(*changed(comp, at))  # noqa: E731
    for bad, st in BAD_TABLE:
        assert call({0: table(**bad)}) == st, bad
    for i in (0, 1, 2, 5, 6, 7, 8):
        assert call({i: None}) == -1, i
    assert call({3: 0}) == -1 and call({4: 65}) == -1
    assert call({9: None}) == -3 and call({10: m.value - 1}) == -3 and call({9: A + 8}) == -2


def test_copy_and_gather_refusals(lib):
    def layers(*pg):
        return (Pages * len(pg))(*pg)
    copy = [layers(pages(), pages()), 2, A, A, None, None, 3, None, None]
    call = lambda at: lib.rkv_page_copy(*changed(copy, at))  # noqa: E731
    for bad, st in BAD_PAGES:
        assert call({0: layers(pages(), pages(**bad))}) == st, bad
    for other in (dict(num_blocks=99), dict(n_kv_heads=4), dict(head_dim=64), dict(block_tokens=32)):
        assert call({0: layers(pages(), pages(**other))}) == -1, other
    for i, x in ((0, None), (1, 0), (1, 129), (2, None), (3, None), (6, -1)):
        assert call({i: x}) == -1, (i, x)
    assert call({6: 0, 2: None}) == 0
    gather = [ctypes.byref(pages()), table(), None, A, S(1024, 128), A, S(1024, 128), 7, A, None, None]
    call = lambda at: lib.rkv_page_gather(*changed(gather, at))  # noqa: E731
    for bad, st in BAD_PAGES:
        assert call({0: ctypes.byref(pages(**bad))}) == st, bad
    for bad, st in BAD_TABLE:
        assert call({1: table(**bad)}) == st, bad
    for i, x in ((0, None), (1, None), (3, None), (4, None), (5, None), (6, None), (7, -1), (8, None),
                 (4, S(1024, 120)), (6, S(0, 128)), (4, S(128, 640))):
        assert call({i: x}) == -1, i
    for i, x in ((3, A + 8), (5, A + 2), (4, S(1028, 128)), (6, S(1024, -128))):
        assert call({i: x}) == -2, i


def test_binding_refuses_what_the_library_cannot_see(lib):
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    u8, f32 = torch.zeros((3, 2, 16, 64), dtype=torch.uint8), torch.zeros((3, 2))
    freq = torch.zeros(32, dtype=torch.float64)
    with pytest.raises(ValueError, match="q must be a CUDA"):
        rkv.head_norm_rotate(bf(4, 2, 64), bf(4, 2, 64), i32(4), freq)
    with pytest.raises(ValueError, match="k must be a CUDA"):
        rkv.head_norm_rotate(None, bf(4, 2, 64), i32(4), freq)
    with pytest.raises(ValueError, match="both None"):
        rkv.head_norm_rotate(None, None, i32(4), freq)
    with pytest.raises(ValueError, match="block_table must be a CUDA"):
        rkv.page_fork(i32(2), i32(2), i32(2, 4), i32(3), i32(1), 16)
    with pytest.raises(ValueError, match="block_table must be a CUDA"):
        rkv.page_compact(i32(2), i32(2, 4), i32(3), i32(1), 16)
    with pytest.raises(TypeError):
        rkv.page_compact(i32(2), i32(2, 4), i32(3), i32(1), None)
    for caches in ([], [(u8, u8, f32)], [(u8, u8, f32, f32)] * 129, [(u8, u8, f32, f32)]):
        with pytest.raises(ValueError):
            rkv.page_copy(caches, i32(2), i32(2))
    with pytest.raises(ValueError, match="k8"):
        rkv.page_gather(u8, u8, f32, f32, i32(2, 4), i32(2), 8)
    t = object.__new__(rkv.PageTable)
    t.sharing = False
    with pytest.raises(ValueError, match="without sharing"):
        t.fork(None)


# ------------------------------------------------------------- pins of the definitions
def test_rotation_is_the_restores():
    g = np.random.default_rng(1)
    x, pos = g.standard_normal((6, 3, 64)), [0, 1, 77, 5000, 131071, 2 ** 31 - 1]
    freq = rkv.rotation_freq(64, 5e5, device="cpu")
    assert freq.dtype == torch.float64 and freq.shape == (32,)
    want = C.rope(x, np.array(pos), 5e5)
    # angles of up to 2^31 radians, whose factors agree to 2^-52
    assert np.abs(OP.norm_rotate(x, pos, freq.tolist()) - want).max() < 2.0 ** 31 * 2.0 ** -50
    assert len(rkv.rotation_freq(0, device="cpu")) == 0


def test_norm_and_pairs():
    g = np.random.default_rng(2)
    x, w = g.standard_normal((2, 1, 64)), g.standard_normal(64)
    y = OP.norm_rotate(x, [3, -1], [], w, 1e-3)
    assert np.allclose(y[0, 0], x[0, 0] / np.sqrt(np.mean(x[0, 0] ** 2) + 1e-3) * w) and np.isnan(y[1]).all()
    # adjacent pairs are half pairs of the values in another order; what is not rotated stays
    order = np.concatenate([np.arange(0, 32, 2), np.arange(1, 32, 2), np.arange(32, 64)])
    f = list(0.3 ** np.arange(16))
    assert np.allclose(OP.norm_rotate(x, [9, 9], f, adjacent=True)[..., order], OP.norm_rotate(x[..., order], [9, 9], f))
    z = OP.norm_rotate(x, [9, 9], f)
    assert np.array_equal(z[..., 32:], x[..., 32:]) and np.allclose((z ** 2).sum(-1), (x ** 2).sum(-1))


def test_fork_definition():
    T = [[3, 5, 9, -1], [4, -1, -1, -1], [-1] * 4]
    lens, free = [40, 16, 0], [7, 1, 0, 0, 0, 0, 0, 0, 0, 0]
    # row 2 becomes row 0's first 24 positions: page 3 shared, the begun one its own
    t, l, f, n, c = OP.fork([0, 1, 0], [-1, -1, 24], lens, T, free, 2, 16)
    assert l == [40, 16, 24] and t.tolist() == [[3, 5, 9, -1], [4, -1, -1, -1], [3, 1, -1, -1]]
    assert n == 1 and c == {2: (5, 1, 8)} and f == free
    # row 0 finishes: only what row 2 does not hold is free; then row 2 itself, cut
    t, l, f, n, c = OP.fork(None, [0, -1, -1], l, t, f, n, 16)
    assert n == 3 and f[:3] == [7, 5, 9] and c == {} and t[0].tolist() == [-1] * 4
    t, l, f, n, c = OP.fork(None, [-1, -1, 3], l, t, f, n, 16)
    assert n == 4 and f[3] == 1 and c == {} and t[2].tolist() == [3, -1, -1, -1]
    # everything swapped round, and a page cut where another row holds it whole
    t, l, f, n, c = OP.fork([2, 2, 1], [2, 3, 15], [0, 16, 32], [[-1] * 2, [8, -1], [8, 6]], [5, 2, 0, 0, 0, 0, 0, 0, 0], 2, 16)
    assert c == {1: (8, 6, 3), 2: (8, 2, 15)} and t.tolist() == [[8, -1], [6, -1], [2, -1]] and n == 1
    assert OP.fork([0], [41], [40], [[3, 5, 9, -1]], free, 2, 16) is None
    assert OP.fork([0, 0], None, [40, 0], T[:2], [0] * 10, 0, 16) is None
    assert OP.fork([1, 0], None, [40, 16], T[:2], [0] * 10, 0, 16)[1] == [16, 40]


def test_compact_definition():
    t, n, moves = OP.compact([40, 16, 0], [[7, 2, 9, 1], [2, -1, -1, -1], [5, -1, -1, -1]], 10, 16)
    assert n == 3 and moves == [(7, 0), (9, 1)]
    assert t.tolist() == [[0, 2, 1, -1], [2, -1, -1, -1], [-1, -1, -1, -1]]


def test_gather_definition_reads_what_append_stored():
    g = np.random.default_rng(3)
    codes, scale = np.zeros((4, 2, 16, 8)), np.ones((4, 2))
    x = np.float64(np.float32(g.standard_normal((23, 2, 8))))
    OP.append(x, codes, scale, [[2, 0], [3, -1]], [20, 3], [0, 20, 23], 16)
    got = OP.gather(codes, scale, [[2, 0], [3, -1]], [20, 3], 16)
    step = np.concatenate([scale[2][None].repeat(16, 0), scale[0][None].repeat(4, 0), scale[3][None].repeat(3, 0)])
    assert got.shape == (23, 2, 8) and np.all(np.abs(got - x) <= np.maximum(np.abs(x) * 2.0 ** -4, step[..., None] * 2.0 ** -10))
