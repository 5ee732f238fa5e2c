"""The full-attention layers' entry points without a GPU: what the library and the binding
refuse, and the float64 definitions pinned against independent facts."""
import ctypes
import math

import numpy as np
import pytest
import torch

import residual_kv_cache_gb300 as rkv
from oracle import pages as OP


class RP:
    """The structures of include/rkv.h's page and prompt entry points."""
    _Strides = ctypes.c_int64 * 2

    class _Pages(ctypes.Structure):
        _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                    ("v_scale", ctypes.c_void_p), ("n_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                    ("block_tokens", ctypes.c_int32), ("num_blocks", ctypes.c_int32)]

    class _Table(ctypes.Structure):
        _fields_ = [("block_table", ctypes.c_void_p), ("seq_len", ctypes.c_void_p), ("batch", ctypes.c_int32),
                    ("max_blocks", ctypes.c_int32)]

    class _Prompt(ctypes.Structure):
        _fields_ = [(n, ctypes.c_void_p) for n in ("q", "k", "v", "out", "lse")] + \
            [(n + "_strides", ctypes.c_int64 * 2) for n in ("q", "k", "v", "out")] + \
            [("cu_q", ctypes.c_void_p), ("cu_k", ctypes.c_void_p)] + \
            [(n, ctypes.c_int32) for n in ("batch", "total_q", "total_k", "n_q_heads", "n_kv_heads", "head_dim")] + \
            [("scale", ctypes.c_double), ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t)]


@pytest.fixture(scope="module")
def lib():
    from residual_kv_cache_gb300 import build
    build.build()
    return rkv.lib()


A = 1 << 20          # an aligned address that is only looked at, never read


def _pages(**kw):
    d = dict(k=A, v=A, k_scale=A, v_scale=A, n_kv_heads=8, head_dim=128, block_tokens=64, num_blocks=100)
    d.update(kw)
    return ctypes.byref(RP._Pages(*(d[n] for n, _ in RP._Pages._fields_)))


def _table(**kw):
    d = dict(block_table=A, seq_len=A, batch=4, max_blocks=50)
    d.update(kw)
    return ctypes.byref(RP._Table(*(d[n] for n, _ in RP._Table._fields_)))


BAD_PAGES = [(dict(k=None), -1), (dict(v_scale=None), -1), (dict(k=A + 8), -2), (dict(n_kv_heads=0), -1),
             (dict(head_dim=96), -1), (dict(block_tokens=8), -1), (dict(block_tokens=48), -1),
             (dict(num_blocks=0), -1), (dict(num_blocks=1 << 22, n_kv_heads=8), -1)]
BAD_TABLE = [(dict(block_table=None), -1), (dict(seq_len=None), -1), (dict(batch=0), -1),
             (dict(batch=8193), -1), (dict(max_blocks=0), -1), (dict(max_blocks=1 << 26), -1), (dict(max_blocks=(1 << 25) - 1), -1)]


def test_plan_and_release_refusals(lib):
    good = [_table(), A, A, A, 100, 64, 16, A, A, A, A, A, A, None, None]

    def plan(**at):
        args = list(good)
        for i, x in at.items():
            args[int(i[1:])] = x
        return lib.rkv_page_plan(*args)
    for bad, st in BAD_TABLE:
        assert plan(a0=_table(**bad)) == st, bad
    assert plan(a0=None) == -1
    for i in (1, 2, 3, 7, 8, 9, 10, 11, 12):
        assert plan(**{f"a{i}": None}) == -1, i
    for i, x in ((4, 0), (4, 1 << 26), (5, 0), (5, 24), (6, -1)):
        assert plan(**{f"a{i}": x}) == -1, (i, x)
    assert b"max_rows" in lib.rkv_last_error()
    rel = [_table(), A, A, A, 100, 64, None, None]
    for i, x in ((0, None), (1, None), (2, None), (3, None), (4, 0), (5, 65)):
        assert lib.rkv_page_release(*(x if j == i else y for j, y in enumerate(rel))) == -1, i
    for bad, st in BAD_TABLE:
        assert lib.rkv_page_release(_table(**bad), *rel[1:]) == st, bad


def test_append_refusals(lib):
    st2 = RP._Strides(1024, 128)
    good = [_pages(), _table(), A, st2, A, st2, 1, 4, A, None, None]

    def app(**at):
        args = list(good)
        for i, x in at.items():
            args[int(i[1:])] = x
        return lib.rkv_page_append(*args)
    for bad, st in BAD_PAGES:
        assert app(a0=_pages(**bad)) == st, bad
    for bad, st in BAD_TABLE:
        assert app(a1=_table(**bad)) == st, bad
    for i in (0, 1, 2, 3, 4, 5, 8):
        assert app(**{f"a{i}": None}) == -1, i
    assert app(a6=2) == -1 and app(a7=-1) == -1
    assert app(a2=A + 4) == -2 and app(a4=A + 2) == -2
    assert app(a3=RP._Strides(1028, 128)) == -2 and app(a5=RP._Strides(1024, -128)) == -2
    assert app(a7=0, a2=None) == 0                       # no rows: nothing is looked at


def test_page_attention_refusals(lib):
    n = ctypes.c_size_t()
    assert lib.rkv_page_attention_workspace(_pages(), _table(), 32, ctypes.byref(n)) == 0 and n.value > 0
    assert lib.rkv_page_attention_workspace(_pages(), _table(), 32, None) == -1
    st2 = RP._Strides(4096, 128)
    good = [_pages(), _table(), A, st2, 32, 0.1, A, None, A, n.value, None, None]

    def att(**at):
        args = list(good)
        for i, x in at.items():
            args[int(i[1:])] = x
        return lib.rkv_page_attention(*args)
    for bad, st in BAD_PAGES:
        assert att(a0=_pages(**bad)) == st, bad
    for bad, st in BAD_TABLE:
        assert att(a1=_table(**bad)) == st, bad
    for i in (0, 1, 2, 3, 6, 8):
        assert att(**{f"a{i}": None}) == -1, i
    for heads in (0, -8, 12, 8 * 17):
        assert att(a4=heads) == -1, heads
    for scale in (0.0, -1.0, math.inf, math.nan):
        assert att(a5=scale) == -1, scale
    assert att(a9=n.value - 1) == -3
    assert att(a2=A + 8) == -2 and att(a6=A + 2) == -2 and att(a8=A + 4) == -2
    assert att(a3=RP._Strides(4096, 100)) == -2


def test_prompt_refusals(lib):
    S = RP._Strides

    def call(**kw):
        d = dict(q=A, k=A, v=A, out=A, lse=None, q_strides=S(4096, 128), k_strides=S(1024, 128),
                 v_strides=S(1024, 128), out_strides=S(4096, 128), cu_q=A, cu_k=A, batch=2, total_q=10,
                 total_k=10, n_q_heads=32, n_kv_heads=8, head_dim=128, scale=0.1, workspace=None,
                 workspace_bytes=0)
        d.update(kw)
        p = RP._Prompt(*(d[n] for n, _ in RP._Prompt._fields_))
        return lib.rkv_prompt_attention(ctypes.byref(p), None, None)
    assert lib.rkv_prompt_attention(None, None, None) == -1
    for bad in (dict(q=None), dict(k=None), dict(v=None), dict(out=None), dict(cu_q=None), dict(cu_k=None),
                dict(batch=0), dict(batch=8193), dict(total_q=-1), dict(total_k=-1), dict(n_q_heads=0),
                dict(n_q_heads=12), dict(n_kv_heads=0), dict(head_dim=96), dict(scale=0.0),
                dict(scale=math.nan), dict(scale=math.inf)):
        assert call(**bad) == -1, bad
    for bad in (dict(q=A + 2), dict(k=A + 8), dict(out=A + 4), dict(q_strides=S(4100, 128)),
                dict(v_strides=S(1024, -128)), dict(out_strides=S(4096, 4))):
        assert call(**bad) == -2, bad
    assert call(total_q=0) == 0
    # rows of out that overlap, and sizes whose items would not fit their counters
    for bad in (dict(out_strides=S(1 << 60, 120)), dict(out_strides=S(120, 1 << 60)), dict(out_strides=S(0, 128)), dict(out_strides=S(4096, 0)), dict(out_strides=S(4088, 128)),
                dict(out_strides=S(4096, 120)), dict(out_strides=S(128, 1272)),
                dict(total_q=2 ** 30, n_q_heads=16)):
        assert call(**bad) == -1, bad

    def workspace(**kw):
        d = dict(total_q=500, total_k=500, n_q_heads=32, n_kv_heads=8, head_dim=128, batch=2, scale=0.1)
        d.update(kw)
        p, n = RP._Prompt(**d), ctypes.c_size_t(7)
        st = lib.rkv_prompt_attention_workspace(ctypes.byref(p), ctypes.byref(n))
        return n.value if st == 0 else st
    assert workspace() == 0 and workspace(total_q=10, total_k=5000) > 0 and workspace(head_dim=96) == -1
    assert lib.rkv_prompt_attention_workspace(None, None) == -1
    n = workspace(total_q=10, total_k=5000)
    assert call(total_k=5000, total_q=10) == -3 and call(total_k=5000, workspace=A, workspace_bytes=n - 1) == -3
    assert call(total_k=5000, workspace=None, workspace_bytes=n) == -3
    assert call(total_k=5000, workspace=A + 4, workspace_bytes=n) == -2


@pytest.mark.parametrize("scale", [1e-46, 1e-31, math.nextafter(1e-30, 0), 1e30, 1e39, -1e-30])
def test_scales_outside_their_range_are_refused(lib, scale):
    """A scale that underflows in fp32 would make NaN of masked scores, one that overflows of all."""
    S = RP._Strides
    p = RP._Prompt(q=A, k=A, v=A, out=A, q_strides=S(4096, 128), k_strides=S(1024, 128), v_strides=S(1024, 128),
                   out_strides=S(4096, 128), cu_q=A, cu_k=A, batch=2, total_q=10, total_k=10, n_q_heads=32,
                   n_kv_heads=8, head_dim=128, scale=scale)
    n = ctypes.c_size_t()
    assert lib.rkv_prompt_attention(ctypes.byref(p), None, None) == -1 and b"scale" in lib.rkv_last_error()
    assert lib.rkv_prompt_attention_workspace(ctypes.byref(p), ctypes.byref(n)) == -1
    assert lib.rkv_page_attention_workspace(_pages(), _table(), 32, ctypes.byref(n)) == 0
    assert lib.rkv_page_attention(_pages(), _table(), A, S(4096, 128), 32, scale, A, None, A, n.value, None, None) == -1
    assert b"scale" in lib.rkv_last_error()


def test_binding_refuses_what_the_library_cannot_see(lib):
    """CPU tensors, other objects and wrong types are refused with ValueError or TypeError
    before any call."""
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    u8, f32 = torch.zeros((3, 2, 16, 64), dtype=torch.uint8), torch.zeros((3, 2))
    with pytest.raises(ValueError, match="block_table must be a CUDA"):
        rkv.page_plan(i32(2), i32(2), i32(2, 4), i32(3), i32(1), 16, 8)
    with pytest.raises(ValueError, match="max_rows"):
        rkv.page_plan(i32(2), i32(2), i32(2, 4), i32(3), i32(1), 16, -1)
    with pytest.raises(ValueError, match="out of range"):
        rkv.page_plan(i32(2), i32(2), i32(2, 4), i32(3), i32(1), 16, 2 ** 31)
    with pytest.raises(TypeError):
        rkv.page_plan(i32(2), i32(2), i32(2, 4), i32(3), i32(1), None, 8)
    with pytest.raises(ValueError, match="block_table"):
        rkv.page_release(i32(2), i32(2), [[1]], i32(3), i32(1), 16)
    with pytest.raises(ValueError, match="k8"):
        rkv.page_append(bf(4, 2, 64), bf(4, 2, 64), u8, u8, f32, f32, i32(2, 4), i32(2), i32(3))
    with pytest.raises(ValueError, match="k8"):
        rkv.page_attention(bf(2, 4, 64), u8, u8, f32, f32, i32(2, 4), i32(2))
    with pytest.raises(ValueError, match="q must be a CUDA"):
        rkv.prompt_attention(bf(4, 4, 64), bf(4, 2, 64), bf(4, 2, 64), i32(2))
    with pytest.raises(ValueError, match="q must be a tensor"):
        rkv.prompt_attention(None, bf(4, 2, 64), bf(4, 2, 64), i32(2))


def test_missing_binding_fails_loudly(tmp_path, monkeypatch):
    from residual_kv_cache_gb300 import pages
    monkeypatch.setattr(pages, "__file__", str(tmp_path / "pages.py"))
    monkeypatch.setattr(pages, "_module", None)
    with pytest.raises(rkv.RkvLibraryMissing):
        rkv.page_release(None, None, None, None, None, 16)


# ------------------------------------------------------------- pins of the definitions
def test_e4m3_rounding_matches_torch():
    x = torch.cat([torch.randn(4000), torch.randn(4000) * 1e-2, torch.tensor([0.0, -0.0, 448.0, 464.0 - 1e-3,
                   2.0 ** -9, 2.0 ** -10, 1.5 * 2.0 ** -10, 17.0, 19.0])]).clamp(-448, 448)
    want = x.to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(OP.e4m3_round(x.double().numpy()), want)
    assert OP.e4m3_round(np.array([1e9]))[0] == 448.0 and np.isnan(OP.e4m3_round(np.array([np.nan]))[0])


def test_scale_is_the_smallest_power_of_two():
    for a in (1e-30, 0.0, 447.9, 448.0, 448.1, 896.0, 1.0, 3.4e38):
        s = OP.scale_of(a)
        assert a <= 448 * s and (s == 2.0 ** -64 or a > 224 * s) and math.frexp(s)[0] == 0.5


def test_append_page_by_page_equals_token_by_token_where_the_scale_holds():
    """Tokens stored one by one hold the same codes as stored at once when the first token
    has the page's largest magnitude; with a growing scale earlier tokens are rounded again,
    off by at most 2^-4 of the value twice, or half a subnormal step."""
    g = np.random.default_rng(3)
    P, N, D = 16, 2, 8
    x = g.standard_normal((20, N, D))
    x[0] *= 100
    x[16] *= 100
    table = [[1, 0]]

    def fresh():
        return np.zeros((2, N, P, D)), np.ones((2, N))
    c1, s1 = fresh()
    OP.append(x, c1, s1, table, [20], [0, 20], P)
    c2, s2 = fresh()
    for t in range(20):
        OP.append(x[t:t + 1], c2, s2, table, [t + 1], [0, 1], P)
    assert np.array_equal(c1, c2) and np.array_equal(s1, s2)
    y = x[::-1].copy()
    c3, s3 = fresh()
    for t in range(20):
        OP.append(y[t:t + 1], c3, s3, table, [t + 1], [0, 1], P)
    got = (c3 * s3[:, :, None, None])[table[0]].transpose(0, 2, 1, 3).reshape(32, N, D)[:20]
    step = (s3[table[0]] * 2.0 ** -10).repeat(P, axis=0)[:20, :, None]
    assert np.all(np.abs(got - y) <= 2 * np.maximum(np.abs(y) * 1.07 * 2.0 ** -4, step))


def test_attention_definitions():
    """One key: its value.  Equal keys: the mean.  A query before every key: zero, -inf."""
    g = np.random.default_rng(4)
    v = g.standard_normal((5, 1, 4))
    q, k = g.standard_normal((5, 2, 4)), np.zeros((5, 1, 4))
    o, lse, _, _ = OP.prompt_attention(q, k, v, [0, 5], [0, 5], 0.5)
    for i in range(5):
        assert np.allclose(o[i], v[:i + 1, 0].mean(0)) and np.allclose(lse[i], math.log(i + 1))
    o, lse, _, _ = OP.prompt_attention(q, k, v, [0, 5], [0, 2], 0.5)
    assert not o[:3].any() and np.all(lse[:3] == -math.inf) and np.allclose(o[3], v[0, 0])
    kp, vp = g.standard_normal((3, 1, 16, 4)), g.standard_normal((3, 1, 16, 4))
    o, lse, _, _ = OP.page_attention(q[:2], kp, vp, [[2, 1], [0, 0]], [17, 0], 16, 0.5)
    kk, vv = np.concatenate([kp[2, 0], kp[1, 0]])[:17], np.concatenate([vp[2, 0], vp[1, 0]])[:17]
    w = np.exp(0.5 * kk @ q[0, 1])
    assert np.allclose(o[0, 1], w @ vv / w.sum()) and not o[1].any() and lse[1, 0] == -math.inf


def test_plan_definition():
    table = np.full((3, 4), -1)
    table[0, 0] = 7
    cu, rows, lens, left, t = OP.plan([3, 0, 33], [15, 0, 0], table, [5, 6, 8, 9, 1], 5, 16, 40)
    assert cu == [0, 3, 3, 36] and lens == [18, 0, 33] and left == 1
    assert t.tolist() == [[7, 1, -1, -1], [-1] * 4, [9, 8, 6, -1]]
    assert rows[:3] == [(0, 15, 7 * 16 + 15), (0, 16, 16), (0, 17, 17)] and rows[-1] == (2, 32, 96)
    assert OP.plan([3, 0, 33], [15, 0, 0], table, [5, 6, 8], 3, 16, 40) is None
    assert OP.plan([3, 0, 33], [15, 0, 0], table, [5, 6, 8, 9, 1], 5, 16, 35) is None
    lens, t, free, n = OP.release([1, 0, 1], lens, t, [5, 0, 0, 0, 0, 0], left, 16)
    assert lens == [0, 0, 0] and n == 6 and free == [5, 7, 1, 9, 8, 6] and np.all(t == -1)
