"""GPU parity of the norm and rotation of query and key rows against the float64 definition.

Tolerance of a value, from the roundings (u = half a step, relative; |a|, |b| its pair's values
before the turn, or the value itself twice where it does not turn):
* norm: a sum of D positive squares in at most 23 roundings, halved by the root, rsqrt to 2 ulp
  (2^-22), and two products: below 18 2^-24;
* angle: upper 32 bits of the turn and their conversion, 2^-25 of a half turn and 2^-32 of a
  turn, below 2 2^-24; sin and cos to 2 ulp of values below 1, 2 2^-24; position times frequency
  in 64 bits on both sides, below pos freq 2^-50; two products and a sum, 3 2^-24;
together below (|a| + |b|) (2^-19 + pos freq 2^-50), and the output's own rounding.
"""
import numpy as np
import pytest
import torch

import residual_kv_cache_gb300 as rkv
from oracle import pages as OP

from _common import np64

pytestmark = pytest.mark.gpu
cuda = pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")
BF, F32 = torch.bfloat16, torch.float32


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def randn(*shape, seed, dtype=BF):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


def check(out, x, positions, freq, weight=None, eps=None, adjacent=False):
    """out against the definition; rows at negative positions hold what `out` held: 7."""
    x, h = np64(x), len(freq)
    f = np64(freq)
    w = None if weight is None else np64(weight)
    ref = OP.norm_rotate(x, positions, f.tolist(), w, eps, adjacent)
    got, u = np64(out), torch.finfo(out.dtype).eps / 2
    with np.errstate(over="ignore", invalid="ignore"):
        y = np.abs(OP.norm_rotate(x, positions, [], w, eps))
        size = 2 * y
        if h:
            a, b = (slice(0, 2 * h, 2), slice(1, 2 * h, 2)) if adjacent else (slice(0, h), slice(h, 2 * h))
            both = y[..., a] + y[..., b]
            size[..., a], size[..., b] = both, both
        angle = np.zeros(x.shape)
        if h:
            pf = np.abs(np.maximum(positions, 0)[:, None, None] * f)
            angle[..., a], angle[..., b] = pf, pf
        tol = size * (2.0 ** -19 + angle * 2.0 ** -50) + u * np.abs(ref) + 1e-37
    for r, p in enumerate(positions):
        if p < 0:
            assert np.all(got[r] == 7), r
        else:
            err = np.abs(got[r] - ref[r])
            assert np.all(err <= tol[r]), (r, p, float((err / tol[r]).max()))


POS = [0, 1, 5, 131071, -1, 77, 2 ** 31 - 1, 16384, 1000003]
CASES = [  # rows, q heads, k heads, D, rotary, adjacent, norm, in, out
    (1, 32, 8, 128, 128, False, True, BF, BF), (9, 28, 4, 128, 128, False, False, BF, BF),
    (16, 5, 5, 128, 64, False, True, BF, BF), (7, 1, 1, 64, 64, True, True, BF, BF),
    (67, 3, 2, 64, 32, False, True, F32, F32), (33, 9, 1, 128, 128, True, True, F32, BF),
    (20, 12, 1, 128, 32, True, False, F32, F32), (40, 16, 8, 64, 64, False, False, BF, BF),
    (5, 7, 3, 128, 0, False, True, BF, BF), (300, 2, 1, 64, 16, False, True, BF, BF)]


@cuda
@pytest.mark.parametrize("case", range(len(CASES)))
@pytest.mark.parametrize("layout", ["own", "projection", "in place", "heads outer"])
def test_matches_the_definition(case, layout):
    n, hq, hk, D, R, adjacent, norm, tin, tout = CASES[case]
    if layout == "in place" and tin != tout:
        tout = tin
    pos = [POS[(i * 5 + case) % len(POS)] for i in range(n)]
    freq = rkv.rotation_freq(R, 1e4 * 10 ** (case % 3))
    wq, wk = (randn(2, D, seed=case + 50, dtype=tin) if norm else (None, None))
    eps = 1e-5 if norm else None
    if layout == "heads outer":
        q, k = (randn(h, n, D, seed=case + h, dtype=tin).transpose(0, 1) for h in (hq, hk))
    else:
        rows = randn(n, hq + 2 * hk, D, seed=case, dtype=tin)
        q, k = rows[:, :hq], rows[:, hq:hq + hk]
        if layout == "own":
            q, k = q.contiguous(), k.contiguous()
    q0, k0 = q.clone(), k.clone()
    live = torch.tensor([p >= 0 for p in pos], device="cuda")
    if layout == "in place":
        q[~live], k[~live] = 7, 7
        rest = rows[:, hq + hk:].clone()
        a, b = rkv.head_norm_rotate(q, k, i32(pos), freq, wq, wk, eps, adjacent, q_out=q, k_out=k)
        assert a is q and b is k and torch.equal(rows[:, hq + hk:], rest)
    else:
        qo, ko = (torch.full((n, h + 1, D), 7, dtype=tout, device="cuda")[:, 1:] for h in (hq, hk))
        a, b = rkv.head_norm_rotate(q, k, i32(pos), freq, wq, wk, eps, adjacent, q_out=qo, k_out=ko)
        assert a is qo and b is ko and torch.equal(q, q0) and torch.equal(k, k0)
        assert (qo._base[:, 0] == 7).all() and (ko._base[:, 0] == 7).all()
    check(a, q0, pos, freq, wq, eps, adjacent)
    check(b, k0, pos, freq, wk, eps, adjacent)


@cuda
def test_outputs_are_made_and_one_of_the_two_may_be_left_out():
    q, k, pos, freq = randn(6, 4, 64, seed=1), randn(6, 3, 64, seed=2), [3, 9, 27, 81, 243, 729], rkv.rotation_freq(64)
    a, b = rkv.head_norm_rotate(q, k, i32(pos), freq)
    assert a.dtype == BF and a.shape == q.shape and b.shape == k.shape
    check(a, q, pos, freq)
    check(b, k, pos, freq)
    c, none = rkv.head_norm_rotate(q, None, i32(pos), freq)
    assert none is None and torch.equal(c, a)
    none, c = rkv.head_norm_rotate(None, k, i32(pos), freq)
    assert none is None and torch.equal(c, b)
    w = randn(64, seed=3)
    c, d = rkv.head_norm_rotate(q, k, i32(pos), freq, k_weight=w, eps=1e-6)       # a weight for one of them
    check(c, q, pos, freq, None, 1e-6)
    check(d, k, pos, freq, w, 1e-6)
    # fp32 rows: a bf16 output for one makes the other bf16; rows and heads that are one in memory
    qf, kf = q.float()[:, :1].expand(6, 4, 64), k.float()[:1].expand(6, 3, 64)
    qo = torch.empty(6, 4, 64, dtype=BF, device="cuda")
    c, d = rkv.head_norm_rotate(qf, kf, i32(pos), freq, eps=1e-6, q_out=qo)
    assert c is qo and d.dtype == BF
    check(c, qf, pos, freq, None, 1e-6)
    check(d, kf, pos, freq, None, 1e-6)
    e = torch.empty_like(q[:0])
    a, b = rkv.head_norm_rotate(e, e, i32([]), freq)
    assert a.shape == e.shape
    # without norm and rotation a row is itself, whatever it holds (a NaN stays one, of any bits)
    odd = randn(6, 4, 64, seed=4)
    odd.view(torch.int16)[0, 0, :6] = torch.tensor([0x7F80, -128, 0x7FC0, -32768, 1, 0x7F7F], dtype=torch.int16)
    a, _ = rkv.head_norm_rotate(odd, None, i32(pos), freq[:0])
    same = ~odd.isnan()
    assert torch.equal(a.view(torch.int16)[same], odd.view(torch.int16)[same]) and a[~same].isnan().all()


@cuda
@pytest.mark.parametrize("dtype", [BF, F32])
def test_magnitudes_at_the_ends_of_the_range(dtype):
    """Squares past fp32 and below it, zero rows, and NaN and infinity, which stay in their head
    (the definition: NaN makes the head NaN, an infinity its own pair NaN and the others 0)."""
    x = randn(8, 3, 128, seed=5, dtype=F32)
    for r, scale in enumerate([1e38, 1e30, 2.0 ** 64, 1e19, 1e-19, 1e-30, 1e-38]):
        x[r] *= scale / 4
    x[7] = 0
    x[0, 1] = 0
    x[0, 1, 5] = 3e38
    x = x.to(dtype)
    pos, freq, w = [0, 1, 2, 3, 4, 5, 6, 7], rkv.rotation_freq(64), randn(128, seed=6, dtype=dtype)
    for eps in (1e-6, 1e-30):
        q, k = rkv.head_norm_rotate(x, x, i32(pos), freq, w, None, eps)
        check(q, x, pos, freq, w, eps)
        check(k, x, pos, freq, None, eps)
    y = x.clone()
    y[3, 1, 7], y[4, 0, 100] = float("nan"), float("inf")
    a, _ = rkv.head_norm_rotate(y, None, i32(pos), freq, w, None, 1e-6)
    same = torch.ones(8, 3, dtype=torch.bool)
    same[3, 1] = same[4, 0] = False
    ref, _ = rkv.head_norm_rotate(x, None, i32(pos), freq, w, None, 1e-6)
    assert torch.equal(a[same], ref[same]) and a[3, 1].isnan().all()
    assert a[4, 0, 100].isnan() and (a[4, 0, 64:].nan_to_num(0) == 0).all() and (a[4, 0, :64] == 0).all()


@cuda
def test_rows_past_two_gigabytes():
    """Offsets of rows that pass 32 bits, in elements and in bytes."""
    base = torch.zeros(2 * (2 ** 30 + 64) + 4 * 128, dtype=BF, device="cuda")
    q = base.as_strided((3, 2, 128), (2 ** 30 + 64, 128, 1))
    q.copy_(randn(3, 2, 128, seed=8))
    x, freq = q.clone(), rkv.rotation_freq(128)
    rkv.head_norm_rotate(q, None, i32([4, 5, 6]), freq, eps=1e-6, q_out=q)
    check(q, x, [4, 5, 6], freq, None, 1e-6)
    assert int((base != 0).sum()) == int((q != 0).sum())


@cuda
def test_many_rows_have_the_bits_of_few():
    """Each row's result depends on the row alone, however the call shares its work."""
    n = 20011
    q, k = randn(n, 9, 128, seed=9), randn(n, 2, 128, seed=10)
    pos = torch.randint(0, 200000, (n,), generator=torch.Generator().manual_seed(1), dtype=torch.int32).cuda()
    w, freq = randn(128, seed=11), rkv.rotation_freq(128, 5e5)
    a, b = rkv.head_norm_rotate(q, k, pos, freq, w, w, 1e-6)
    for r in (0, 1, 4863, 4864, 15000, n - 1):
        c, d = rkv.head_norm_rotate(q[r:r + 1], k[r:r + 1], pos[r:r + 1], freq, w, w, 1e-6)
        assert torch.equal(a[r:r + 1], c) and torch.equal(b[r:r + 1], d)
    rows = [0, 1, n // 2, n - 1]
    check(a[rows], q[rows], pos[rows].tolist(), freq, w, 1e-6)


@cuda
def test_graph_replay_and_other_streams():
    q, k, freq = randn(11, 4, 64, seed=12), randn(11, 2, 64, seed=13), rkv.rotation_freq(64)
    pos = i32(list(range(11)))
    want = rkv.head_norm_rotate(q, k, pos, freq, eps=1e-6)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = rkv.head_norm_rotate(q, k, pos, freq, eps=1e-6, stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = rkv.head_norm_rotate(q, k, pos, freq, eps=1e-6)
    pos.add_(1000)
    q.mul_(3)
    graph.replay()
    again = rkv.head_norm_rotate(q, k, pos, freq, eps=1e-6)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(out, again)) and not torch.equal(again[1], want[1])


@cuda
def test_binding_refusals():
    q, k, pos, freq = randn(4, 4, 64, seed=1), randn(4, 2, 64, seed=2), i32([0] * 4), rkv.rotation_freq(64)
    call = rkv.head_norm_rotate
    for bad in (dict(q=q.half()), dict(k=k.float()), dict(k=k[:3]), dict(k=randn(4, 2, 128, seed=1)),
                dict(positions=pos[:3]), dict(positions=pos.long()), dict(freq=freq.float()), dict(freq=freq[None]),
                dict(freq=freq.cpu()), dict(q_weight=randn(64, seed=1)), dict(q_weight=q[0, 0].float(), eps=1e-6),
                dict(q_weight=q[0, 0, :32], eps=1e-6), dict(eps=0.0), dict(eps=float("nan")), dict(freq=freq[:12]),
                dict(freq=torch.cat([freq, freq])), dict(q_out=q[:3]), dict(q_out=torch.empty_like(q, dtype=torch.half)),
                dict(q_out=q.float()), dict(q_out=q[:, :1].expand(4, 4, 64)), dict(q=q[..., ::2], k=k[..., ::2]),
                dict(k=None, k_out=k), dict(k=None, k_weight=k[0, 0], eps=1e-6), dict(q=q[0])):
        args = dict(dict(q=q, k=k, positions=pos, freq=freq), **bad)
        with pytest.raises((ValueError, rkv.RkvError)):
            call(**args)
    with pytest.raises(TypeError):
        call(q, k, pos, freq, eps="small")
