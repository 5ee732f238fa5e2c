"""GPU parity of the full-attention layers' operators against their float64 definitions.

Tolerances, per element, from the roundings (u = half a step, relative):
* plan, release, codes and scales: equal (whole numbers, powers of two, one rounding each);
* prompt attention: the output's bf16 rounding (u = 2^-8), each weight's bf16 rounding
  (2^-8 of sum w |v| at most), and fp32 scores: a D-term sum is off by at most
  D 2^-24 sum |q||k|, twice that (relative) in a weight over its normaliser, doubled
  again for the scale, the subtraction and exp2, whose arguments are below 2^8;
* page attention: the same with weights of 12 significant bits (2^-12) of the largest
  weight's scale: 2^-11 of sum w |v| covers it and the range kept below the maximum;
  (each weight is within 2^-15 of itself down to 2^-18 of the head's largest and within 2^-11
  down to 2^-28, which the cases with a dominant key reach: 2^-24 and less, 2^-11 of the sum);
* lse: the fp32 score error and 2^-20 of its magnitude.
"""
import math

import numpy as np
import pytest
import torch

import residual_kv_cache_gb300 as rkv
from oracle import pages as OP

from _common import np64

pytestmark = pytest.mark.gpu
cuda = pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def gen(seed):
    return torch.Generator().manual_seed(seed)


def randn(*shape, seed, dtype=torch.bfloat16):
    return torch.randn(shape, generator=gen(seed)).to(dtype).cuda()


def close(out, ref, a, big, D, weight_u, out_u=2.0 ** -8):
    tol = out_u * np.abs(ref) + (weight_u + 4 * D * 2.0 ** -24 * big + 2.0 ** -14) * a + 1e-30
    err = np.abs(np64(out) - ref)
    assert np.all(err <= tol), float((err / tol).max())


def close_lse(lse, ref, big, D):
    got = np64(lse)
    none = np.isneginf(ref)
    assert np.array_equal(np.isneginf(got), none)
    fin = ~none
    assert np.all(np.abs(got[fin] - ref[fin]) <= 2 * D * 2.0 ** -24 * big + 2.0 ** -20 * (1 + np.abs(ref[fin])))


# -------------------------------------------------------------------------------- plan
def _plan_inputs(new, lens, P, M, spare, seed):
    g = np.random.default_rng(seed)
    have = [-(-x // P) for x in lens]
    need = [max(0, -(-(x + y) // P) - h) for x, y, h in zip(lens, new, have)]
    ids = g.permutation(sum(have) + sum(need) + spare)
    table, at = np.full((len(lens), M), -1), 0
    for b, h in enumerate(have):
        table[b, :h] = ids[at:at + h]
        at += h
    free = ids[at:]
    return table, np.concatenate([free, np.zeros(len(ids) - len(free), np.int64)]), len(free)


PLANS = [  # lens, new, P
    ([0], [1], 16), ([15, 16, 17, 0], [1, 1, 1, 0], 16), ([0, 0, 0], [0, 0, 0], 64),
    ([5] * 33, [1] * 33, 64), ([0, 100, 127, 128, 0], [700, 0, 1, 0, 129], 128),
    (list(range(0, 1200, 2)), [(7 * i) % 50 for i in range(600)], 32),
    ([0], [40000], 16), ([3000, 0], [0, 20011], 64), ([i % 33 for i in range(5000)], [1] * 5000, 16),
    ([0] * 8192, [0] * 8000 + [1] * 192, 16)]


@cuda
@pytest.mark.parametrize("case", range(len(PLANS)))
@pytest.mark.parametrize("inplace", [False, True])
def test_plan_matches_the_definition(case, inplace):
    lens, new, P = PLANS[case]
    M = max(1, max(-(-(a + b) // P) for a, b in zip(lens, new))) + 1
    table, free, nf = _plan_inputs(new, lens, P, M, 2, case)
    rows = sum(new) + 5
    cu, ref_rows, lens2, left, table2 = OP.plan(new, lens, table, free, nf, P, rows)
    t, ln, n = i32(table), i32(lens), i32([nf])
    lo, no = (ln, n) if inplace else (torch.full_like(ln, -7), torch.full_like(n, -7))
    flags = i32([0])
    for _ in range(1 if inplace else 2):                    # repeatable when not in place
        p = rkv.page_plan(i32(new), ln, t, i32(free), n, P, rows, lo, no, flags=flags)
        assert p.cu_rows.tolist() == cu and lo.tolist() == lens2 and no.tolist() == [left]
        assert np.array_equal(t.cpu().numpy(), table2)
        got = torch.stack([p.row_seq, p.row_pos, p.row_slot]).cpu().numpy().T
        assert np.array_equal(got[:len(ref_rows)], np.array(ref_rows).reshape(-1, 3))
        assert np.all(got[len(ref_rows):] == -1)
    assert flags.item() == 0
    if not inplace:
        assert ln.tolist() == lens and n.tolist() == [nf]


@cuda
@pytest.mark.parametrize("why", ["rows", "pages", "table", "negative", "negative_len", "free"])
def test_plan_that_does_not_fit_changes_nothing(why):
    lens, new, P, M = [10, 20, 0], [30, 0, 50], 16, 4
    table, free, nf = _plan_inputs(new, lens, P, M, 0, 1)
    rows, bit = 80, rkv.FLAG_NO_SPACE
    if why == "rows":
        rows = 79
    elif why == "pages":
        nf -= 1
    else:
        bit = rkv.FLAG_BAD_INDEX
        if why == "table":
            new[2] = 65
        elif why == "negative":
            new[1] = -1
        elif why == "negative_len":
            lens[1] = -3
        else:
            nf = len(free) + 1
    for inplace in (False, True):
        t, ln, n, flags = i32(table), i32(lens), i32([nf]), i32([0])
        lo, no = (ln, n) if inplace else (torch.full_like(ln, -7), torch.full_like(n, -7))
        p = rkv.page_plan(i32(new), ln, t, i32(free), n, P, rows, lo, no, flags=flags)
        assert flags.item() == bit
        assert p.cu_rows.tolist() == [0] * 4 and lo.tolist() == lens and no.tolist() == [nf]
        assert np.array_equal(t.cpu().numpy(), table)
        assert torch.all(p.row_seq == -1) and torch.all(p.row_pos == -1) and torch.all(p.row_slot == -1)


@cuda
def test_plan_of_the_largest_row_maps():
    """max_rows up to 2^31 - 1 (26 GB of maps): rows are counted without a sign, so that none
    lands before the maps and every one past the total is -1."""
    lens, new, P = [5, 0, 40], [30, 7, 100000], 16
    table, free, nf = _plan_inputs(new, lens, P, 7000, 2, 3)
    cu, ref_rows, lens2, left, table2 = OP.plan(new, lens, table, free, nf, P, 2 ** 31 - 1)
    t, ln, n, flags = i32(table), i32(lens), i32([nf]), i32([0])
    p = rkv.page_plan(i32(new), ln, t, i32(free), n, P, 2 ** 31 - 1, flags=flags)
    assert flags.item() == 0 and p.cu_rows.tolist() == cu and ln.tolist() == lens2 and n.item() == left
    assert np.array_equal(t.cpu().numpy(), table2)
    for x, want in zip((p.row_seq, p.row_pos, p.row_slot), np.array(ref_rows).T):
        assert x.shape == (2 ** 31 - 1,) and np.array_equal(x[:cu[-1]].cpu().numpy(), want)
        assert all((c == -1).all().item() for c in x[cu[-1]:].split(1 << 28))
    del p, x
    torch.cuda.empty_cache()


@cuda
def test_release_matches_the_definition_and_refuses_what_does_not_fit():
    g = np.random.default_rng(5)
    lens = [int(x) for x in g.integers(0, 300, size=700)]
    fin = [int(x) for x in g.integers(0, 3, size=700)]
    table, free, nf = _plan_inputs([0] * 700, lens, 16, 20, 9, 6)
    l2, t2, f2, n2 = OP.release(fin, lens, table, free, nf, 16)
    t, ln, f, n, flags = i32(table), i32(lens), i32(free), i32([nf]), i32([0])
    rkv.page_release(i32(fin), ln, t, f, n, 16, flags=flags)
    assert ln.tolist() == l2 and n.item() == n2 and flags.item() == 0
    assert np.array_equal(t.cpu().numpy(), t2) and f[:n2].tolist() == [int(x) for x in f2[:n2]]
    for bad in ("list", "length"):
        t, ln, f, n, flags = i32(table), i32(lens), i32(free), i32([nf]), i32([0])
        if bad == "list":
            n.fill_(len(free) - n2 + nf + 1)
        else:
            ln[fin.index(1)] = 16 * 20 + 1
        before = [x.clone() for x in (t, ln, f, n)]
        rkv.page_release(i32(fin), ln, t, f, n, 16, flags=flags)
        assert flags.item() == (rkv.FLAG_NO_SPACE if bad == "list" else rkv.FLAG_BAD_INDEX)
        assert all(torch.equal(x, y) for x, y in zip(before, (t, ln, f, n)))


@cuda
@pytest.mark.parametrize("room", ["much", "just", "too little"])
def test_release_leaves_out_entries_that_are_no_page(room):
    """Entries outside the pages are flagged and never reach the free list, nor a later plan;
    the list needs room for the pages that are there alone."""
    g = np.random.default_rng(7)
    lens = [int(x) for x in g.integers(0, 3000, size=60)]
    fin = [int(x) for x in g.integers(0, 2, size=60)]
    table, free, nf = _plan_inputs([0] * 60, lens, 16, 190, 40, 8)
    num = len(free)
    for b in range(60):
        if lens[b] > 600:
            table[b, [0, 7, 36, 37]] = -1, num, 10 ** 9, -2 ** 31
    t2, l2, good = table.copy(), list(lens), []
    for b in range(60):
        if fin[b]:
            n = -(-lens[b] // 16)
            good += [int(x) for x in table[b, :n] if 0 <= x < num]
            t2[b, :n], l2[b] = -1, 0
    assert len(good) < sum(-(-n // 16) for n, x in zip(lens, fin) if x)
    nf = {"much": nf, "just": num - len(good), "too little": num - len(good) + 1}[room]
    had = [int(x) for x in g.integers(0, num, size=nf)]
    f = torch.full((num,), -9, dtype=torch.int32, device="cuda")
    f[:nf] = i32(had)
    t, ln, n, flags = i32(table), i32(lens), i32([nf]), i32([0])
    before = [x.clone() for x in (t, ln, f, n)]
    rkv.page_release(i32(fin), ln, t, f, n, 16, flags=flags)
    if room == "too little":
        assert flags.item() == rkv.FLAG_NO_SPACE
        assert all(torch.equal(x, y) for x, y in zip(before, (t, ln, f, n)))
        return
    assert flags.item() == rkv.FLAG_BAD_INDEX
    want = had + good
    assert n.item() == len(want) and f[:len(want)].tolist() == want
    assert ln.tolist() == l2 and np.array_equal(t.cpu().numpy(), t2)
    flags.zero_()
    p = rkv.page_plan(i32([16 * len(good)]), i32([0]), i32(np.full((1, num), -1)), f, n, 16, 16 * len(good), flags=flags)
    assert flags.item() == 0 and (p.row_slot >= 0).all()


@cuda
def test_release_of_many_pages():
    """More pages than a pass of the kernel takes, from sequences of all lengths."""
    g = np.random.default_rng(9)
    lens = [int(x) for x in g.integers(0, 40, size=8192)]
    lens[100], lens[101], lens[8191] = 130000, 0, 64000
    fin = [int(x) for x in g.integers(0, 3, size=8192)]
    fin[100] = fin[8191] = 1
    M, P = -(-130000 // 16), 16
    have = [-(-x // P) for x in lens]
    ids, at = g.permutation(sum(have) + 9), np.concatenate([[0], np.cumsum(have)])
    t = torch.full((8192, M), -1, dtype=torch.int32, device="cuda")
    for b in range(8192):
        t[b, :have[b]] = i32(ids[at[b]:at[b + 1]])
    f = torch.full((len(ids),), -9, dtype=torch.int32, device="cuda")
    f[:9] = i32(ids[at[-1]:])
    want = [int(x) for x in ids[at[-1]:]] + [int(x) for b in range(8192) if fin[b] for x in ids[at[b]:at[b + 1]]]
    ln, n, flags = i32(lens), i32([9]), i32([0])
    rkv.page_release(i32(fin), ln, t, f, n, P, flags=flags)
    assert flags.item() == 0 and n.item() == len(want) and f[:len(want)].tolist() == want
    assert ln.tolist() == [0 if fin[b] else lens[b] for b in range(8192)]
    left = (t >= 0).sum(1).tolist()
    assert left == [0 if fin[b] else have[b] for b in range(8192)]


# ------------------------------------------------------------------------------ append
def _f8(codes):
    return np64(codes.view(torch.float8_e4m3fn).float())


def _cache(num, N, P, D, seed):
    """Pages of random codes (no NaN) and small scales."""
    g = gen(seed)
    c = torch.randn((2, num, N, P, D), generator=g).to(torch.float8_e4m3fn).view(torch.uint8).cuda()
    s = torch.exp2(torch.randint(-9, -5, (2, num, N), generator=g).float()).cuda()
    return c[0], c[1], s[0], s[1]


@cuda
@pytest.mark.parametrize("P,D,dtype", [(16, 64, torch.bfloat16), (16, 128, torch.float32), (32, 128, torch.bfloat16),
                                       (64, 128, torch.bfloat16), (64, 64, torch.float32), (128, 128, torch.float32),
                                       (128, 64, torch.bfloat16)])
@pytest.mark.parametrize("what", ["decode", "mixed", "prompt", "few"])
def test_append_matches_the_definition(P, D, dtype, what):
    N = 9 if what == "few" else 3
    old = {"decode": [0, 5, P - 1, P, 3 * P + 7], "mixed": [0, 5, P, 0, 2 * P - 1, 9], "prompt": [0],
           "few": [0, 7, P - 3, 2 * P, 1] + [P] * 20}[what]
    new = {"decode": [1] * 5, "mixed": [3 * P + 1, 1, 0, P, 2 * P + 2, 0], "prompt": [5 * P + 3],
           "few": [2 * P // 3, 0, 9, 3, 1] + [0] * 20}[what]
    lens, cu = [a + b for a, b in zip(old, new)], [0] + np.cumsum(new).tolist()
    M = max(-(-x // P) for x in lens) + 1
    table, _, _ = _plan_inputs([0] * len(lens), lens, P, M, 3, 11)
    num = int(table.max()) + 4
    k8, v8, ks, vs = _cache(num, N, P, D, 12)
    ref = [(_f8(k8), np64(ks)), (_f8(v8), np64(vs))]
    n = sum(new)
    kv = torch.randn((n + 2, 2 * N + 1, D), generator=gen(13)) * torch.exp2(
        torch.randint(-8, 4, (n + 2, 2 * N + 1, 1), generator=gen(14)).float())
    kv = kv.to(dtype).cuda()
    k, v = kv[:, :N], kv[:, N + 1:]                         # strided views; two rows too many
    flags = i32([0])
    rkv.page_append(k, v, k8, v8, ks, vs, i32(table), i32(lens), i32(cu), flags=flags)
    for x, codes, scale, (rc, rs) in ((k, k8, ks, ref[0]), (v, v8, vs, ref[1])):
        OP.append(np64(x), rc, rs, table.tolist(), lens, cu, P)
        assert np.array_equal(np64(scale), rs)
        assert np.array_equal(_f8(codes), rc)
    assert flags.item() == 0


@cuda
def test_append_of_zeros_infinities_and_nan():
    P, N, D = 16, 2, 64
    x = torch.zeros((3, N, D))
    x[1, 0, 5], x[1, 0, 6], x[2, 0, 7], x[2, 0, 8] = math.inf, -math.inf, math.nan, 3.0
    x[0, 1, 0] = 1e-30                                       # below the smallest scale's codes
    for dt in (torch.float32, torch.bfloat16):
        xx = x.to(dt).cuda()
        k8, v8, ks, vs = _cache(2, N, P, D, 15)
        rc, rs = _f8(k8), np64(ks)
        rkv.page_append(xx, xx, k8, v8, ks, vs, i32([[1]]), i32([3]), i32([0, 3]))
        OP.append(np64(xx), rc, rs, [[1]], [3], [0, 3], P)
        assert np.array_equal(np64(ks), rs) and np.array_equal(_f8(k8), rc, equal_nan=True)
        assert _f8(k8)[1, 0, 1, 5] == 448 and np.isnan(_f8(k8)[1, 0, 2, 7]) and rs[1, 1] == 2.0 ** -64


@cuda
def test_append_leaves_out_what_is_out_of_range():
    """Bad page ids, lengths past the table and offsets past the rows: those rows are left
    out and flagged, the others stored."""
    P, N, D = 16, 2, 64
    x = randn(6, N, D, seed=16)
    for case in ("id", "negative_id", "length", "rows", "offset"):
        k8, v8, ks, vs = _cache(4, N, P, D, 17)
        rc, rs = _f8(k8), np64(ks)
        table, lens, cu = [[0, 1], [2, 3], [1, 0]], [3, 18, 0], [0, 3, 6, 6]
        flags = i32([0])
        t2, l2, c2 = [list(r) for r in table], list(lens), list(cu)
        if case == "id":
            t2[0][0] = 4
        elif case == "negative_id":
            t2[0][0] = -1
        elif case == "length":
            l2[0] = 33
        elif case == "rows":
            c2[3] = 7                                       # more rows than the third length holds
        else:
            c2[0] = -2
        rkv.page_append(x, x, k8, v8, ks, vs, i32(t2), i32(l2), i32(c2), flags=flags)
        keep = [0, 0, 3, 3] if case != "rows" else cu[:2] + [6, 6]
        if case == "rows":
            OP.append(np64(x), rc, rs, table, lens, cu, P)
        else:
            OP.append(np64(x), rc, rs, table, [0, 18, 0], [3, 3, 6, 6], P)
        assert np.array_equal(np64(ks), rs) and np.array_equal(_f8(k8), rc), (case, keep)
        assert flags.item() == rkv.FLAG_BAD_INDEX


@cuda
def test_append_flags_rows_that_are_not_there():
    """Offsets past the rows: the rows that exist are stored."""
    P, N, D = 16, 2, 64
    x = randn(5, N, D, seed=18)
    for narrow in (False, True):                            # both kernels (by rows a sequence)
        B = 5 if narrow else 1
        k8, v8, ks, vs = _cache(3, N, P, D, 19)
        rc, rs = _f8(k8), np64(ks)
        flags = i32([0])
        rkv.page_append(x, x, k8, v8, ks, vs, i32([[1, 2]] * B), i32([9] + [0] * (B - 1)), i32([0] + [9] * B),
                        flags=flags)
        OP.append(np64(x), rc, rs, [[1, 2]] * B, [5] + [0] * (B - 1), [0] + [5] * B, P)
        assert np.array_equal(np64(ks), rs) and np.array_equal(_f8(k8), rc)
        assert flags.item() == rkv.FLAG_BAD_INDEX


# --------------------------------------------------------------------- page attention
def _paged(lens, N, P, D, seed, poison=True, spread=0):
    """Pages holding random K/V for sequences of these lengths; NaN codes and scales
    everywhere else.  Returns the library's tensors and the stored values in float64."""
    M = max(1, max(-(-x // P) for x in lens)) + 1
    table, _, _ = _plan_inputs([0] * len(lens), lens, P, M, 3, seed)
    num = int(table.max()) + 4
    k8, v8, ks, vs = _cache(num, N, P, D, seed + 1)
    if spread:
        ks *= torch.exp2(torch.randint(0, 3, ks.shape, generator=gen(seed + 2)).float()).cuda()
        vs *= torch.exp2(torch.randint(-spread, spread + 1, vs.shape, generator=gen(seed + 3)).float()).cuda()
    ks *= 8
    val = [_f8(c) * np64(s)[:, :, None, None] for c, s in ((k8, ks), (v8, vs))]
    if poison:
        used = torch.zeros((num, P), dtype=torch.bool, device="cuda")
        for b, n in enumerate(lens):
            for t in range(-(-n // P)):
                used[table[b, t], :min(P, n - t * P)] = True
        for c in (k8, v8):
            c.masked_fill_(~used[:, None, :, None], 0x7F)
        empty = ~used.any(1)
        ks[empty], vs[empty] = math.nan, math.inf
    return (k8, v8, ks, vs), i32(table), table, val


ATTEND = [  # lens, Hq, N, P, D
    ([1], 1, 1, 16, 128), ([0, 1, 2, 15, 16, 17], 8, 2, 16, 64), ([127, 128, 129, 0, 255], 28, 4, 64, 128),
    ([1000], 32, 8, 64, 128), ([300, 5, 77], 32, 2, 32, 128), ([513, 1, 64], 9, 1, 128, 128),
    ([700, 650], 12, 1, 16, 64), ([40] * 70, 5, 5, 32, 64), ([5000, 3, 2047], 14, 2, 64, 64),
    ([130] * 3, 24, 2, 128, 128), ([300, 5, 900], 24, 4, 64, 128), ([257, 0, 1500], 10, 2, 16, 64),
    ([129, 2000], 10, 1, 32, 128), ([640, 33, 1], 26, 2, 64, 64)]


@cuda
@pytest.mark.parametrize("case", range(len(ATTEND)))
def test_page_attention_matches_the_definition(case):
    lens, Hq, N, P, D = ATTEND[case]
    cache, table, tb, (kv, vv) = _paged(lens, N, P, D, 100 + case)
    q = randn(len(lens), Hq + 1, D, seed=200 + case)[:, 1:]             # a strided view
    lse = torch.empty((len(lens), Hq), device="cuda")
    flags = i32([0])
    sc = 1 / math.sqrt(D)
    out = rkv.page_attention(q, *cache, table, i32(lens), lse=lse, flags=flags)
    ref, rl, a, big = OP.page_attention(np64(q), kv, vv, tb, lens, P, sc)
    close(out, ref, a, big, D, 2.0 ** -11)
    close_lse(lse, rl, big, D)
    assert flags.item() == 0
    again = rkv.page_attention(q, *cache, table, i32(lens))
    assert torch.equal(again, out)                                       # no order of atomics


@cuda
@pytest.mark.parametrize("spread", [0, 10])
def test_page_attention_peaked_and_wide_scales(spread):
    """Large scores (one key takes nearly all), a growing maximum, and value scales that
    differ by 2^20 between pages."""
    lens, Hq, N, P, D = [900, 260], 16, 2, 16, 128
    cache, table, tb, (kv, vv) = _paged(lens, N, P, D, 300, spread=spread)
    for mult in (0.01, 6.0):
        q = randn(2, Hq, D, seed=301) * mult
        out = rkv.page_attention(q, *cache, table, i32(lens), scale=0.09)
        ref, _, a, big = OP.page_attention(np64(q), kv, vv, tb, lens, P, 0.09)
        # weights are held to 12 bits of the largest weight times page scale seen: the error of
        # an element is relative to the largest of its head and dimension's sums
        close(out, ref, a.max(axis=-1, keepdims=True) + 0 * a, big, D, 2.0 ** -11)


@cuda
def test_page_attention_leaves_out_bad_pages_and_cuts_lengths():
    lens, Hq, N, P, D = [100, 64, 40], 8, 2, 16, 128
    cache, table, tb, (kv, vv) = _paged(lens, N, P, D, 400, poison=False)
    q = randn(3, Hq, D, seed=401)
    t2, flags = table.clone(), i32([0])
    t2[0, 2], t2[1, 1], t2[2, 0] = -1, 10 ** 6, -5
    out = rkv.page_attention(q, *cache, t2, i32([100, 64, 10 ** 9]), flags=flags)
    assert flags.item() == rkv.FLAG_BAD_INDEX
    keep = [[0, 1, 3, 4, 5, 6], [0, 2, 3], list(range(1, t2.shape[1]))]
    for b, pages in enumerate(keep):
        ids = [int(t2[b, j]) for j in pages if 0 <= int(t2[b, j]) < kv.shape[0]]
        n = {0: 84, 1: 48, 2: 16 * len(ids)}[b]
        ref, _, a, big = OP.page_attention(np64(q[b:b + 1]), kv, vv, [ids], [n], P, 1 / math.sqrt(D))
        close(out[b:b + 1], ref, a, big, D, 2.0 ** -11)
    out = rkv.page_attention(q, *cache, table, i32([-4, 0, 40]), flags=flags)
    assert not out[:2].any() and out[2].any()


@cuda
def test_page_attention_nan_stays_with_its_head_and_sequence():
    lens, Hq, N, P, D = [140, 140], 8, 2, 64, 128
    cache, table, tb, (kv, vv) = _paged(lens, N, P, D, 500)
    q = randn(2, Hq, D, seed=501)
    clean = rkv.page_attention(q, *cache, table, i32(lens))
    q2 = q.clone()
    q2[0, 5, 3], q2[0, 1, 0] = math.nan, math.inf
    out = rkv.page_attention(q2, *cache, table, i32(lens))
    assert torch.isnan(out[0, 5]).all() and torch.isnan(out[0, 1]).all()
    same = torch.ones((2, Hq), dtype=torch.bool, device="cuda")
    same[0, 5] = same[0, 1] = False
    assert torch.equal(out[same], clean[same])
    cache[1][int(tb[1, 1]), 1, 7, 9] = 0x7F                              # a stored NaN of V, head 1
    out = rkv.page_attention(q, *cache, table, i32(lens))
    bad = torch.isnan(out)
    want = torch.zeros_like(bad)
    want[1, 4:, 9] = True
    assert torch.equal(bad, want) and torch.equal(out[~bad], clean[~bad])


# ------------------------------------------------- page attention beside a dominant key
def _softmax64(q, k, v, lens, scale):
    """q [B, G, D] against one key/value head's rows k, v [T, D], all in binary64 on the GPU.
    Returns what oracle.pages.page_attention does, as arrays."""
    o, a, lse, big = [], [], [], 0.0
    for b, n in enumerate(lens):
        s = scale * (q[b] @ k[:n].T)
        m = s.max(-1, keepdim=True).values
        w = torch.exp(s - m)
        l = w.sum(-1, keepdim=True)
        o.append(w @ v[:n] / l)
        a.append(w @ v[:n].abs() / l)
        lse.append((m + torch.log(l))[:, 0])
        big = max(big, scale * (q[b].abs() @ k[:n].abs().T).max().item())
    return [torch.stack(x).cpu().numpy() for x in (o, lse, a)] + [big]


def _sunk(T, B, G, P, D, at, mass, std, small, loud, seed):
    """B sequences of T positions that share their pages, one key/value head: scores of
    deviation `std`, of which the key at `at` takes `mass` of the weight; values of mean 0.5,
    2^-6 of that at the key if `small`.  loud: one other page's values are 2^8 times as large."""
    g = gen(seed)
    M = -(-T // P)
    page = torch.randperm(M, generator=g)
    kc = torch.randn((T, D), generator=g) * 16 * std
    kc[:, 0] = 0
    kc[at] = 0
    kc[at, 0] = 448
    vc = (torch.randn((T, D), generator=g) * 0.5 + 1) * 16
    if small:
        vc[at] /= 64
    codes = torch.full((2, M * P, D), 0x7F, dtype=torch.uint8)
    for i, c in enumerate((kc, vc)):
        codes[i, :T] = c.to(torch.float8_e4m3fn).view(torch.uint8)
    k8, v8 = (torch.empty((M, 1, P, D), dtype=torch.uint8) for _ in range(2))
    k8[page, 0], v8[page, 0] = codes[0].view(M, P, D), codes[1].view(M, P, D)
    ks, vs = torch.full((M, 1), 2.0 ** -4), torch.full((M, 1), 2.0 ** -5)
    if loud:
        vs[page[(at // P + M // 2) % M], 0] *= 256
    cache = [x.cuda() for x in (k8, v8, ks, vs)]
    val = [c.cuda()[page.cuda(), 0].view(torch.float8_e4m3fn).double() * s.cuda()[page.cuda()].double()[:, :, None]
           for c, s in ((k8, ks), (v8, vs))]
    k, v = (x.reshape(-1, D)[:T] for x in val)
    q = torch.randn((B, G, D), generator=g).to(torch.bfloat16).cuda()
    q[:, :, 0] = 0
    s = torch.einsum("bgd,td->bgt", q.double(), k) / math.sqrt(D)
    s[:, :, at] = -math.inf
    q[:, :, 0] = ((torch.logsumexp(s, -1) + math.log(mass / (1 - mass))) * math.sqrt(D) / 28).to(torch.bfloat16)
    return q, cache, page.to(torch.int32).repeat(B, 1).cuda(), k, v


SINK = [  # T, B, G, P, D, at, mass, std, small, loud
    (1000, 3, 4, 64, 128, 0, 0.9, 1.0, True, False), (1000, 160, 12, 16, 64, 500, 0.99, 1.0, False, False),
    (1000, 160, 8, 32, 128, 999, 0.5, 0.1, True, False), (16384, 1, 4, 64, 128, 0, 0.99, 1.0, True, False),
    (16384, 156, 4, 64, 128, 0, 0.9, 1.0, True, False), (16384, 156, 2, 16, 64, 8000, 0.99, 0.1, True, False),
    (16384, 156, 16, 128, 128, 0, 0.99, 1.0, True, False), (16384, 156, 9, 64, 64, 8191, 0.5, 0.0, True, False),
    (16384, 156, 7, 32, 128, 0, 0.9, 1.0, False, True), (16384, 156, 12, 64, 128, 300, 0.9, 0.1, True, True),
    (131072, 1, 4, 64, 128, 0, 0.9, 1.0, True, False), (131072, 156, 4, 64, 128, 0, 0.9, 1.0, True, False),
    (131072, 156, 4, 64, 128, 0, 0.99, 0.0, True, False), (131072, 156, 8, 32, 64, 65536, 0.99, 1.0, True, False),
    (131072, 156, 16, 64, 128, 0, 0.5, 0.1, True, False), (131072, 156, 10, 128, 64, 70001, 0.99, 0.1, False, False)]


@cuda
@pytest.mark.parametrize("case", range(len(SINK)))
def test_page_attention_keeps_the_weights_beside_a_dominant_key(case):
    """One key takes most of the weight, as in the long contexts of trained models; the many
    others, 2^-8 to 2^-24 of it each, are most of the result where its value is small.  The
    bound is that of any other input.  (156 sequences: a CTA weighs the whole of one against
    the key; 1 and 3: a CTA has a share of one.)"""
    T, B, G, P, D = SINK[case][:5]
    q, cache, table, k, v = _sunk(*SINK[case], seed=1400 + case)
    lse = torch.empty((B, G), device="cuda")
    flags = i32([0])
    out = rkv.page_attention(q, *cache, table, i32([T] * B), lse=lse, flags=flags)
    assert flags.item() == 0
    ref, rl, a, big = _softmax64(q.double(), k, v, [T] * B, 1 / math.sqrt(D))
    close(out, ref, a, big, D, 2.0 ** -11)
    close_lse(lse, rl, big, D)


@cuda
def test_page_attention_of_more_than_a_second_a_sequence():
    """Sequences (of the same few pages) that take a CTA longer than its bounded waits last: four
    of 4 10^8 positions for each CTA.  Equal scores: the sums are exact."""
    T, B, N, P, D = 400_000_000, 152, 4, 128, 64
    k8 = torch.zeros((64, N, P, D), dtype=torch.uint8, device="cuda")
    one = torch.ones((64, N), device="cuda")
    table = (torch.arange(-(-T // P), dtype=torch.int32, device="cuda") % 64).repeat(B, 1)
    lse, flags = torch.empty((B, N), device="cuda"), i32([0])
    out = rkv.page_attention(randn(B, N, D, seed=1450), k8, k8, one, one, table, i32([T] * B), lse=lse, flags=flags)
    assert flags.item() == 0 and not out.any()
    assert torch.all((lse.double() - math.log(T)).abs() <= 2.0 ** -20 * math.log(T))
    del table
    torch.cuda.empty_cache()


# ------------------------------------------------------------------- prompt attention
PROMPT = [  # lq, lk, Hq, N, D
    ([1], [1], 1, 1, 128), ([1, 2, 3], [1, 2, 3], 4, 2, 64), ([77], [77], 32, 8, 128),
    ([128, 0, 129, 1, 127], [128, 0, 129, 1, 127], 14, 2, 128), ([300, 45], [300, 45], 3, 3, 64),
    ([260], [700], 8, 2, 128), ([5, 1, 130], [400, 257, 130], 7, 1, 64), ([200, 10], [60, 0], 4, 1, 128),
    ([33] * 9, [33] * 9, 5, 1, 128), ([513], [513], 2, 1, 128), ([100, 20], [0, 300], 4, 2, 64),
    ([300], [5000], 2, 1, 128), ([1], [9001], 7, 1, 64), ([100, 0, 64, 300], [0, 90, 3000, 700], 6, 2, 128),
    ([129, 1, 1, 1], [640, 2000, 1, 300], 3, 1, 64), ([1000], [1000], 5, 1, 64),
    ([100, 0, 64, 200], [0, 90, 9000, 7000], 6, 2, 128), ([128, 0, 257], [9128, 300, 5000], 2, 2, 64)]


def _cu(lens):
    return [0] + np.cumsum(lens).tolist()


@cuda
@pytest.mark.parametrize("case", range(len(PROMPT)))
def test_prompt_attention_matches_the_definition(case):
    lq, lk, Hq, N, D = PROMPT[case]
    cq, ck = _cu(lq), _cu(lk)
    pad = 7                                                  # rows behind the last sequence
    q = randn(cq[-1] + pad, Hq, D, seed=600 + case)
    kv = randn(ck[-1] + pad, 2 * N, D, seed=700 + case) * 2
    kv[ck[-1]:] = math.nan
    q[cq[-1]:] = math.inf
    k, v = kv[:, :N], kv[:, N:]
    out = torch.full((cq[-1] + pad, Hq, D), 5.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((cq[-1] + pad, Hq), 5.0, device="cuda")
    flags = i32([0])
    got = rkv.prompt_attention(q, k, v, i32(cq), i32(ck), out=out, lse=lse, flags=flags)
    assert got is out and flags.item() == 0
    ref, rl, a, big = OP.prompt_attention(np64(q[:cq[-1]]), np64(k[:ck[-1]]), np64(v[:ck[-1]]), cq, ck,
                                          1 / math.sqrt(D))
    close(out[:cq[-1]], ref, a, big, D, 2.0 ** -8)
    close_lse(lse[:cq[-1]], rl, big, D)
    assert torch.all(out[cq[-1]:] == 5.0) and torch.all(lse[cq[-1]:] == 5.0)


@cuda
@pytest.mark.parametrize("layout", ["packed", "heads_first", "fused"])
def test_prompt_attention_layouts(layout):
    T, Hq, N, D = 200, 6, 2, 128
    q, k, v = randn(T, Hq, D, seed=801), randn(T, N, D, seed=802), randn(T, N, D, seed=803)
    base = rkv.prompt_attention(q, k, v, i32([0, 150, T]))
    out = None
    if layout == "heads_first":
        q, k, v = (x.transpose(0, 1).contiguous().transpose(0, 1) for x in (q, k, v))
        out = torch.empty((Hq, T, D), dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    elif layout == "fused":
        x = torch.cat([q, k, v, q[:, :1]], dim=1)
        q, k, v = x[:, :Hq], x[:, Hq:Hq + N], x[:, Hq + N:Hq + 2 * N]
    assert torch.equal(rkv.prompt_attention(q, k, v, i32([0, 150, T]), out=out), base)
    # a batch of the same rows, one head's keys for all heads of a group
    one = rkv.prompt_attention(q, k[:, :1], v[:, :1], i32([0, 150, T]))
    assert torch.equal(one[:, :3], base[:, :3])


@cuda
def test_prompt_attention_keeps_sequences_apart():
    """NaN and infinities in one sequence leave the others' bits as they are, and large
    scores neither overflow nor lose rows."""
    lens, Hq, N, D = [70, 100, 150], 4, 2, 128
    cu = _cu(lens)
    q, k, v = randn(320, Hq, D, seed=811), randn(320, N, D, seed=812), randn(320, N, D, seed=813)
    base = rkv.prompt_attention(q, k, v, i32(cu))
    for t in (q, k, v):
        bad = t.clone()
        bad[70:170:7] = math.nan
        bad[75:170:9] = math.inf
        args = [bad if x is t else x for x in (q, k, v)]
        out = rkv.prompt_attention(*args, i32(cu))
        assert torch.equal(out[:70], base[:70]) and torch.equal(out[170:], base[170:])
    k2 = k.clone()
    k2[40:] = math.nan                                       # keys that no earlier row sees
    assert torch.equal(rkv.prompt_attention(q, k2, v, i32(cu))[:40], base[:40])
    big = rkv.prompt_attention(q * 64, k * 16, v, i32(cu))
    ref, _, a, s = OP.prompt_attention(np64(q * 64), np64(k * 16), np64(v), cu, cu, 1 / math.sqrt(D))
    close(big, ref, a, s, D, 2.0 ** -8)


STRAY = [  # lq, lk, Hq, N, D: whole pairs, shares, more pairs than CTAs; a second sequence of clean rows
    (300, 300, 4, 2, 128), (300, 300, 3, 3, 64), (200, 6000, 4, 2, 128), (130, 7001, 7, 1, 64),
    (500, 640, 80, 40, 64), (400, 400, 100, 50, 128), (90, 50, 4, 2, 128), (257, 129, 2, 1, 64)]


@cuda
@pytest.mark.parametrize("case", range(len(STRAY)))
@pytest.mark.parametrize("inplace", [False, True])
def test_prompt_attention_hidden_values_have_no_effect(case, inplace):
    """NaN and infinities of V reach the rows that see them and no row before: one element, a
    whole row, all rows from one on (a padded prompt), both infinities of one channel."""
    lq, lk, Hq, N, D = STRAY[case]
    cq, ck = [0, lq, lq + 40], [0, lk, lk + 40]
    q = randn(cq[-1], Hq, D, seed=1500 + case)
    k, v0 = randn(ck[-1], N, D, seed=1520 + case), randn(ck[-1], N, D, seed=1540 + case)
    clean = rkv.prompt_attention(q, k, v0, i32(cq), i32(ck))
    few = min(Hq, 6)                                        # heads that are checked one by one
    heads = sorted({*range(few), Hq - 1})
    first = max(0, lk - lq)                                 # (the first keys that some query does not see)
    for what in ("element", "row", "rest", "infinities"):
        v = v0.clone()
        if what == "element":
            v[first + (lk - first) // 2, 0, 5], v[lk - 1, N - 1, D - 1] = math.nan, math.inf
        elif what == "row":
            v[first + (lk - first) // 3], v[lk - 2] = math.nan, -math.inf
        elif what == "rest":
            v[first + (lk - first) // 2:lk] = math.nan
        else:
            v[first + (lk - first) // 4, :, 3], v[lk - 3, :, 3] = math.inf, -math.inf
            v[lk - 20, :, 7] = -math.inf
        args, flags = q.clone(), i32([0])
        out = rkv.prompt_attention(args, k, v, i32(cq), i32(ck), out=args if inplace else None, flags=flags)
        assert flags.item() == 0 and torch.equal(out[lq:], clean[lq:])
        for h in heads:
            n = slice(h // (Hq // N), h // (Hq // N) + 1)
            ref, _, a, big = OP.prompt_attention(np64(q[:lq, h:h + 1]), np64(k[:lk, n]), np64(v[:lk, n]), [0, lq],
                                                 [0, lk], 1 / math.sqrt(D))
            got, fin = np64(out[:lq, h:h + 1]), np.isfinite(ref)
            assert np.array_equal(got[~fin], ref[~fin], equal_nan=True), what
            close(torch.from_numpy(got[fin]), ref[fin], a[fin], big, D, 2.0 ** -8)
        bad = ~torch.isfinite(out)
        same = torch.isfinite(clean) & ~bad                  # of all heads: what is finite is what it was, nearly
        assert torch.allclose(out[same].float(), clean[same].float(), rtol=2 ** -6, atol=2 ** -6)


@cuda
@pytest.mark.parametrize("lk", [300, 6000])                 # whole pairs, and in shares
@pytest.mark.parametrize("D", [64, 128])
def test_prompt_attention_bits_are_the_sequences_own(lk, D):
    """The next sequence's queries lie in the same tile of rows: whatever they are, and also
    where they are overwritten meanwhile, the first one's bits are the same."""
    lq, T, Hq, N = 70, 190, 6, 2
    cq, ck = i32([0, lq, T]), i32([0, lk, lk + 200])
    q, k, v = randn(T, Hq, D, seed=841), randn(lk + 200, N, D, seed=842) * 2, randn(lk + 200, N, D, seed=843)
    base = rkv.prompt_attention(q, k, v, cq, ck)
    for rows in (math.nan, math.inf, -1e30, 1e4, 0.0):
        other = q.clone()
        other[lq:] = rows
        assert torch.equal(rkv.prompt_attention(other, k, v, cq, ck)[:lq], base[:lq]), rows
    loud = q.clone()
    loud[lq:] *= 300
    assert torch.equal(rkv.prompt_attention(loud, k, v, cq, ck)[:lq], base[:lq])
    assert torch.equal(rkv.prompt_attention(q, k, v, cq, ck, out=q), base)


@cuda
@pytest.mark.parametrize("scale", [1e-30, 1e-20, 2e-3])
def test_small_scales_weigh_alike(scale):
    """Scores that are next to nothing: the mean of what a row sees, masked keys left out."""
    T, Hq, N, D = 150, 4, 2, 64
    q, k, v = randn(T, Hq, D, seed=816), randn(T, N, D, seed=817), randn(T, N, D, seed=818)
    out = rkv.prompt_attention(q, k, v, i32([0, 70, T]), scale=scale)
    ref, _, a, big = OP.prompt_attention(np64(q), np64(k), np64(v), [0, 70, T], [0, 70, T], scale)
    close(out, ref, a, big, D, 2.0 ** -8)
    cache, table, tb, (kv, vv) = _paged([130, 7], 2, 32, D, 819)
    out = rkv.page_attention(q[:2], *cache, table, i32([130, 7]), scale=scale)
    ref, _, a, big = OP.page_attention(np64(q[:2]), kv, vv, tb, [130, 7], 32, scale)
    close(out, ref, a, big, D, 2.0 ** -11)


@cuda
def test_prompt_attention_cuts_bad_offsets():
    T, Hq, N, D = 40, 2, 1, 64
    q, k, v = randn(T, Hq, D, seed=821), randn(T, N, D, seed=822), randn(T, N, D, seed=823)
    for cu in ([0, 30, 10 ** 6], [-5, 20, 40], [0, 30, 20]):
        flags, out = i32([0]), torch.zeros((T, Hq, D), dtype=torch.bfloat16, device="cuda")
        rkv.prompt_attention(q, k, v, i32(cu), out=out, flags=flags)
        assert flags.item() == rkv.FLAG_BAD_INDEX
    assert torch.equal(out[:30], rkv.prompt_attention(q, k, v, i32([0, 30]))[:30])


@cuda
def test_prompt_attention_broadcast_rows_and_heads_in_place_and_without_keys():
    cu = i32([0, 100, 150])
    q, k, v = randn(150, 8, 128, seed=831), randn(150, 4, 128, seed=832), randn(150, 4, 128, seed=833)
    base = rkv.prompt_attention(q, k, v, cu)
    one = rkv.prompt_attention(q, k[:, :1].expand(150, 4, 128), v[:, :1].expand(150, 4, 128), cu)
    assert torch.equal(one, rkv.prompt_attention(q, k[:, :1], v[:, :1], cu))
    row = rkv.prompt_attention(q[:1].expand(150, 8, 128), k, v, cu)
    assert torch.equal(row, rkv.prompt_attention(q[:1].repeat(150, 1, 1), k, v, cu))
    q2 = q.clone()
    assert rkv.prompt_attention(q2, k, v, cu, out=q2) is q2 and torch.equal(q2, base)
    assert not rkv.prompt_attention(q[:5], k[:0], v[:0], i32([0, 5]), i32([0, 0])).any()
    assert rkv.prompt_attention(q[:0], k, v, i32([0, 0]), i32([0, 150])).shape == (0, 8, 128)


@cuda
@pytest.mark.parametrize("B", [6, 32, 33])
def test_prompt_attention_of_more_pairs_than_ctas(B):
    """Every CTA takes several pairs, of sequences of all lengths, with fewer and with more keys
    than queries, among them empty ones."""
    g = np.random.default_rng(900 + B)
    top = 6000 // B
    lq = np.where(g.random(B) < 0.15, 0, g.integers(1, top, size=B))
    lq[0] = top
    lk = np.where(g.random(B) < 0.5, lq, g.integers(0, 2 * top, size=B))
    Hq, N, D = 30, 10, 64
    assert ((-(-lq // 128) * 3 + 1) // 2).sum() * N > 2 * 160
    cq, ck = _cu(lq.tolist()), _cu(lk.tolist())
    q = randn(cq[-1], Hq, D, seed=861)
    k, v = randn(ck[-1], N, D, seed=862), randn(ck[-1], N, D, seed=863)
    flags = i32([0])
    out = rkv.prompt_attention(q, k, v, i32(cq), i32(ck), flags=flags)
    assert flags.item() == 0
    ref, _, a, big = OP.prompt_attention(np64(q), np64(k), np64(v), cq, ck, 0.125)
    close(out, ref, a, big, D, 2.0 ** -8)


@cuda
def test_prompt_attention_of_more_than_a_second_an_item():
    """Pairs that take a CTA longer than its bounded waits last: 3 for each CTA, one query row
    over 1.2 10^8 keys (the keys of one head, read by all)."""
    T, N = 120_000_000, 456
    q = randn(1, 2 * N, 64, seed=871)
    kv = torch.zeros((T, 1, 64), dtype=torch.bfloat16, device="cuda")
    lse, flags = torch.empty((1, 2 * N), device="cuda"), i32([0])
    out = rkv.prompt_attention(q, kv.expand(T, N, 64), kv.expand(T, N, 64), i32([0, 1]), i32([0, T]), lse=lse,
                               flags=flags)
    assert flags.item() == 0 and not out.any()
    assert torch.all((lse.double() - math.log(T)).abs() <= 2.0 ** -20 * math.log(T))
    del kv
    torch.cuda.empty_cache()


@cuda
@pytest.mark.parametrize("B", [33, 700, 8192])
def test_many_short_sequences(B):
    """Batches past a warp, past a block and at the limit, half the sequences empty: prompts of
    up to two tokens, and decode steps over up to 39."""
    g = np.random.default_rng(B)
    lens = g.integers(0, 3, size=B).tolist()
    cu = _cu(lens)
    q, k, v = randn(cu[-1], 4, 64, seed=841), randn(cu[-1], 2, 64, seed=842), randn(cu[-1], 2, 64, seed=843)
    flags = i32([0])
    out = rkv.prompt_attention(q, k, v, i32(cu), flags=flags)
    ref, _, a, big = OP.prompt_attention(np64(q), np64(k), np64(v), cu, cu, 0.125)
    close(out, ref, a, big, 64, 2.0 ** -8)
    lens = g.integers(0, 40, size=B)
    lens[g.integers(0, B, size=B // 2)] = 0
    cache, table, tb, (kv, vv) = _paged(lens.tolist(), 2, 16, 64, 850)
    q = randn(B, 4, 64, seed=851)
    out = rkv.page_attention(q, *cache, table, i32(lens), flags=flags)
    ref, _, a, big = OP.page_attention(np64(q), kv, vv, tb, lens.tolist(), 16, 0.125)
    close(out, ref, a, big, 64, 2.0 ** -11)
    assert flags.item() == 0


# --------------------------------------------------------------------- the run together
@cuda
def test_serving_loop_with_graph_replay():
    """Prompts planned, attended and stored, decode steps captured once and replayed, a
    request released and its slot reused: every step against the definition over all rows
    that the requests have had."""
    B, Hq, N, D, P = 3, 8, 2, 128, 16
    table = rkv.PageTable(B, 12, 24, P)
    cache = rkv.PagedCache(N, D, 24, P)
    for t in (cache.k8, cache.v8):
        t.fill_(0x7F)
    hist = [[] for _ in range(B)]                            # (k, v) rows of each sequence
    step_new = [40, 0, 33]

    def check(o, q):
        kv = [np.concatenate(h) if h else np.zeros((0, 2, N, D)) for h in hist]
        ks = np64(cache.k_scale)
        for b in range(B):
            n = len(kv[b])
            assert n == table.seq_len[b].item()
            if n == 0:
                assert not o[b].any()
                continue
            ids = table.block_table[b, :-(-n // P)].cpu().numpy()
            val = [_f8(c)[ids] * np64(s)[ids][:, :, None, None] for c, s in
                   ((cache.k8, cache.k_scale), (cache.v8, cache.v_scale))]
            rows = [x.transpose(0, 2, 1, 3).reshape(-1, N, D)[:n] for x in val]
            for i in range(2):                               # stored rows: two roundings at most
                s = (ks if i == 0 else np64(cache.v_scale))[ids].repeat(P, axis=0)[:n, :, None]
                assert np.all(np.abs(rows[i] - kv[b][:, i]) <=
                              2 * np.maximum(np.abs(kv[b][:, i]) * 1.07 * 2.0 ** -4, s * 2.0 ** -10))
            vals = [x for x in val]
            ref, _, a, big = OP.page_attention(np64(q[b:b + 1]), vals[0], vals[1], [list(range(len(ids)))], [n], P,
                                               1 / math.sqrt(D))
            close(o[b:b + 1], ref, a, big, D, 2.0 ** -11)

    def remember(k, v, cu):
        for b in range(B):
            a, c = cu[b], cu[b + 1]
            if c > a:
                hist[b].append(np.stack([np64(k[a:c]), np64(v[a:c])], axis=1))

    # prompts of sequences 0 and 2
    q, k, v = randn(80, Hq, D, seed=901), randn(80, N, D, seed=902), randn(80, N, D, seed=903)
    plan = table.plan(i32(step_new), 80)
    o = rkv.prompt_attention(q, k, v, plan.cu_rows, flags=table.flags)
    cache.append(k, v, table, plan)
    cu = plan.cu_rows.tolist()
    assert cu == [0, 40, 40, 73]
    ref, _, a, big = OP.prompt_attention(np64(q[:73]), np64(k[:73]), np64(v[:73]), cu, cu, 1 / math.sqrt(D))
    close(o[:73], ref, a, big, D, 2.0 ** -8)
    remember(k, v, cu)
    qd = randn(B, Hq, D, seed=904)
    check(cache.attend(qd, table), qd)

    # decode: captured once, replayed with new rows and lengths
    new, kd, vd = i32([1, 1, 1]), randn(B, N, D, seed=905), randn(B, N, D, seed=906)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        p = table.plan(new, B)
        cache.append(kd, vd, table, p)
        od = cache.attend(qd, table)
    for step in range(20):
        kd.copy_(randn(B, N, D, seed=1000 + step) * (1 + step % 3))
        vd.copy_(randn(B, N, D, seed=1100 + step))
        qd.copy_(randn(B, Hq, D, seed=1200 + step))
        new.copy_(i32([1, step % 2, 1]))
        graph.replay()
        remember(kd, vd, p.cu_rows.tolist())
        if step % 6 == 5:
            check(od, qd)

    # the first request ends; its slot takes another
    before = table.n_free.item()
    pages = -(-len(np.concatenate(hist[0])) // P)
    table.release(i32([1, 0, 0]))
    hist[0] = []
    assert table.n_free.item() == before + pages
    q, k, v = randn(50, Hq, D, seed=911), randn(50, N, D, seed=912), randn(50, N, D, seed=913)
    plan = table.plan(i32([50, 0, 0]), 64)
    cache.append(k, v, table, plan)
    remember(k, v, plan.cu_rows.tolist())
    check(cache.attend(qd, table), qd)
    assert table.flags.item() == 0


@cuda
def test_streams_and_calls_at_once():
    """Calls on two streams at once and a side stream's call: the results of calls alone."""
    lens = [3000, 17, 900]
    cache, table, _, _ = _paged(lens, 4, 64, 128, 1300)
    qs = [randn(3, 16, 128, seed=1301 + i) for i in range(6)]
    x = [randn(700, 8, 128, seed=1310 + i) for i in range(6)]
    cu, ln = i32([0, 300, 700]), i32(lens)
    alone = [(rkv.page_attention(q, *cache, table, ln), rkv.prompt_attention(t, t[:, :2], t[:, 2:4], cu))
             for q, t in zip(qs, x)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for i, (q, t) in enumerate(zip(qs, x)):
        s = streams[i % 2]
        got.append((rkv.page_attention(q, *cache, table, ln, stream=s),
                    rkv.prompt_attention(t, t[:, :2], t[:, 2:4], cu, stream=s)))
    torch.cuda.synchronize()
    for (a, b), (c, d) in zip(alone, got):
        assert torch.equal(a, c) and torch.equal(b, d)


# --------------------------------------------------------------------------- refusals
@cuda
def test_binding_refusals():
    """Shapes, types, strides, devices and streams that a call cannot use are refused before
    anything is launched; the library's own refusals arrive as RkvError."""
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    q, k = bf(6, 4, 64), bf(6, 2, 64)
    cu = i32([0, 6])
    ok = lambda **kw: rkv.prompt_attention(**{**dict(q=q, k=k, v=k, cu_q=cu), **kw})  # noqa: E731
    ok()
    odd = torch.zeros((6, 4, 67), dtype=torch.bfloat16, device="cuda")[:, :, :64]
    for bad in (dict(q=q.float()), dict(q=q[0]), dict(k=bf(6, 2, 128)), dict(v=bf(5, 2, 64)), dict(q=odd),
                dict(q=bf(6, 64, 4).transpose(1, 2)), dict(cu_q=cu.long()), dict(cu_q=cu[None]),
                dict(cu_k=i32([0, 3, 6])), dict(cu_q=cu.cpu()), dict(k=k.cpu()), dict(out=bf(6, 4, 128)),
                dict(lse=bf(6, 4)), dict(flags=i32([0, 0])), dict(scale=0.0), dict(scale=math.nan),
                dict(scale=math.inf), dict(scale=-1.0)):
        with pytest.raises(ValueError):
            ok(**bad)
    with pytest.raises(TypeError):
        ok(scale="x")
    with pytest.raises(AttributeError):
        ok(stream=7)
    with pytest.raises(rkv.RkvError) as e:
        ok(q=bf(6, 3, 64))                                   # 3 query heads over 2
    assert e.value.status == -1
    ok(q=odd[:1, :1], k=k[:, :1], v=k[:, :1], cu_q=i32([0, 1]), cu_k=i32([0, 6]))   # strides of one row, one head

    u8, f = torch.zeros((3, 2, 16, 64), dtype=torch.uint8, device="cuda"), torch.ones((3, 2), device="cuda")
    t, ln = i32([[0, 1], [2, 0]]), i32([1, 1])
    att = lambda **kw: rkv.page_attention(**{**dict(q=bf(2, 4, 64), k8=u8, v8=u8, k_scale=f, v_scale=f,  # noqa: E731
                                                    block_table=t, seq_len=ln), **kw})
    att()
    for bad in (dict(q=bf(3, 4, 64)), dict(q=bf(2, 4, 128)), dict(k8=u8.view(torch.int8)), dict(v8=u8[:2]),
                dict(k_scale=f.double()), dict(v_scale=f.t()), dict(block_table=t.long()), dict(seq_len=i32([1])),
                dict(block_table=t[0]), dict(out=bf(2, 4, 64).transpose(0, 1)), dict(lse=torch.zeros(8, device="cuda"))):
        with pytest.raises(ValueError):
            att(**bad)
    for bad in (dict(k8=u8[:, :, :8].contiguous(), v8=u8[:, :, :8].contiguous()), dict(q=bf(2, 34, 64))):
        with pytest.raises(rkv.RkvError):
            att(**bad)
    app = lambda **kw: rkv.page_append(**{**dict(k=bf(2, 2, 64), v=bf(2, 2, 64), k8=u8.clone(), v8=u8.clone(),  # noqa: E731
                                                 k_scale=f.clone(), v_scale=f.clone(), block_table=t, seq_len=ln,
                                                 cu_rows=i32([0, 1, 2])), **kw})
    app()
    for bad in (dict(v=bf(2, 2, 64).float()), dict(k=bf(2, 3, 64)), dict(k=bf(2, 2, 64).half(), v=bf(2, 2, 64).half()),
                dict(cu_rows=i32([0, 2])), dict(v=bf(3, 2, 64))):
        with pytest.raises(ValueError):
            app(**bad)
    pl = lambda **kw: rkv.page_plan(**{**dict(new_tokens=i32([1, 1]), seq_len=ln.clone(), block_table=t.clone(),  # noqa: E731
                                              free_blocks=i32([0, 1, 2]), n_free=i32([3]), block_tokens=16,
                                              max_rows=4), **kw})
    pl()
    for bad in (dict(new_tokens=i32([1])), dict(n_free=i32([3, 3])), dict(free_blocks=i32([[0]])),
                dict(seq_len_out=i32([1])), dict(n_free_out=i32([]))):
        with pytest.raises(ValueError):
            pl(**bad)
    with pytest.raises(rkv.RkvError):
        pl(block_tokens=20)
