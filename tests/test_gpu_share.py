"""GPU parity of the operators on pages that several sequences hold: forks, cuts and releases in
the table, compaction, copies in the caches, and stored rows gathered.  Every result is a whole
number, a copied byte or a product that bf16 holds: equal."""
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


def randn(*shape, seed, dtype=torch.bfloat16):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


# -------------------------------------------------------------------------------- fork
def _table(lens, P, M, spare, seed, share=0.0, pool=None):
    """Rows of random pages; with probability `share` a row begins with whole pages of an earlier
    one.  (table, free, n_free)"""
    g = np.random.default_rng(seed)
    B = len(lens)
    have = [-(-n // P) for n in lens]
    ids = g.permutation(sum(have) + spare if pool is None else pool)
    table, at = np.full((B, M), -1), 0
    for b in range(B):
        common = 0
        if b and g.random() < share:
            a = int(g.integers(b))
            common = int(g.integers(0, min(lens[a], lens[b]) // P + 1))
            table[b, :common] = table[a, :common]
        n = have[b] - common
        table[b, common:have[b]] = ids[at:at + n]
        at += n
    free = np.zeros(len(ids), np.int64)
    free[:len(ids) - at] = ids[at:]
    return table, free, len(ids) - at


def _run_fork(source, length, finished, lens, table, free, nf, P, inplace=True, flags=None):
    B, M = table.shape
    t, ln, f, n = i32(table), i32(lens), i32(free), i32([nf])
    flags = i32([0]) if flags is None else flags
    opt = lambda x: None if x is None else i32(x)  # noqa: E731
    to, lo, no = (t, ln, n) if inplace else (torch.full_like(t, -9), torch.full_like(ln, -9), torch.full_like(n, -9))
    for _ in range(1 if inplace else 2):                 # repeatable when not in place
        c = rkv.page_fork(opt(source), ln, t, f, n, P, length=opt(length), finished=opt(finished), block_table_out=to,
                          seq_len_out=lo, n_free_out=no, flags=flags)
    if not inplace:
        assert np.array_equal(t.cpu().numpy(), table) and ln.tolist() == list(lens) and n.item() == nf
    return to.cpu().numpy(), lo.tolist(), f.cpu().numpy(), no.item(), c, flags.item()


def _check_fork(source, length, finished, lens, table, free, nf, P, inplace):
    src = list(range(len(lens))) if source is None else list(source)
    if finished is not None:
        src = [-1 if x else s for s, x in zip(src, finished)]
    t2, l2, f2, n2, copies = OP.fork(src, length, lens, table, free, nf, P)
    t, ln, f, n, c, flags = _run_fork(source, length, finished, lens, table, free, nf, P, inplace)
    assert flags == 0 and ln == l2 and n == n2 and f.tolist() == [int(x) for x in f2]
    assert np.array_equal(t, t2)
    B = len(lens)
    want = [copies.get(b, (-1, -1, 0)) for b in range(B)]
    assert c.count is None and list(zip(c.src.tolist(), c.dst.tolist(), c.rows.tolist())) == want
    return copies, n2 - nf


def _random_fork(B, top, P, seed):
    g = np.random.default_rng(seed)
    lens = [int(x) for x in g.integers(0, top + 1, size=B)]
    source = [int(x) for x in g.integers(-1, B, size=B)]
    own = g.random(B) < 0.4
    source = [b if own[b] else source[b] for b in range(B)]
    length = []
    for b in range(B):
        n = lens[source[b]] if source[b] >= 0 else 9
        kind = g.integers(0, 4)
        length.append(-1 if kind == 0 else n if kind == 1 else n // P * P if kind == 2 else int(g.integers(0, n + 1)))
    finished = [int(x) for x in (g.random(B) < 0.15) * g.integers(1, 9, size=B)]
    return lens, source, length, finished


FORKS = [(1, 40, 16), (2, 0, 16), (3, 17, 16), (16, 300, 64), (33, 129, 32), (61, 1000, 16), (256, 600, 128),
         (700, 90, 16), (5, 20000, 16)]


@cuda
@pytest.mark.parametrize("case", range(len(FORKS)))
@pytest.mark.parametrize("share", [0.0, 0.7])
@pytest.mark.parametrize("inplace", [False, True])
def test_fork_matches_the_definition(case, share, inplace):
    B, top, P = FORKS[case]
    lens, source, length, finished = _random_fork(B, top, P, case + (100 if share else 0))
    M = -(-top // P) + 2
    table, free, nf = _table(lens, P, M, B + 3, case, share)
    args = (lens, table, free, nf, P, inplace)
    _check_fork(source, length, finished, *args)
    _check_fork(source, None, None, *args)
    _check_fork(None, [min(x, n) for x, n in zip(length, lens)], None, *args)
    _check_fork(None, None, finished, *args)
    _check_fork([(b + 1) % B for b in range(B)], None, None, *args)
    c, gone = _check_fork(None, None, None, *args)         # nothing asked: nothing done
    assert gone == 0 and (share or not c)
    _check_fork([-1] * B, None, None, *args)


@cuda
def test_fork_orders_what_it_frees_and_takes():
    """All rows let go of pages that many hold; begun pages of one row go to all others."""
    P, B = 16, 64
    lens = [P * 9 + 5] * B
    table = np.full((B, 12), -1)
    table[:, :9] = np.arange(9)[::-1]
    table[:, 9] = 9 + np.arange(B)[::-1]
    free = np.concatenate([np.arange(9 + B, 9 + 2 * B), np.zeros(9 + B, np.int64)])
    args = (lens, table, free, B, P)
    for inplace in (False, True):
        copies, gone = _check_fork([40] * B, None, None, *args, inplace)
        assert len(copies) == B - 1 and gone == 0          # 63 begun pages go, 63 copies come
        copies, gone = _check_fork([-1] * B, None, None, *args, inplace)
        assert gone == 9 + B and not copies
        copies, gone = _check_fork(None, [P * 3] * B, None, *args, inplace)
        assert gone == 6 + B and not copies
        copies, gone = _check_fork(None, [P * 3 + 1] * B, None, *args, inplace)
        assert gone == 5 + B - (B - 1) and sorted(copies) == list(range(1, B))
    # copies out of what the same call frees: no free page before it
    full = np.zeros(9 + B, np.int64)
    copies, gone = _check_fork([40] * B, None, None, lens, table, full, 0, P, True)
    assert len(copies) == B - 1 and gone == 0


@cuda
@pytest.mark.parametrize("inplace", [False, True])
def test_fork_of_the_largest_batch_and_of_long_rows(inplace):
    """8192 rows on a wide table, and rows of 20000 pages: every CTA of the cluster has work."""
    g = np.random.default_rng(1)
    lens = [int(x) for x in g.integers(0, 60, size=8192)]
    lens[77] = 16 * 300
    table, free, nf = _table(lens, 16, 301, 9000, 2, 0.3)
    source = [int(x) for x in g.integers(-1, 8192, size=8192)]
    _check_fork(source, None, None, lens, table, free, nf, 16, inplace)
    lens = [16 * 20000 - 3, 5, 16 * 19999 + 1]
    table, free, nf = _table(lens, 16, 20001, 20, 3, 0.9)
    _check_fork([2, 0, 0], [-1, 16 * 12345 + 7, -1], None, lens, table, free, nf, 16, inplace)


@cuda
def test_fork_in_a_pool_of_more_pages_than_shared_memory_takes():
    lens, source, length, finished = _random_fork(20, 400, 16, 4)
    table, free, nf = _table(lens, 16, 30, 60000, 5, 0.5)
    for inplace in (False, True):
        _check_fork(source, length, finished, lens, table, free, nf, 16, inplace)


@cuda
@pytest.mark.parametrize("why", ["source", "length", "above", "len", "table", "n_free", "space", "list"])
@pytest.mark.parametrize("inplace", [False, True])
def test_fork_that_does_not_fit_changes_nothing(why, inplace):
    lens, P, M = [40, 16, 33, 0], 16, 4
    table, free, nf = _table(lens, P, M, 3, 5)
    source, length, bit = [0, 1, 0, 0], [-1, -1, -1, 20], rkv.FLAG_BAD_INDEX
    if why == "source":
        source[2] = 4
    elif why == "length":
        length[3], lens[0] = 41, 40
    elif why == "above":
        source[1], length[1] = 1, 17
    elif why == "len":
        lens[1] = -2
    elif why == "table":
        lens[1] = P * M + 1
    elif why == "n_free":
        nf = len(free) + 1
    elif why == "space":
        source, nf, bit = [0, 1, 2, 0], 0, rkv.FLAG_NO_SPACE
    else:
        source, length, nf, bit = [0, 1, -1, -1], [-1, -1, -1, -1], len(free) - 2, rkv.FLAG_NO_SPACE
    t, ln, f, n, c, flags = _run_fork(source, length, None, lens, table, free, nf, P, inplace)
    assert flags == bit and np.array_equal(t, table) and ln == lens and n == nf and f.tolist() == free.tolist()
    assert c.src.tolist() == c.dst.tolist() == [-1] * 4 and c.rows.tolist() == [0] * 4


@cuda
def test_fork_keeps_entries_that_are_no_page():
    """Such an entry moves with its row, is flagged, and reaches neither list nor copies; of an
    id in a row twice one goes to the list."""
    P = 16
    table = np.array([[0, -7, 2, 99], [3, 10 ** 9, -1, -1], [4, 4, -1, -1], [-1] * 4])
    lens, free = [60, 20, 32, 0], [5, 6, 7, 8, 0, 0, 0, 0, 0, 0]
    for inplace in (False, True):
        t, ln, f, n, c, flags = _run_fork([-1, 1, -1, 1], None, None, lens, table, free, 4, P, inplace)
        assert flags == rkv.FLAG_BAD_INDEX and ln == [0, 20, 0, 20]
        assert t.tolist() == [[-1] * 4, [3, 10 ** 9, -1, -1], [-1] * 4, [3, 10 ** 9, -1, -1]]
        assert n == 7 and f[:7].tolist() == [5, 6, 7, 8, 0, 2, 4] and c.src.tolist() == [-1] * 4


@cuda
def test_fork_flags_a_free_entry_that_is_no_page():
    table, lens, free = np.array([[0, 1], [-1, -1]]), [20, 0], [2, 99, 3, 4]
    for inplace in (False, True):
        t, ln, f, n, c, flags = _run_fork([0, 0], None, None, lens, table, free, 2, 16, inplace)
        assert flags == rkv.FLAG_BAD_INDEX and t.tolist() == [[0, 1], [0, 99]] and c.dst.tolist() == [-1, 99]
        flag = i32([0])                                    # and such a copy is left out
        cache = _cache(4, 2, 16, 64, 1)
        before = [x.clone() for x in cache]
        rkv.page_copy([cache], *c, flags=flag)
        assert flag.item() == rkv.FLAG_BAD_INDEX and all(torch.equal(x, y) for x, y in zip(cache, before))


@cuda
def test_release_of_a_sharing_table_is_the_plain_one_where_nothing_is_shared():
    g = np.random.default_rng(5)
    lens = [int(x) for x in g.integers(0, 300, size=700)]
    fin = [int(x) for x in g.integers(0, 3, size=700)]
    table, free, nf = _table(lens, 16, 20, 9, 6)
    got = []
    for sharing in (False, True):
        pt = rkv.PageTable(700, 20, len(free), 16, sharing=sharing)
        for x, y in ((pt.block_table, table), (pt.seq_len, lens), (pt.free_blocks, free), (pt.n_free, [nf])):
            x.copy_(i32(y))
        pt.release(i32(fin))
        got.append((pt.block_table.tolist(), pt.seq_len.tolist(), pt.free_blocks.tolist(), pt.n_free.item(), pt.flags.item()))
    assert got[0] == got[1]
    with pytest.raises(ValueError):
        rkv.PageTable(2, 2, 2).fork(i32([0, 0]))


# ----------------------------------------------------------------------------- compact
COMPACTS = [([0], 16, 3), ([1], 16, 0), ([16 * 3], 16, 40), ([5, 0, 129, 64], 64, 7), (list(range(0, 900, 3)), 16, 500),
            ([16 * 20000], 16, 20011), ([i % 50 for i in range(8192)], 16, 3000), ([100] * 33, 32, 100000),
            ([100] * 300, 16, 700000), ([5, 300], 16, 1000000)]          # more pages than shared memory takes


@cuda
@pytest.mark.parametrize("case", range(len(COMPACTS)))
@pytest.mark.parametrize("share", [0.0, 0.7])
@pytest.mark.parametrize("inplace", [False, True])
def test_compact_matches_the_definition(case, share, inplace):
    lens, P, spare = COMPACTS[case]
    M = max(1, max(-(-n // P) for n in lens)) + 1
    table, free, _ = _table(lens, P, M, spare, case, share)
    num = len(free)
    t2, live, moves = OP.compact(lens, table, num, P)
    t, ln, f, n, flags = i32(table), i32(lens), torch.full((num,), -9, dtype=torch.int32, device="cuda"), i32([-9]), i32([0])
    to = t if inplace else torch.full_like(t, -9)
    c = rkv.page_compact(ln, t, f, n, P, block_table_out=to, flags=flags)
    assert flags.item() == 0 and n.item() == num - live and c.count.item() == len(moves) and c.rows is None
    assert np.array_equal(to.cpu().numpy(), t2) and ln.tolist() == lens
    assert f.tolist() == list(range(num - 1, live - 1, -1)) + [-9] * live
    src, dst = c.src.tolist(), c.dst.tolist()
    assert list(zip(src, dst))[:len(moves)] == moves and len(src) == num // 2
    assert src[len(moves):] == dst[len(moves):] == [-1] * (num // 2 - len(moves))
    if not inplace:
        assert np.array_equal(t.cpu().numpy(), table)
        c = rkv.page_compact(ln, to.clone(), f, n, P, block_table_out=to, flags=flags)     # nothing left to do
        assert c.count.item() == 0 and np.array_equal(to.cpu().numpy(), t2)


@cuda
def test_compact_flags_what_is_out_of_range():
    table = np.array([[9, -7, 2, -1], [12, 10 ** 9, -1, -1]])
    for inplace in (False, True):
        t, f, n, flags = i32(table), i32([5] * 12), i32([3]), i32([0])
        to = t if inplace else torch.full_like(t, -9)
        c = rkv.page_compact(i32([40, 20]), t, f, n, 16, block_table_out=to, flags=flags)
        assert flags.item() == rkv.FLAG_BAD_INDEX and n.item() == 10 and c.count.item() == 2
        assert c.src.tolist()[:2] == [2, 9] and c.dst.tolist()[:2] == [0, 1]
        assert to.tolist() == [[1, -7, 0, -1], [12, 10 ** 9, -1, -1]]
        for lens in ([40, -1], [65, 20]):
            t, f, n, flags = i32(table), i32([5] * 12), i32([3]), i32([0])
            to = t if inplace else torch.full_like(t, -9)
            c = rkv.page_compact(i32(lens), t, f, n, 16, block_table_out=to, flags=flags)
            assert flags.item() == rkv.FLAG_BAD_INDEX and n.item() == 3 and f.tolist() == [5] * 12
            assert to.tolist() == table.tolist() and c.count.item() == 0 and set(c.src.tolist()) == {-1}


# ------------------------------------------------------------------------ copy, gather
def _cache(num, N, P, D, seed, layers=None):
    """Pages of random codes (NaN codes among them) and scales."""
    g = torch.Generator().manual_seed(seed)
    lead = (num,) if layers is None else (layers, num)
    c = torch.randint(0, 256, (2, *lead, N, P, D), generator=g, dtype=torch.uint8).cuda()
    s = torch.exp2(torch.randint(-20, 20, (2, *lead, N), generator=g).float()).cuda()
    return c[0], c[1], s[0], s[1]


@cuda
@pytest.mark.parametrize("shape", [(7, 1, 16, 64, 1), (40, 3, 64, 128, 5), (30, 8, 128, 64, 2), (24, 2, 32, 128, 128)])
@pytest.mark.parametrize("part", [False, True])
def test_copy_matches_the_definition(shape, part):
    num, N, P, D, L = shape
    k8, v8, ks, vs = _cache(num, N, P, D, 3, L)
    g = np.random.default_rng(num)
    pairs = num // 3
    ids = g.permutation(num)[:2 * pairs]
    src, dst = ids[:pairs].tolist() + [-1, -1], ids[pairs:].tolist() + [-1, -5]
    rows = [int(x) for x in g.integers(0, P + 1, size=len(src))] if part else None
    rest = [x for x in range(num) if x not in ids]
    bad = [(num, rest[0]), (rest[0], num), (-1, rest[0]), (rest[0], -1)] + ([(rest[0], rest[0])] if part else [])
    want = [x.cpu().numpy().copy() for x in (k8, v8, ks, vs)]
    for layer in range(L):
        for c, s in ((want[0], want[2]), (want[1], want[3])):
            OP.copy_pages(c[layer], s[layer], src, dst, rows)
    caches = list(zip(k8, v8, ks, vs))
    flags = i32([0])
    opt = lambda x: None if x is None else i32(x)  # noqa: E731
    rkv.page_copy(caches, i32(src + [rest[0]] * 3), i32(dst + [rest[1]] * 3), opt(rows and rows + [P] * 3),
                  i32([len(src)]), flags=flags)                       # pairs past the count are none
    assert flags.item() == 0
    for x, y in zip((k8, v8, ks, vs), want):
        assert np.array_equal(x.cpu().numpy(), y)
    rkv.page_copy(caches, i32([a for a, _ in bad]), i32([b for _, b in bad]), i32([1] * 4 + [P + 1]) if part else None,
                  flags=flags)
    assert flags.item() == rkv.FLAG_BAD_INDEX
    flags.zero_()
    for n in (0, -3):
        rkv.page_copy(caches, i32([rest[0]]), i32([rest[1]]), None, i32([n]), flags=flags)
    rkv.page_copy(caches, i32([]), i32([]), flags=flags)
    assert flags.item() == 0
    for x, y in zip((k8, v8, ks, vs), want):
        assert np.array_equal(x.cpu().numpy(), y)
    rkv.page_copy(caches, i32([rest[0]]), i32([rest[1]]), None, i32([100]), flags=flags)      # a count past the list
    assert torch.equal(k8[:, rest[1]], k8[:, rest[0]]) and torch.equal(vs[:, rest[1]], vs[:, rest[0]])


@cuda
def test_copy_of_more_pairs_than_warps_and_past_two_gigabytes():
    num, N, P, D = 40000, 8, 64, 128
    k8 = torch.zeros((num, N, P, D), dtype=torch.uint8, device="cuda")
    v8 = torch.zeros_like(k8)
    ks, vs = torch.arange(num * N, device="cuda").float().view(num, N), torch.zeros((num, N), device="cuda")
    k8[:] = (torch.arange(num, device="cuda") % 251).to(torch.uint8)[:, None, None, None]
    v8[:] = (torch.arange(num, device="cuda") % 241).to(torch.uint8)[:, None, None, None]
    ids = torch.randperm(num, generator=torch.Generator().manual_seed(1)).to(torch.int32).cuda()
    src, dst = ids[:9001].contiguous(), ids[9001:18002].contiguous()
    rkv.page_copy([(k8, v8, ks, vs)], src, dst)
    s, d = src.long(), dst.long()
    assert torch.equal(k8[d][:, 0, 0], k8[s][:, 0, 0]) and torch.equal(ks[d], ks[s])
    # every byte of a page is the page's own, or its source's
    of = torch.arange(num, device="cuda")
    of[d] = s
    for i in range(0, num, 4000):
        sl = slice(i, i + 4000)
        assert (k8[sl] == (of[sl] % 251).to(torch.uint8)[:, None, None, None]).all()
        assert (v8[sl] == (of[sl] % 241).to(torch.uint8)[:, None, None, None]).all()


def _stored(codes, scale):
    return np64(codes.view(torch.float8_e4m3fn).float()), np64(scale)


GATHERS = [([1], 1, 64, 16), ([0, 17, 0, 0, 64, 5, 0], 3, 64, 16), ([1000], 8, 128, 64), ([77, 128, 129], 2, 128, 128),
           ([i * 37 % 300 for i in range(61)], 4, 128, 16), ([0, 0], 5, 64, 32), ([2000, 0, 31], 1, 128, 32)]


@cuda
@pytest.mark.parametrize("case", range(len(GATHERS)))
@pytest.mark.parametrize("given", ["made", "out", "strided", "odd", "length"])
def test_gather_matches_the_definition(case, given):
    lens, N, D, P = GATHERS[case]
    table, free, _ = _table(lens, P, max(1, max(-(-n // P) for n in lens)) + 1, 3, case, 0.5)
    k8, v8, ks, vs = _cache(len(free), N, P, D, case)
    take, length = lens, None
    if given == "length":
        take = [n * (b % 3) // 2 if b % 3 else n - n // 3 for b, n in enumerate(lens)]
        take = [min(x, n) for x, n in zip(take, lens)]
        length = i32(take)
    total, flags, more = sum(take), i32([0]), {}
    rows = total + (0 if given == "made" else 5)
    if given == "strided":
        buf = torch.full((rows, 2 * N + 1, D), 7, dtype=torch.bfloat16, device="cuda")
        more = dict(k_out=buf[:, :N], v_out=buf[:, N:2 * N])
    elif given == "odd":                                   # rows that start on 16 bytes, not on 32
        buf = torch.full((rows, (2 * N + 1) * D + 8), 7, dtype=torch.bfloat16, device="cuda")
        more = dict(k_out=buf[:, 8:8 + N * D].view(rows, N, D), v_out=buf[:, 8 + N * D:8 + 2 * N * D].view(rows, N, D))
    elif given != "made":
        more = dict(k_out=torch.full((N, rows, D), 7, dtype=torch.bfloat16, device="cuda").transpose(0, 1),
                    v_out=torch.full((rows, N, D), 7, dtype=torch.bfloat16, device="cuda"))
    k, v, cu = rkv.page_gather(k8, v8, ks, vs, i32(table), i32(lens), None if more else rows, length, flags=flags, **more)
    assert flags.item() == 0 and cu.tolist() == np.concatenate([[0], np.cumsum(take)]).tolist()
    assert k.shape == v.shape == (rows, N, D) and (not more or k is more["k_out"])
    for x, codes, scale in ((k, k8, ks), (v, v8, vs)):
        want = OP.gather(*_stored(codes, scale), table, take, P)
        assert np.array_equal(np64(x)[:total], want, equal_nan=True)
        assert (x[total:] == 7).all() if more else True
    if given == "strided":
        assert (buf[:, 2 * N] == 7).all()
    if given == "odd":
        assert (buf[:, :8] == 7).all() and (buf[:, 8 + 2 * N * D:] == 7).all()


@cuda
def test_gather_of_all_codes_at_all_scales():
    """Code times scale as bf16 holds it; from 2^128 on infinite."""
    k8 = torch.arange(256, dtype=torch.uint8).repeat(185, 1, 1).view(185, 1, 2, 128).repeat(1, 1, 8, 1).cuda()
    ks = torch.exp2(torch.arange(-64, 121).double()).float().view(185, 1).cuda()
    k, v, _ = rkv.page_gather(k8, k8, ks, ks, i32(np.arange(185)[None]), i32([185 * 16]), 185 * 16)
    ref = (k8.view(torch.float8_e4m3fn).float().double() * ks.double().view(185, 1, 1, 1)).view(185 * 16, 1, 128)
    ref = torch.where(ref.abs() >= 2.0 ** 128, torch.copysign(torch.full_like(ref, np.inf), ref), ref)
    for x in (k, v):
        assert np.array_equal(np64(x), ref.cpu().numpy(), equal_nan=True)


@cuda
def test_gather_refuses_what_does_not_fit_and_zeroes_bad_pages():
    lens, N, D, P = [40, 0, 33], 2, 64, 16
    table, free, _ = _table(lens, P, 4, 3, 1)
    k8, v8, ks, vs = _cache(len(free), N, P, D, 2)
    out = lambda: torch.full((80, N, D), 7, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    for rows, length, ln, bit in ((72, None, lens, rkv.FLAG_NO_SPACE), (80, [41, 0, 0], lens, rkv.FLAG_BAD_INDEX),
                                  (80, [0, -1, 0], lens, rkv.FLAG_BAD_INDEX), (80, None, [-1, 0, 5], rkv.FLAG_BAD_INDEX),
                                  (80, [1, 1, 1], [5, 6, 65], rkv.FLAG_BAD_INDEX)):
        ko, vo, flags = out(), out(), i32([0])
        _, _, cu = rkv.page_gather(k8, v8, ks, vs, i32(table), i32(ln), rows, None if length is None else i32(length),
                                   k_out=ko, v_out=vo, flags=flags)
        assert flags.item() == bit and cu.tolist() == [0] * 4 and (ko == 7).all() and (vo == 7).all()
    bad = table.copy()
    bad[0, 1], bad[2, 2] = len(free), -1
    flags = i32([0])
    k, v, cu = rkv.page_gather(k8, v8, ks, vs, i32(bad), i32(lens), 73, flags=flags)
    assert flags.item() == rkv.FLAG_BAD_INDEX and cu.tolist() == [0, 40, 40, 73]
    for x, codes, scale in ((k, k8, ks), (v, v8, vs)):
        want = OP.gather(*_stored(codes, scale), table, lens, P)
        want[16:32], want[72:73] = 0, 0
        assert np.array_equal(np64(x), want, equal_nan=True)


@cuda
def test_gather_of_many_rows_and_pages_past_two_gigabytes():
    num, N, P, D = 20000, 8, 128, 128
    k8 = torch.zeros((num, N, P, D), dtype=torch.uint8, device="cuda")
    k8[:, :, :, 0] = 0x38                                                       # 1.0
    ks = torch.exp2((torch.arange(num * N, device="cuda") % 64 - 32).float()).view(num, N)
    lens = [128 * 300 + 7, 3, 128 * 500]
    ids = torch.randperm(num, generator=torch.Generator().manual_seed(4))
    table = torch.full((3, 501), -1)
    table[0, :301], table[1, :1], table[2, :500] = ids[:301], ids[301:302], ids[302:802]
    table[0, 0], table[2, 1] = num - 1, num - 2
    k, v, cu = rkv.page_gather(k8, k8, ks, ks, table.to(torch.int32).cuda(), i32(lens), sum(lens) + 9)
    pages = torch.cat([table[b, torch.arange(n) // P] for b, n in enumerate(lens)]).cuda()
    for x in (k, v):
        x = x[:sum(lens)]
        assert torch.equal(x[:, :, 0].float(), ks[pages]) and (x[:, :, 1:] == 0).all()
    assert cu.tolist() == [0, lens[0], lens[0] + 3, sum(lens)]


# ------------------------------------------------------------------- as they are used
def _serve(steps, cache, table):
    """Append rows of k, v ([rows, N, D]) to slots: steps of (new tokens, k, v)."""
    for new, k, v in steps:
        plan = table.plan(i32(new), k.shape[0])
        cache.append(k, v, table, plan)
        assert table.flags.item() == 0


@cuda
@pytest.mark.parametrize("P,D", [(16, 64), (64, 128)])
def test_forked_requests_are_those_that_share_nothing(P, D):
    """A prompt stored once and forked to three requests, which go on with rows of their own: the
    decode attention's bits are those of three requests that stored all of it."""
    N, Hq, L = 2, 8, 2
    kp, vp = randn(L, 3 * P + 5, N, D, seed=1), randn(L, 3 * P + 5, N, D, seed=2)
    kn, vn = randn(9, L, 3, N, D, seed=3), randn(9, L, 3, N, D, seed=4)
    q = randn(9, L, 3, Hq, D, seed=5)
    shared = rkv.PageTable(4, 8, 30, P, sharing=True)
    alone = rkv.PageTable(3, 8, 30, P)
    caches = [[rkv.PagedCache(N, D, 30, P) for _ in range(L)] for _ in range(2)]
    for c in caches[0] + caches[1]:
        for x in c.arrays():
            x.view(torch.uint8).fill_(0x7E)                    # stale bytes: 448, and scales past use
    plan = shared.plan(i32([3 * P + 5, 0, 0, 0]), 3 * P + 5)
    for layer, c in enumerate(caches[0]):
        c.append(kp[layer], vp[layer], shared, plan)
    copies = shared.fork(i32([0, 0, 0, -1]))
    rkv.page_copy(caches[0], *copies, flags=shared.flags)
    assert copies.rows.tolist() == [0, 5, 5, 0] and shared.n_free.item() == 30 - 6
    plan = alone.plan(i32([3 * P + 5] * 3), 9 * P + 15)
    for layer, c in enumerate(caches[1]):
        c.append(kp[layer].repeat(3, 1, 1), vp[layer].repeat(3, 1, 1), alone, plan)
    for s in range(9):
        plan = shared.plan(i32([1, 1, 1, 0]), 3)
        plan2 = alone.plan(i32([1, 1, 1]), 3)
        for layer in range(L):
            a, b = caches[0][layer], caches[1][layer]
            a.append(kn[s, layer], vn[s, layer], shared, plan)
            b.append(kn[s, layer], vn[s, layer], alone, plan2)
            o = a.attend(torch.cat([q[s, layer], q[s, layer, :1]]), shared)
            assert torch.equal(o[:3], b.attend(q[s, layer], alone)) and (o[3] == 0).all()
        if s == 4:                                             # the pool is compacted in between
            copies = shared.compact()
            rkv.page_copy(caches[0], *copies, flags=shared.flags)
            assert shared.n_free.item() == 30 - 6 and shared.block_table.max().item() == 5
    # two of the three end: the prompt's pages stay, and go with the last one
    shared.release(i32([1, 0, 1, 0]))
    o = caches[0][0].attend(torch.cat([q[0, 0], q[0, 0, :1]]), shared)
    assert torch.equal(o[1], caches[1][0].attend(q[0, 0], alone)[1])
    shared.release(i32([0, 1, 0, 0]))
    assert shared.n_free.item() == 30 and sorted(shared.free_blocks.tolist()) == list(range(30))
    assert shared.flags.item() == 0 and alone.flags.item() == 0


@cuda
def test_a_prompt_behind_a_stored_prefix_and_cut_drafts():
    """Keys are normed and rotated, stored, forked to a new request, gathered, and attended by the
    rest of its prompt; drafts are stored, cut, and other rows take their place.  Against the
    definitions over what the pages hold."""
    N, Hq, D, P = 2, 4, 64, 16
    table = rkv.PageTable(3, 12, 24, P, sharing=True)
    cache = rkv.PagedCache(N, D, 24, P)
    freq, w = rkv.rotation_freq(D, 5e5), randn(D, seed=9)
    q, k, v = randn(60, Hq, D, seed=1), randn(60, N, D, seed=2), randn(60, N, D, seed=3)
    plan = table.plan(i32([60, 0, 0]), 64)                     # a padded step
    pad = lambda x: torch.cat([x, torch.full_like(x[:4], float("nan"))])  # noqa: E731
    qr, kr = rkv.head_norm_rotate(pad(q), pad(k), plan.row_pos, freq, w, w, 1e-6, q_out=pad(q), k_out=pad(k))
    wk = np64(w)
    ref = OP.norm_rotate(np64(k), list(range(60)), np64(freq).tolist(), wk, 1e-6)
    # within the norm's and rotation's tolerance: at most 2^-19 of the pair (its norm below the
    # row's, sqrt(D) max w) and half a bf16 step
    assert np.all(np.abs(np64(kr[:60]) - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -18 * np.sqrt(D) * np.abs(wk).max())
    cache.append(kr, pad(v), table, plan)
    copies = table.fork(i32([0, 0, -1]), i32([-1, 37, -1]))
    rkv.page_copy([cache], *copies, flags=table.flags)
    # 20 more rows of request 1, over its 37 stored ones and themselves
    plan = table.plan(i32([0, 20, 0]), 20)
    q2, k2, v2 = randn(20, Hq, D, seed=4), randn(20, N, D, seed=5), randn(20, N, D, seed=6)
    q2, k2 = rkv.head_norm_rotate(q2, k2, plan.row_pos, freq, w, w, 1e-6)
    cache.append(k2, v2, table, plan)
    kk, vv, cu = cache.gather(table, 70, length=i32([0, 57, 0]))
    o = rkv.prompt_attention(q2, kk, vv, plan.cu_rows, cu, flags=table.flags)
    assert table.flags.item() == 0 and cu.tolist() == [0, 0, 57, 57]
    bt, ln = table.block_table.cpu().numpy(), table.seq_len.tolist()
    ks, vs = (OP.gather(*_stored(c, s), bt[1:2], [57], P) for c, s in ((cache.k8, cache.k_scale), (cache.v8, cache.v_scale)))
    assert np.array_equal(np64(kk[:57]), ks) and np.array_equal(np64(vv[:57]), vs)
    want, _, a, big = OP.prompt_attention(np64(q2), ks, vs, [0, 20], [0, 57], D ** -0.5)
    tol = 2.0 ** -8 * np.abs(want) + (2.0 ** -8 + 4 * D * 2.0 ** -24 * big + 2.0 ** -14) * a + 1e-30
    assert np.all(np.abs(np64(o) - want) <= tol)
    # drafts of request 0: four stored, three of them cut, two others stored
    plan = table.plan(i32([4, 0, 0]), 4)
    kd, vd = randn(4, N, D, seed=7), randn(4, N, D, seed=8)
    cache.append(kd, vd, table, plan)
    copies = table.fork(None, i32([61, -1, -1]))
    assert set(copies.src.tolist()) == {-1}                    # its last page is its own
    plan = table.plan(i32([2, 0, 0]), 2)
    cache.append(kd[2:], vd[2:], table, plan)
    q3 = randn(3, Hq, D, seed=9)
    o = cache.attend(q3, table)
    bt, ln = table.block_table.cpu().numpy(), table.seq_len.tolist()
    assert ln == [63, 57, 0] and table.flags.item() == 0
    stored = [x * s[:, :, None, None] for x, s in (_stored(cache.k8, cache.k_scale), _stored(cache.v8, cache.v_scale))]
    want, _, a, big = OP.page_attention(np64(q3), *stored, bt, ln, P, D ** -0.5)
    tol = 2.0 ** -8 * np.abs(want) + (2.0 ** -11 + 4 * D * 2.0 ** -24 * big + 2.0 ** -14) * a + 1e-30
    assert np.all(np.abs(np64(o) - want) <= tol)
    got = OP.gather(*_stored(cache.k8, cache.k_scale), bt, [63, 0, 0], P)[60:]
    # stored values: half a step of E4M3, or of its smallest step at the page's scale
    step = float(cache.k_scale[int(bt[0, 3])].max()) * 2.0 ** -10
    assert np.all(np.abs(got - np64(kd)[[0, 2, 3]]) <= np.maximum(np.abs(np64(kd)[[0, 2, 3]]) * 2.0 ** -4, step))


@cuda
def test_beam_search_step_captured_and_replayed():
    """A step of plan, append, attend, fork and copies in one graph: replayed, its bits are those of
    the calls made one by one, as are the table and the free list."""
    N, Hq, D, P, B, steps = 2, 4, 64, 16, 6, 40
    g = np.random.default_rng(3)
    sources = [[3 * (b // 3) + int(x) for b, x in enumerate(g.integers(0, 3, size=B))] for _ in range(steps)]
    ks, vs, qs = randn(steps, B, N, D, seed=1), randn(steps, B, N, D, seed=2), randn(steps, B, Hq, D, seed=3)
    got = []
    for captured in (False, True):
        table = rkv.PageTable(B, 5, 40, P, sharing=True)
        cache = rkv.PagedCache(N, D, 40, P)
        for x in cache.arrays():
            x.zero_()
        k, v, q, src, one = ks[0].clone(), vs[0].clone(), qs[0].clone(), i32(sources[0]), i32([1] * B)

        def step():
            plan = table.plan(one, B)
            cache.append(k, v, table, plan)
            o = cache.attend(q, table)
            rkv.page_copy([cache], *table.fork(src), flags=table.flags)
            return o
        outs = []
        if captured:
            for x, y in ((k, ks), (v, vs), (q, qs)):
                x.copy_(y[0])
            outs.append(step().clone())                        # the first call outside the capture
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                o = step()
        for s in range(len(outs), steps):
            for x, y in ((k, ks), (v, vs), (q, qs)):
                x.copy_(y[s])
            src.copy_(i32(sources[s]))
            if captured:
                graph.replay()
            else:
                o = step()
            outs.append(o.clone())
        assert table.flags.item() == 0
        bt, n = table.block_table, table.n_free.item()
        held = set(bt[bt >= 0].tolist())
        assert held.isdisjoint(table.free_blocks[:n].tolist()) and len(held) + n == 40
        got.append((torch.stack(outs), bt.clone(), table.free_blocks[:n].clone()))
    for x, y in zip(*got):
        assert torch.equal(x, y)


@cuda
def test_calls_wait_for_what_precedes_them():
    """Each call reads what the operation right before it writes, a kernel, a fill, a copy or another
    stream's, made one by one and captured, and again and again: the results follow."""
    N, D, P, n = 2, 64, 16, 4000
    k8, v8, ks, vs = _cache(600, N, P, D, 9)
    big = torch.zeros(1 << 26, device="cuda")
    table, lens = i32(np.arange(500)[None]), i32([0])
    q, pos, freq = randn(n, 3, D, seed=1), i32([0] * n), rkv.rotation_freq(D)
    host_len, host_pos = torch.tensor([16 * 400], dtype=torch.int32).pin_memory(), torch.arange(n, dtype=torch.int32).pin_memory()
    src, dst, free, nf = i32([-1]), i32([-1]), i32([0] * 600), i32([0])
    side = torch.cuda.Stream()

    def chain():
        big.add_(1)                                        # some time during which the rest may run ahead
        lens.copy_(host_len, non_blocking=True)
        k, v, cu = rkv.page_gather(k8, v8, ks, vs, table, lens, 6400)
        pos.copy_(host_pos, non_blocking=True)
        pos.add_(big[0].int() * 0 + 3)
        a, _ = rkv.head_norm_rotate(q, None, pos, freq, eps=1e-6)
        b, _ = rkv.head_norm_rotate(a, None, pos, freq, eps=1e-6)          # reads what the last call wrote
        src.fill_(5)
        dst.fill_(599)
        rkv.page_copy([(k8, v8, ks, vs)], src, dst)
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            big.add_(1)
            lens.fill_(16 * 300)
        main.wait_stream(side)
        out, cut, left = torch.empty_like(table), torch.empty_like(lens), torch.empty_like(nf)
        free2 = free.clone()
        rkv.page_fork(None, lens, table, free2, nf, P, length=lens // 2, block_table_out=out, seq_len_out=cut, n_free_out=left)
        c = rkv.page_compact(cut, out, free2, left, P, block_table_out=out)
        k2, v2, cu2 = rkv.page_gather(k8, v8, ks, vs, out, cut, 2400)
        return k, v, cu, a, b, k8.clone(), ks.clone(), out, cut, left, free2, c.count, k2, v2, cu2

    def reset():
        lens.zero_()
        pos.zero_()
        src.fill_(-1)
        dst.fill_(-1)
        k8[599], ks[599] = 0, 1
    same = lambda x, y: all(torch.equal(a.view(torch.uint8) if a.element_size() < 4 else a,  # noqa: E731
                                        b.view(torch.uint8) if b.element_size() < 4 else b) for a, b in zip(x, y))
    reset()
    want = [x.clone() for x in chain()]
    torch.cuda.synchronize()
    assert want[2].tolist() == [0, 6400] and want[8].item() == 2400 and want[9].item() == 450 and want[14].tolist() == [0, 2400]
    check_a = OP.norm_rotate(np64(q[:5]), [3, 4, 5, 6, 7], np64(freq).tolist(), None, 1e-6)
    assert np.all(np.abs(np64(want[3][:5]) - check_a) <= 2.0 ** -8 * np.abs(check_a) + 2.0 ** -18 * np.sqrt(D))
    assert torch.equal(want[5][599], k8[5]) and np.array_equal(
        np64(want[0]), OP.gather(*_stored(k8, ks), np.arange(500)[None], [6400], P), equal_nan=True)
    for _ in range(20):
        reset()
        assert same(chain(), want)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = chain()
    for _ in range(20):
        reset()
        graph.replay()
        assert same(got, want)


@cuda
def test_two_streams_at_once():
    """Calls on different buffers in two streams give what they give alone."""
    def make(seed):
        lens, source, length, _ = _random_fork(256, 600, 16, seed)
        table, free, nf = _table(lens, 16, 40, 300, seed, 0.5)
        cache = _cache(len(free), 2, 16, 64, seed)
        return i32(lens), i32(table), i32(free), i32([nf]), i32(source), i32(length), cache

    def go(s, stream=None):
        ln, t, f, n, source, length, cache = s
        to, lo, no = torch.empty_like(t), torch.empty_like(ln), torch.empty_like(n)
        f = f.clone()
        c = rkv.page_fork(source, ln, t, f, n, 16, length=length, block_table_out=to, seq_len_out=lo, n_free_out=no)
        k, v, cu = rkv.page_gather(*cache, t, ln, 80000)
        f2, n2 = f.clone(), n.clone()
        m = rkv.page_compact(lo, to, f2, n2, 16, block_table_out=torch.empty_like(to))
        total = int(ln.sum().item()) if stream is None else None
        return [*c[:3], to, lo, no, f, m.src, m.dst, m.count, f2[:int(n2.item())] if stream is None else f2, cu, k, v], total
    states = [make(s) for s in (1, 2)]
    want = [go(s) for s in states]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        got = []
        for s, stream in zip(states, streams):
            with torch.cuda.stream(stream):
                got.append(go(s, stream)[0])
        torch.cuda.synchronize()
        for a, (b, total) in zip(got, want):
            for i, (x, y) in enumerate(zip(a, b)):
                if i >= 12:                                    # rows past the total are not written
                    x, y = x[:total], y[:total]
                assert torch.equal(x[:len(y)], y) or torch.equal(x[:len(y)].view(torch.int16), y.view(torch.int16))


@cuda
def test_binding_refusals():
    lens, table, free, nf = i32([5, 0]), i32([[0, -1], [-1, -1]]), i32([1, 2, 0]), i32([2])
    fork = dict(source=i32([0, 0]), seq_len=lens, block_table=table, free_blocks=free, n_free=nf, block_tokens=16)
    for bad in (dict(source=i32([0])), dict(source=lens.long()), dict(length=i32([1])), dict(finished=lens.cpu()),
                dict(block_table_out=table[:, :1]), dict(seq_len_out=i32([1])), dict(n_free_out=i32([1, 2])),
                dict(block_tokens=24), dict(flags=i32([0, 0])), dict(n_free=None), dict(block_table=table.T),
                dict(free_blocks=free[:0])):
        with pytest.raises((ValueError, rkv.RkvError)):
            rkv.page_fork(**dict(fork, **bad))
    comp = dict(seq_len=lens, block_table=table, free_blocks=free, n_free=nf, block_tokens=16)
    for bad in (dict(block_table_out=table.long()), dict(block_tokens=8), dict(n_free=nf.float()), dict(seq_len=i32([1]))):
        with pytest.raises((ValueError, rkv.RkvError)):
            rkv.page_compact(**dict(comp, **bad))
    c = _cache(3, 2, 16, 64, 1)
    other = _cache(4, 2, 16, 64, 1)
    for caches, src, dst, more in (([c, other], i32([0]), i32([1]), {}), ([c], i32([0]), i32([1, 2]), {}),
                                   ([c], lens.long(), lens.long(), {}), ([c], i32([0]), i32([1]), dict(rows=i32([1, 2]))),
                                   ([c], i32([0]), i32([1]), dict(count=i32([]))), ([c[:3]], i32([0]), i32([1]), {}),
                                   ([list(c)], i32([0]), i32([1]), {})):
        with pytest.raises((ValueError, rkv.RkvError)):
            rkv.page_copy(caches, src, dst, **more)
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    for more in (dict(), dict(max_rows=-1), dict(k_out=bf(9, 2, 64)), dict(k_out=bf(9, 2, 64), v_out=bf(8, 2, 64)),
                 dict(k_out=bf(9, 1, 64).expand(9, 2, 64), v_out=bf(9, 2, 64)),
                 dict(k_out=bf(9, 2, 64).float(), v_out=bf(9, 2, 64)), dict(max_rows=9, length=i32([1])),
                 dict(max_rows=10, k_out=bf(9, 2, 64), v_out=bf(9, 2, 64))):
        with pytest.raises((ValueError, rkv.RkvError)):
            rkv.page_gather(*c, table, lens, **more)
