"""GPU calls of the operators around the paged cache whose buffers share memory, and those that the
library's own loop makes seldom: each against the same call on buffers of its own."""
import weakref

import numpy as np
import pytest
import torch

import residual_kv_cache_gb300 as rkv

pytestmark = pytest.mark.gpu
cuda = pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def rows_of_pages(batch, width, block, seed):
    """(table, lengths, free list, free count): rows of pages of their own, in random order."""
    g = np.random.default_rng(seed)
    lens = g.integers(1, width * block + 1, size=batch)
    have = -(-lens // block)
    ids = g.permutation(int(have.sum()) + 2 * batch)
    table, at = np.full((batch, width), -1), 0
    for b, n in enumerate(have):
        table[b, :n] = ids[at:at + n]
        at += n
    free = np.zeros(len(ids), np.int64)
    free[:2 * batch] = ids[at:]
    return table, lens, free, 2 * batch


@cuda
@pytest.mark.parametrize("batch,width", [(9, 40), (256, 40), (700, 20), (8192, 5)])      # 1, 8, 16 and 16 CTAs
@pytest.mark.parametrize("shared", ["source", "length"])
@pytest.mark.parametrize("inplace", [False, True])
def test_fork_whose_lengths_go_where_its_arguments_are(batch, width, shared, inplace):
    """seq_len_out may be source or length: every CTA reads those before one writes, also where the
    call is refused."""
    table, lens, free, nf = rows_of_pages(batch, width, 16, batch)
    g = np.random.default_rng(1)
    source = g.integers(-1, batch, size=batch)
    length = np.array([g.integers(0, lens[s] + 1) if s >= 0 else 3 for s in source])
    for bad in (False, True):
        src, cut = source.copy(), length.copy()
        if bad:
            src[-1], cut[-1] = batch - 1, lens[-1] + 1

        def call(alias):
            t, ln, f, n, a, b, flags = i32(table), i32(lens), i32(free), i32([nf]), i32(src), i32(cut), i32([0])
            to = t if inplace else torch.empty_like(t)
            out = {"source": a, "length": b}[shared] if alias else torch.empty_like(ln)
            c = rkv.page_fork(a, ln, t, f, n, 16, length=b, block_table_out=to, seq_len_out=out, flags=flags)
            return [to, out, f, n, flags, *c[:3]]
        want = [x.tolist() for x in call(False)]
        assert want[4] == [rkv.FLAG_BAD_INDEX if bad else 0]
        assert (want[1] == lens.tolist() and want[0] == table.tolist()) == bad
        for _ in range(20):
            assert [x.tolist() for x in call(True)] == want


@cuda
@pytest.mark.parametrize("n", [1, 7, 3000])
@pytest.mark.parametrize("layout", ["parts of rows", "heads in turn", "rows in turn", "heads outer", "rows in turn, heads outer"])
@pytest.mark.parametrize("inplace", [False, True])
def test_head_rows_side_by_side_in_one_buffer(n, layout, inplace):
    """Queries and keys that lie in one buffer without sharing a value, in every order of rows and
    heads: the bits of buffers of their own."""
    H, D = 3, 64
    buf = torch.randn((6, n * H * D), generator=torch.Generator().manual_seed(n)).to(torch.bfloat16).cuda().view(-1)
    view = lambda *s: buf[:int(np.prod(s))].view(*s)  # noqa: E731
    if layout == "parts of rows":
        b = view(n, 2 * H, D)
        q, k = b[:, :H], b[:, H:]
    elif layout == "heads in turn":
        b = view(n, H, 2, D)
        q, k = b[:, :, 0], b[:, :, 1]
    elif layout == "rows in turn":
        b = view(n, 2, H, D)
        q, k = b[:, 0], b[:, 1]
    elif layout == "heads outer":
        b = view(2, H, n, D)
        q, k = b[0].transpose(0, 1), b[1].transpose(0, 1)
    else:
        b = view(H, n, 2, D)
        q, k = b[:, :, 0].transpose(0, 1), b[:, :, 1].transpose(0, 1)
    pos, freq = torch.arange(n, dtype=torch.int32, device="cuda"), rkv.rotation_freq(D)
    want = rkv.head_norm_rotate(q.contiguous(), k.contiguous(), pos, freq, eps=1e-6)
    before = buf.clone()
    if inplace:
        qo, ko = q, k
    else:
        other = torch.zeros_like(buf)
        qo, ko = (other.as_strided(x.shape, x.stride(), x.storage_offset()) for x in (q, k))
    a, c = rkv.head_norm_rotate(q, k, pos, freq, eps=1e-6, q_out=qo, k_out=ko)
    assert torch.equal(a, want[0]) and torch.equal(c, want[1])
    assert inplace or torch.equal(buf, before)
    # one for the other: read while it is written
    if n > 1:
        for bad in (dict(q_out=qo, k_out=qo), dict(q_out=k, k_out=ko), dict(q_out=q, k_out=q)):
            with pytest.raises(rkv.RkvError, match="overlap"):
                rkv.head_norm_rotate(q, k, pos, freq, eps=1e-6, **bad)


@cuda
@pytest.mark.parametrize("layout", ["parts of rows", "heads in turn", "rows in turn", "heads outer"])
def test_gather_into_one_buffer(layout):
    N, D, P, lens = 3, 64, 16, [37, 0, 50]
    table, _, _, _ = rows_of_pages(3, 4, P, 1)
    table[:] = np.arange(12).reshape(3, 4)
    g = torch.Generator().manual_seed(1)
    k8, v8 = torch.randint(0, 127, (2, 12, N, P, D), generator=g, dtype=torch.uint8).cuda()
    ks, vs = torch.exp2(torch.randint(-9, 9, (2, 12, N), generator=g).float()).cuda()
    n = sum(lens)
    call = lambda **kw: rkv.page_gather(k8, v8, ks, vs, i32(table), i32(lens), **kw)  # noqa: E731
    want = call(max_rows=n)
    buf = lambda *s: torch.full(s, 7, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    if layout == "parts of rows":
        b = buf(n, 2 * N, D)
        k, v = b[:, :N], b[:, N:]
    elif layout == "heads in turn":
        b = buf(n, N, 2, D)
        k, v = b[:, :, 0], b[:, :, 1]
    elif layout == "rows in turn":
        b = buf(n, 2, N, D)
        k, v = b[:, 0], b[:, 1]
    else:
        b = buf(2, N, n, D)
        k, v = b[0].transpose(0, 1), b[1].transpose(0, 1)
    got = call(k_out=k, v_out=v)
    assert got[0] is k and got[1] is v and all(torch.equal(x, y) for x, y in zip(got, want))
    with pytest.raises(rkv.RkvError, match="k and v overlap"):
        call(k_out=k, v_out=k)


@cuda
def test_tables_that_overlap_without_being_one():
    """A table that lies a row further in the same buffer is refused; one right behind the other is
    another table, in one buffer or not."""
    table, lens, free, nf = rows_of_pages(6, 4, 16, 3)
    source = [1, 2, 3, 4, 5, -1]

    def call(at):
        buf = torch.full((12, 4), -9, dtype=torch.int32, device="cuda")
        buf[:6] = i32(table)
        ln, f, n = i32(lens), i32(free), i32([nf])
        rkv.page_fork(i32(source), ln, buf[:6], f, n, 16, block_table_out=buf[at:at + 6])
        c = rkv.page_compact(ln, buf[at:at + 6], f, n, 16)
        return buf[at:at + 6].tolist(), ln.tolist(), f[:n.item()].tolist(), c.count.item()
    want = call(6)
    assert call(0) == want
    t = torch.full((12, 4), -1, dtype=torch.int32, device="cuda")
    for at in (1, 5):
        with pytest.raises(rkv.RkvError, match="overlaps"):
            call(at)
        with pytest.raises(rkv.RkvError, match="overlaps"):
            rkv.page_compact(i32(lens), t[:6], i32(free), i32([nf]), 16, block_table_out=t[at:at + 6])


@cuda
def test_copy_keeps_its_caches_until_the_launch():
    """arrays() of a cache that makes its tensors, and that empties the list: all caches are copied,
    and what was made lives until then."""
    k8 = torch.randint(0, 127, (3, 4, 1, 16, 64), generator=torch.Generator().manual_seed(1), dtype=torch.uint8).cuda()
    ks = torch.arange(12.0, device="cuda").view(3, 4, 1)
    seen = []

    class Cache:
        def __init__(self, layer):
            self.layer = layer

        def arrays(self):
            caches.clear()
            assert all(ref() is not None for ref in seen)
            made = tuple(x[self.layer].view(x[self.layer].shape) for x in (k8, k8, ks, ks))
            seen.extend(weakref.ref(x) for x in made)
            return made
    caches = [Cache(layer) for layer in range(3)]
    rkv.page_copy(caches, i32([1]), i32([3]))
    assert caches == [] and len(seen) == 12 and all(ref() is None for ref in seen)
    assert torch.equal(k8[:, 3], k8[:, 1]) and ks[:, 3].flatten().tolist() == [1, 5, 9]

    seen.clear()

    class Fails:
        def arrays(self):
            raise KeyError("no arrays")
    with pytest.raises(KeyError):
        rkv.page_copy([Cache(0), Fails()], i32([1]), i32([3]))


@cuda
@pytest.mark.parametrize("batch", [5, 300])
def test_release_of_a_sharing_table_with_a_bad_length_is_refused_until_it_is_mended(batch):
    table, lens, free, nf = rows_of_pages(batch, 40, 16, 9)
    pt = rkv.PageTable(batch, 40, len(free), 16, sharing=True)
    for x, y in ((pt.block_table, table), (pt.seq_len, lens), (pt.free_blocks, free), (pt.n_free, [nf])):
        x.copy_(i32(y))
    pt.seq_len[2] = 40 * 16 + 1                                # a row that does not finish
    before = [x.clone() for x in (pt.block_table, pt.seq_len, pt.free_blocks, pt.n_free)]
    fin = i32([b != 2 for b in range(batch)])
    pt.release(fin)
    assert pt.flags.item() == rkv.FLAG_BAD_INDEX
    assert all(torch.equal(x, y) for x, y in zip(before, (pt.block_table, pt.seq_len, pt.free_blocks, pt.n_free)))
    pt.seq_len[2], pt.flags[0] = int(lens[2]), 0
    pt.release(fin)
    assert pt.flags.item() == 0 and pt.seq_len.tolist() == [int(lens[2]) if b == 2 else 0 for b in range(batch)]
    assert pt.n_free.item() == len(free) - -(-int(lens[2]) // 16)


@cuda
def test_weights_that_do_not_start_on_four_bytes_are_refused():
    q, pos, freq = torch.ones((4, 2, 64), dtype=torch.bfloat16, device="cuda"), i32([0, 1, 2, 3]), rkv.rotation_freq(64)
    packed = torch.randn(129, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    with pytest.raises(rkv.RkvError, match="weights 4-byte"):
        rkv.head_norm_rotate(q, None, pos, freq, q_weight=packed[65:], eps=1e-6)
    a, _ = rkv.head_norm_rotate(q, None, pos, freq, q_weight=packed[64:128], eps=1e-6)
    b, _ = rkv.head_norm_rotate(q, None, pos, freq, q_weight=packed[64:128].clone(), eps=1e-6)
    assert torch.equal(a, b)
