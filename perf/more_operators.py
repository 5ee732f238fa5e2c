"""What is timed of the operators around the paged cache: queries' and keys' norm and rotation before the
attention, and pages that several sequences hold (forked, cut, freed and compacted in the table, copied in
the caches, and gathered as rows for a prompt behind a stored prefix).

Cases name an operator by "op" and its sizes; head counts are those of this repository's workloads
(8 key/value heads of 128 with 32 query heads, 4 with 28) and small generic ones.
"""
import math

import numpy as np
import torch

own = False


# ----------------------------------------------------------------------------- cases
def listed():
    return [
        # one token of each of 16 decoding requests: all latency
        dict(name="rotate_decode", op="rotate", batch=16, new=1, old=16384, hq=32, n=8, d=128, rotary=128,
             adjacent=False, norm=True, dtype="bf16", base=5e5),
        # ragged prompts in a step of fixed size (its last rows are nobody's), rotation alone
        dict(name="rotate_packed", op="rotate", batch=8, new=1900, old=100000, hq=28, n=4, d=128, rotary=128,
             adjacent=False, norm=False, dtype="bf16", base=1e6),
        # a prompt of 32768 tokens: all bandwidth
        dict(name="rotate_long", op="rotate", batch=1, new=32768, old=0, hq=32, n=8, d=128, rotary=128,
             adjacent=False, norm=True, dtype="bf16", base=5e5),
        # a step of beam search: 4 requests of 4 beams, each beam goes on from one of its request's
        dict(name="fork_beams", op="fork", kind="beams", batch=16, group=4, block=64, length=16384),
        # a serving step of 256 slots: drafts cut, requests finished, prefixes handed to new requests
        dict(name="fork_mixed", op="fork", kind="mixed", batch=256, group=1, block=16, length=4100),
        # the begun pages of 4 forked requests in the caches of 28 layers
        dict(name="copy_forked", op="copy", pairs=16, absent=4, num=100, layers=28, n=4, d=128, block=64, part=True),
        # the pages that a compaction moves, in 8 layers
        dict(name="copy_moved", op="copy", pairs=701, absent=0, num=1500, layers=8, n=8, d=128, block=64, part=False),
        # a small pool, half of it in use
        dict(name="compact_small", op="compact", batch=16, block=64, length=2000, spare=1.0),
        # 256 requests on pages of 16, three quarters of the pool in use
        dict(name="compact_large", op="compact", batch=256, block=16, length=8000, spare=0.33),
        # a stored prefix of a thousand tokens for one new prompt
        dict(name="gather_one", op="gather", batch=1, n=8, d=128, block=64, length=1000),
        # ragged prefixes in small pages
        dict(name="gather_ragged", op="gather", batch=61, n=4, d=128, block=16, length=5000),
        # a long context
        dict(name="gather_long", op="gather", batch=2, n=8, d=128, block=64, length=65536),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rotate", "rotate", "fork", "copy", "compact", "gather", "gather"])
    hq, n = rng.choice([(32, 8), (28, 4), (16, 8), (40, 8), (12, 1), (5, 5), (18, 2)])
    d = rng.choice([64, 128, 128])
    block = rng.choice([16, 32, 64, 128])
    if op == "rotate":
        batch = _log_int(rng, 1, 64)
        new = 1 if rng.random() < 0.4 else _log_int(rng, 1, 12000 // batch)
        return dict(op=op, batch=batch, new=new, old=_log_int(rng, 1, 130000), hq=hq, n=n, d=d,
                    rotary=rng.choice([d, d, d // 2, 32]), adjacent=rng.random() < 0.3, norm=rng.random() < 0.6,
                    dtype=rng.choice(["bf16", "bf16", "fp32"]), base=rng.choice([1e4, 5e5, 1e6]))
    if op == "fork":
        length = _log_int(rng, 1, 16384)
        most = max(4, min(512, 131072 * block // (length + block)))
        if rng.random() < 0.5:
            group = rng.choice([2, 3, 4, 8])
            return dict(op=op, kind="beams", batch=group * _log_int(rng, 1, max(1, most // group)), group=group,
                        block=block, length=length)
        return dict(op=op, kind="mixed", batch=_log_int(rng, 2, most), group=1, block=block, length=length)
    if op == "copy":
        layers = _log_int(rng, 1, 32)
        page = n * d * block
        pairs = _log_int(rng, 1, max(1, min(2000, (1 << 28) // (page * layers))))
        return dict(op=op, pairs=pairs, absent=rng.randrange(0, pairs + 1) // 2,
                    num=2 * pairs + _log_int(rng, 1, 100), layers=layers, n=n, d=d, block=block,
                    part=rng.random() < 0.5)
    if op == "compact":
        length = _log_int(rng, 1, 16384)
        return dict(op=op, batch=_log_int(rng, 1, max(1, min(512, 131072 * block // (length + block)))),
                    block=block, length=length, spare=rng.choice([0.1, 0.33, 1.0, 3.0]))
    batch = _log_int(rng, 1, 64)
    return dict(op=op, batch=batch, n=n, d=d, block=block, length=_log_int(rng, 1, 131072 // batch))


def _lengths(case, what, lo):
    """Lengths of the case's sequences, spread over [lo, nominal]; one has the nominal length."""
    nominal, batch = case[what], case["batch"]
    g = np.random.default_rng([nominal, len(what), batch])
    lens = g.integers(min(lo, nominal), nominal + 1, size=batch)
    lens[g.integers(batch)] = nominal
    return lens


def _shape(case, seed):
    """The case's lengths, on the host: the same requests, in another order for another seed."""
    op = case["op"]
    if op == "copy":
        return ()
    if op == "fork" and case["kind"] == "beams":          # a request's beams are equally long
        one = dict(case, batch=case["batch"] // case["group"])
        lens = _lengths(one, "length", 1 + case["length"] // 4)
        return (np.random.default_rng(seed).permutation(lens).repeat(case["group"]),)
    order = np.random.default_rng(seed).permutation(case["batch"])
    if op == "rotate":
        return _lengths(case, "new", 1)[order], _lengths(case, "old", 0)[order]
    return (_lengths(case, "length", 1 + case["length"] // 4)[order],)


def _forks(case, seed):
    """The case's table and what becomes of its rows, on the host: lengths, pages (numbered in order of
    their first holder, -1 past them), sources and new lengths (None: the sources' own)."""
    (lens,) = _shape(case, seed)
    P, B = case["block"], case["batch"]
    have = -(-lens // P)
    M = int(have.max()) + 1
    g = np.random.default_rng([11, seed])
    j = np.arange(M)[None, :]
    if case["kind"] == "beams":
        first = (np.arange(B) // case["group"]) * case["group"]
        common = (lens // P) * 3 // 4                     # whole pages of the prompt, held by all beams
        held_by = np.where(j < common[:, None], first[:, None], np.arange(B)[:, None])
        source = first + g.integers(0, case["group"], size=B)
        length = None
    else:
        held_by = np.broadcast_to(np.arange(B)[:, None], (B, M))
        kind = np.random.default_rng([5, B]).permutation(B) % 8      # 0, 1: an empty slot, 2: finished
        kind[int(lens.argmax())] = 7
        lens = np.where(kind < 2, 0, lens)
        have = -(-lens // P)
        live = np.flatnonzero(kind > 2)
        parent = live[g.integers(0, len(live), size=B)]
        source = np.where(kind == 0, parent, np.where(kind == 2, -1, np.arange(B)))
        cut = np.maximum(1, lens - g.integers(0, 9, size=B))
        length = np.where(kind == 0, np.maximum(1, lens[parent] * 3 // 4), np.where(kind > 4, cut, lens))
    mine = (held_by == np.arange(B)[:, None]) & (j < have[:, None])
    number = np.cumsum(mine.reshape(-1)).reshape(B, M) - 1
    table = np.where(j < have[:, None], number[held_by, j], -1)
    return lens, table, source, length


def work(case):
    op = case["op"]
    if op == "rotate":
        rows, wide = _shape(case, 0)[0].sum(), 4 if case["dtype"] == "fp32" else 2
        return {"bytes": int(rows * ((case["hq"] + case["n"]) * case["d"] * 2 * wide + 4)), "flops": 0}
    if op == "fork":
        lens, table, source, length = _forks(case, 0)
        B, M = table.shape
        return {"bytes": int(4 * ((table >= 0).sum() + B * M + 7 * B)), "flops": 0}
    if op == "copy":
        pairs = case["pairs"] - case["absent"]
        page = case["n"] * case["d"] * case["block"]
        return {"bytes": int(case["layers"] * pairs * 2 * 2 * (page // (2 if case["part"] else 1) + 4 * case["n"])),
                "flops": 0}
    (lens,) = _shape(case, 0)
    P = case["block"]
    if op == "compact":
        used = -(-lens // P)
        num = int(used.sum() * (1 + case["spare"])) + 3
        return {"bytes": int(4 * (used.sum() + case["batch"] * (int(used.max()) + 2) + 2 * (num // 2)
                                  + num - used.sum())), "flops": 0}
    return {"bytes": int(lens.sum() * 2 * case["n"] * case["d"] * 3), "flops": 0}


# ---------------------------------------------------------------------------- inputs
def _channel(d, device, g):
    """Keys have a few strong channels."""
    return torch.exp(0.7 * torch.randn(d, generator=g, device=device))


def _filled(shape, channel, device, g):
    """Codes and scales of pages [..., N, P, D] filled with normal values."""
    codes = torch.empty(shape, dtype=torch.uint8, device=device)
    scale = torch.empty(shape[:-2], dtype=torch.float32, device=device)
    flat, fs = codes.view(-1, *shape[-3:]), scale.view(-1, shape[-3])
    step = max(1, (1 << 27) // (shape[-3] * shape[-2] * shape[-1]))
    for i in range(0, len(flat), step):
        x = torch.randn(flat[i:i + step].shape, generator=g, device=device) * channel
        s = torch.exp2(torch.ceil(torch.log2(x.abs().amax(dim=(2, 3)) / 448)))
        flat[i:i + step] = (x / s[:, :, None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
        fs[i:i + step] = s
    return codes, scale


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    op = case["op"]
    i32 = lambda a: torch.as_tensor(np.ascontiguousarray(a), dtype=torch.int32).to(dev)  # noqa: E731
    if op == "rotate":
        new, old = _shape(case, seed)
        hq, n, d, R = case["hq"], case["n"], case["d"], case["rotary"]
        total = int(new.sum())
        rows = total + (0 if case["new"] == 1 else total // 16)       # a padded step: nobody's rows last
        pos = np.full(rows, -1, dtype=np.int64)
        pos[:total] = np.arange(total) - (np.cumsum(new) - new).repeat(new) + old.repeat(new)
        dt = torch.float32 if case["dtype"] == "fp32" else torch.bfloat16
        # heads of one projection's output, side by side in its rows
        x = torch.randn((rows, hq + 2 * n, d), generator=g, device=dev)
        x[:, hq:hq + n] *= _channel(d, dev, g)
        x = x.to(dt)
        wq, wk = ((1 + 0.2 * torch.randn((2, d), generator=g, device=dev)).to(dt) if case["norm"] else (None, None))
        return dict(op=op, q=x[:, :hq], k=x[:, hq:hq + n], wq=wq, wk=wk, pos=i32(pos),
                    rotary=R, adjacent=case["adjacent"], eps=1e-6 if case["norm"] else None,
                    freq=torch.from_numpy(case["base"] ** (-np.arange(0, R, 2) / R)).to(dev),
                    q_out=torch.zeros((rows, hq, d), dtype=dt, device=dev),
                    k_out=torch.zeros((rows, n, d), dtype=dt, device=dev))
    if op == "copy":
        L, num, n, P, d = case["layers"], case["num"], case["n"], case["block"], case["d"]
        shape = (L, num + 1, n, P, d)                     # the last page is nobody's
        k8, ks = _filled(shape, _channel(d, dev, g), dev, g)
        v8, vs = _filled(shape, torch.ones(d, device=dev), dev, g)
        ids = torch.randperm(num, generator=g, device=dev, dtype=torch.int32)[:2 * case["pairs"]].view(2, -1)
        gone = torch.randperm(case["pairs"], generator=g, device=dev)[:case["absent"]]
        ids[:, gone] = -1
        rows = torch.randint(1, P, (case["pairs"],), generator=g, device=dev, dtype=torch.int32)
        return dict(op=op, k8=k8, v8=v8, ks=ks, vs=vs, src=ids[0].contiguous(), dst=ids[1].contiguous(),
                    rows=rows if case["part"] else None, caches=list(zip(k8, v8, ks, vs)))
    if op == "fork":
        lens, table, source, length = _forks(case, seed)
        used = int(table.max()) + 1                       # pages of the pool: the same for every seed
        num = int((-(-_shape(case, seed)[0] // case["block"])).sum()) * 9 // 8 + 2 * case["batch"]
        ids = torch.randperm(num, generator=g, device=dev, dtype=torch.int32)
        t = torch.from_numpy(table).to(dev)
        free = torch.zeros(num, dtype=torch.int32, device=dev)
        free[:num - used] = ids[used:]
        return dict(op=op, table=torch.where(t >= 0, ids[t.clamp_min(0)], -1).to(torch.int32).contiguous(),
                    len=i32(lens), source=i32(source), length=None if length is None else i32(length),
                    free=free, n_free=i32([num - used]), block=case["block"],
                    table_out=torch.full(table.shape, -1, dtype=torch.int32, device=dev),
                    len_out=i32(lens), n_free_out=i32([0]))
    (lens,) = _shape(case, seed)
    P = case["block"]
    used = -(-lens // P)
    num = int(used.sum() * (1 + (case["spare"] if op == "compact" else 0))) + 3
    M = int(used.max()) + 2
    j = np.arange(M)[None, :]
    t = torch.from_numpy(np.where(j < used[:, None], (np.cumsum(used) - used)[:, None] + j, -1)).to(dev)
    ids = torch.randperm(num, generator=g, device=dev, dtype=torch.int32)
    table = torch.where(t >= 0, ids[t.clamp_min(0)], -1).to(torch.int32).contiguous()
    if op == "compact":
        free = torch.zeros(num, dtype=torch.int32, device=dev)
        free[:num - int(used.sum())] = ids[int(used.sum()):]
        return dict(op=op, table=table, len=i32(lens), free=free, n_free=i32([num - int(used.sum())]), block=P,
                    table_out=torch.full_like(table, -1))
    n, d, total = case["n"], case["d"], int(lens.sum())
    k8, ks = _filled((num, n, P, d), _channel(d, dev, g), dev, g)
    v8, vs = _filled((num, n, P, d), torch.ones(d, device=dev), dev, g)
    rows = total + total // 16
    k, v = torch.zeros((2, rows, n, d), dtype=torch.bfloat16, device=dev)
    return dict(op=op, k8=k8, v8=v8, ks=ks, vs=vs, table=table, len=i32(lens), k=k, v=v)


# ----------------------------------------------------------------------- plain forms
def _rotate_plain(s):
    pos, R = s["pos"].double(), s["rotary"]
    angle = pos[:, None, None] * s["freq"]
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    live = (s["pos"] >= 0)[:, None, None]

    def one(x, w, out):
        y = x.float()
        if s["eps"] is not None:
            y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + s["eps"]) * w.float()
        if s["adjacent"]:
            a, b = y[..., :R:2], y[..., 1:R:2]
            z = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        else:
            a, b = y[..., :R // 2], y[..., R // 2:R]
            z = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        return out.copy_(torch.where(live, torch.cat([z, y[..., R:]], -1).to(out.dtype), out))
    return one(s["q"], s["wq"], s["q_out"]), one(s["k"], s["wk"], s["k_out"])


def _fork_plain(s):
    table, lens, source, P = s["table"].long(), s["len"].long(), s["source"].long(), s["block"]
    B, M = table.shape
    num = len(s["free"])
    dev = table.device
    b, j = torch.arange(B, device=dev)[:, None], torch.arange(M, device=dev)[None, :]
    new_len = lens[source.clamp_min(0)] if s["length"] is None else s["length"].long()
    new_len = torch.where(source >= 0, new_len, 0)
    last = (new_len + P - 1) // P - 1
    row = torch.where(j <= last[:, None], table[source.clamp_min(0)], num)           # num: no page
    begun = (j == last[:, None]) & (new_len % P != 0)[:, None]
    whole = torch.zeros(num + 1, dtype=torch.bool, device=dev)
    whole[torch.where(begun, num, row).flatten()] = True
    keeper = torch.full((num + 1,), B, device=dev)
    keeper.scatter_reduce_(0, torch.where(begun, row, num).flatten(), b.expand(B, M).flatten(), "amin")
    page = row.gather(1, last.clamp_min(0)[:, None])[:, 0]
    copied = begun.any(1) & (whole[page] | (keeper[page] != b[:, 0]))
    # pages that no row holds any more, in the order of their first holder
    held = whole | (keeper < B)
    old = torch.where(j < ((lens + P - 1) // P)[:, None], table, num).flatten()
    place = torch.arange(B * M, device=dev)
    first = torch.full((num + 1,), B * M, device=dev).scatter_reduce_(0, old, place, "amin")
    freed = (old < num) & ~held[old] & (first[old] == place)
    n_free = s["n_free"].long()
    at = torch.where(freed, n_free + torch.cumsum(freed, 0) - 1, num)
    free = torch.cat([s["free"], s["free"][:1]]).scatter_(0, at, old.to(torch.int32))[:num]
    s["free"].copy_(free)
    end = n_free + freed.sum()
    taken = free[(end - torch.cumsum(copied, 0)).clamp(0, num - 1)].long()
    row = torch.where(begun & copied[:, None], taken[:, None], row)
    s["table_out"].copy_(torch.where(j <= last[:, None], row, -1))
    s["len_out"].copy_(new_len)
    s["n_free_out"].copy_(end - copied.sum())
    src, dst = torch.where(copied, page, -1), torch.where(copied, taken, -1)
    return (src.to(torch.int32), dst.to(torch.int32), torch.where(copied, new_len % P, 0).to(torch.int32),
            s["table_out"], s["len_out"], s["free"], s["n_free_out"])


def _copy_plain(s):
    spare = s["k8"].shape[1] - 1
    src, dst = (torch.where(s[x] >= 0, s[x], spare).long() for x in ("src", "dst"))
    for codes, scale in ((s["k8"], s["ks"]), (s["v8"], s["vs"])):
        moved = codes[:, src]
        if s["rows"] is not None:
            p = torch.arange(codes.shape[3], device=codes.device)
            moved = torch.where((p < s["rows"][:, None])[:, None, :, None], moved, codes[:, dst])
        codes[:, dst] = moved
        scale[:, dst] = scale[:, src]
    return tuple(x.view(torch.float8_e4m3fn) for x in (s["k8"], s["v8"])) + (s["ks"], s["vs"])


def _compact_plain(s):
    table, P, num = s["table"].long(), s["block"], len(s["free"])
    j = torch.arange(table.shape[1], device=table.device)[None, :]
    used = j < ((s["len"].long() + P - 1) // P)[:, None]
    page = torch.where(used, table, num)
    live = torch.zeros(num + 1, dtype=torch.bool, device=table.device)
    live[page.flatten()] = True
    live = live[:num]
    n_live = live.sum()
    i = torch.arange(num, device=table.device)
    moves, hole = live & (i >= n_live), ~live & (i < n_live)
    src, dst = (torch.full((num // 2 + 1,), -1, device=table.device).scatter_(
        0, torch.where(x, torch.cumsum(x, 0) - 1, num // 2), torch.where(x, i, -1))[:num // 2] for x in (moves, hole))
    to = torch.where(moves, dst[(torch.cumsum(moves, 0) - 1).clamp(0, max(0, num // 2 - 1))], i)
    s["table_out"].copy_(torch.where(used, to[table.clamp(0, num - 1)], -1))
    s["free"].copy_(torch.where(i < num - n_live, num - 1 - i, s["free"]))
    s["n_free"].copy_(num - n_live)
    return (src.to(torch.int32), dst.to(torch.int32), moves.sum().to(torch.int32).view(1), s["table_out"],
            s["free"], s["n_free"])


def _gather_plain(s):
    length, P = s["len"].long(), s["k8"].shape[2]
    end = torch.cumsum(length, 0)
    r = torch.arange(len(s["k"]), device=end.device)
    seq = torch.searchsorted(end, r, right=True).clamp_max(len(length) - 1)
    live = r < end[-1]
    pos = torch.where(live, r - (end - length)[seq], 0)
    page, off = s["table"].long()[seq, pos // P], pos % P
    for codes, scale, out in ((s["k8"], s["ks"], s["k"]), (s["v8"], s["vs"], s["v"])):
        x = codes.view(torch.uint8)[page, :, off].view(torch.float8_e4m3fn).float() * scale[page][..., None]
        out.copy_(torch.where(live[:, None, None], x.to(torch.bfloat16), out))
    return s["k"], s["v"], torch.cat([torch.zeros_like(end[:1]), end]).to(torch.int32)


def run(s):
    op = s["op"]
    if own:
        import residual_kv_cache_gb300 as rkv
        if op == "rotate":
            return rkv.head_norm_rotate(s["q"], s["k"], s["pos"], s["freq"], q_weight=s["wq"], k_weight=s["wk"],
                                        eps=s["eps"], adjacent=s["adjacent"], q_out=s["q_out"], k_out=s["k_out"])
        if op == "fork":
            c = rkv.page_fork(s["source"], s["len"], s["table"], s["free"], s["n_free"], s["block"],
                              length=s["length"], block_table_out=s["table_out"], seq_len_out=s["len_out"],
                              n_free_out=s["n_free_out"])
            return c.src, c.dst, c.rows, s["table_out"], s["len_out"], s["free"], s["n_free_out"]
        if op == "copy":
            rkv.page_copy(s["caches"], s["src"], s["dst"], s["rows"])
            return tuple(x.view(torch.float8_e4m3fn) for x in (s["k8"], s["v8"])) + (s["ks"], s["vs"])
        if op == "compact":
            c = rkv.page_compact(s["len"], s["table"], s["free"], s["n_free"], s["block"],
                                 block_table_out=s["table_out"])
            return c.src, c.dst, c.count, s["table_out"], s["free"], s["n_free"]
        return rkv.page_gather(s["k8"], s["v8"], s["ks"], s["vs"], s["table"], s["len"], k_out=s["k"], v_out=s["v"])
    return {"rotate": _rotate_plain, "fork": _fork_plain, "copy": _copy_plain, "compact": _compact_plain,
            "gather": _gather_plain}[op](s)


# -------------------------------------------------------------- the definition, in 64 bits
def exact(case, seed):
    op = case["op"]
    if op in ("fork", "compact"):                         # whole numbers
        return None
    s = prepare(case, seed)
    if op == "rotate":
        R, res = case["rotary"], []
        live = s["pos"] >= 0
        z = torch.polar(torch.ones((), dtype=torch.float64, device=s["pos"].device),
                        s["pos"][live].double()[:, None, None] * s["freq"])
        for x, w, out in ((s["q"], s["wq"], s["q_out"]), (s["k"], s["wk"], s["k_out"])):
            y = x[live].double()
            if case["norm"]:
                y = y / torch.sqrt(y.square().sum(-1, keepdim=True) / y.shape[-1] + s["eps"]) * w.double()
            first, second = (slice(0, R, 2), slice(1, R, 2)) if case["adjacent"] else (slice(0, R // 2), slice(R // 2, R))
            turned = torch.complex(y[..., first].contiguous(), y[..., second].contiguous()) * z
            y[..., first], y[..., second] = turned.real, turned.imag
            full = out.double()
            full[live] = y
            res.append(full)
        return tuple(res)
    if op == "copy":
        out = [x.view(torch.float8_e4m3fn).float() for x in (s["k8"], s["v8"])] + [s["ks"].clone(), s["vs"].clone()]
        src, dst = s["src"].tolist(), s["dst"].tolist()
        rows = [case["block"]] * len(src) if s["rows"] is None else s["rows"].tolist()
        for a, b, r in zip(src, dst, rows):
            if a >= 0:
                for x in out[:2]:
                    x[:, b, :, :r] = x[:, a, :, :r]
                for x in out[2:]:
                    x[:, b] = x[:, a]
        return tuple(x.double() for x in out)
    P, length = case["block"], s["len"].tolist()
    if sum(length) // P + len(length) > 20000:
        return None
    res, at = [s["k"].double(), s["v"].double()], 0
    for t, ids in zip(length, s["table"].tolist()):
        for p in range(-(-t // P)):
            r = min(P, t - p * P)
            for out, codes, scale in zip(res, (s["k8"], s["v8"]), (s["ks"], s["vs"])):
                x = codes[ids[p], :, :r].view(torch.float8_e4m3fn).double() * scale[ids[p]].double()[:, None, None]
                out[at:at + r] = x.transpose(0, 1)
            at += r
    return res[0], res[1], None
