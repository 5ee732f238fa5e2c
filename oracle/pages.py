"""Full-attention layers written out in float64: the plan of a step's pages, K/V rows in
8-bit pages, the decode attention over them and the causal attention of packed prompts; norm
and rotation of query and key rows; pages that several sequences hold.

Test infrastructure, like the rest of ``oracle/``; it shares no code with the CUDA library.
Everything is the operators' definitions, one element, page or row at a time.
"""
from __future__ import annotations

import math

import numpy as np

__all__ = ["plan", "release", "scale_of", "e4m3_round", "append", "page_attention", "prompt_attention",
           "norm_rotate", "fork", "compact", "copy_pages", "gather"]


def plan(new, lens, table, free, n_free, P, max_rows):
    """(cu, rows [(seq, pos, slot)], lens', n_free', table') of one step, or None where it
    does not fit.  free[:n_free] is taken from its end."""
    new, lens, table = [int(x) for x in new], [int(x) for x in lens], np.array(table)
    M = table.shape[1]
    if any(a < 0 or b < 0 or a + b > M * P for a, b in zip(new, lens)):
        return None
    need = [-(-(a + b) // P) - -(-b // P) for a, b in zip(new, lens)]
    if sum(new) > max_rows or sum(need) > n_free:
        return None
    taken, rows, cu = n_free, [], [0]
    for b, (a, old) in enumerate(zip(new, lens)):
        have = -(-old // P)
        for i in range(need[b]):
            taken -= 1
            table[b, have + i] = free[taken]
        for p in range(old, old + a):
            rows.append((b, p, int(table[b, p // P]) * P + p % P))
        cu.append(cu[-1] + a)
    return cu, rows, [a + b for a, b in zip(new, lens)], taken, table


def release(finished, lens, table, free, n_free, P):
    """(lens', table', free', n_free') after giving back the marked sequences' pages."""
    lens, table, free = list(lens), np.array(table), list(free)
    for b, f in enumerate(finished):
        if f:
            for j in range(-(-lens[b] // P)):
                free[n_free] = int(table[b, j])
                n_free += 1
                table[b, j] = -1
            lens[b] = 0
    return lens, table, free, n_free


def scale_of(amax: float) -> float:
    """The smallest power of two s >= 2^-64 with amax <= 448 s."""
    e = -64
    while math.ldexp(448.0, e) < amax:
        e += 1
    return math.ldexp(1.0, e)


def e4m3_round(x):
    """Nearest E4M3 value, ties to even, saturating at 448; NaN stays."""
    x = np.asarray(x, np.float64)
    _, e = np.frexp(np.where(np.isfinite(x), x, 0.0))
    ulp = np.exp2(np.maximum(e - 1, -6) - 3.0)
    with np.errstate(invalid="ignore"):
        r = np.rint(x / ulp) * ulp
    return np.where(np.isnan(x), np.nan, np.clip(r, -448.0, 448.0))


def append(x, codes, scale, table, lens, cu, P):
    """Stores packed rows x [n, N, D] in the pages: codes [blocks, N, P, D] (the E4M3 values
    as float64) and scale [blocks, N], both changed in place."""
    for b in range(len(lens)):
        n = cu[b + 1] - cu[b]
        lo = lens[b] - n
        for page in range(lo // P, -(-lens[b] // P)) if n else ():
            t0, t1 = max(lo, page * P), min(lens[b], (page + 1) * P)
            blk, off = table[b][page], t0 - page * P
            rows = x[cu[b] + t0 - lo:cu[b] + t1 - lo]
            for h in range(x.shape[1]):
                r = rows[:, h]
                fin = np.abs(r[np.isfinite(r)])
                s = scale_of(fin.max() if fin.size else 0.0)
                if off:
                    old = scale[blk, h]
                    s = max(s, old)
                    codes[blk, h, :off] = e4m3_round(codes[blk, h, :off] * (old / s))
                codes[blk, h, off:off + t1 - t0] = e4m3_round(r / s)
                scale[blk, h] = s


def _softmax_rows(s, v):
    """(o, lse, sum of weight |v|) for scores s [n] against v [n, D]."""
    if s.size == 0:
        z = np.zeros(v.shape[1])
        return z, -math.inf, z
    m = s.max()
    w = np.exp(s - m)
    return w @ v / w.sum(), m + math.log(w.sum()), w @ np.abs(v) / w.sum()


def page_attention(q, k, v, table, lens, P, scale):
    """q [B, Hq, D]; k, v [blocks, N, P, D] the stored values (codes times scales).  Returns
    (o, lse, a, s): a = sum of weight |v| and s = the largest scale sum |q||k|, for error
    bounds."""
    B, Hq, D = q.shape
    G = Hq // k.shape[1]
    o, a = np.zeros((B, Hq, D)), np.zeros((B, Hq, D))
    lse, big = np.full((B, Hq), -math.inf), 0.0
    for b in range(B):
        ids = [int(i) for i in table[b][:-(-lens[b] // P)]]
        for hq in range(Hq):
            kk = np.concatenate([k[i, hq // G] for i in ids] or [np.zeros((0, D))])[:lens[b]]
            vv = np.concatenate([v[i, hq // G] for i in ids] or [np.zeros((0, D))])[:lens[b]]
            o[b, hq], lse[b, hq], a[b, hq] = _softmax_rows(scale * (kk @ q[b, hq]), vv)
            if len(kk):
                big = max(big, scale * (np.abs(kk) @ np.abs(q[b, hq])).max())
    return o, lse, a, big


def prompt_attention(q, k, v, cu_q, cu_k, scale):
    """Packed causal attention: q [Tq, Hq, D], k, v [Tk, N, D].  Returns (o, lse, a, s) as
    page_attention does; rows past cu_q[-1] are zero."""
    Hq, D = q.shape[1:]
    G = Hq // k.shape[1]
    o, a = np.zeros(q.shape), np.zeros(q.shape)
    lse, big = np.full(q.shape[:2], -math.inf), 0.0
    for b in range(len(cu_q) - 1):
        lq, lk = cu_q[b + 1] - cu_q[b], cu_k[b + 1] - cu_k[b]
        for h in range(Hq):
            kk, vv = k[cu_k[b]:cu_k[b + 1], h // G], v[cu_k[b]:cu_k[b + 1], h // G]
            for i in range(lq):
                n = max(0, lk - lq + i + 1)
                r = cu_q[b] + i
                o[r, h], lse[r, h], a[r, h] = _softmax_rows(scale * (kk[:n] @ q[r, h]), vv[:n])
                if n:
                    big = max(big, scale * (np.abs(kk[:n]) @ np.abs(q[r, h])).max())
    return o, lse, a, big


def norm_rotate(x, positions, freq, weight=None, eps=None, adjacent=False):
    """Rows x [n, H, D] divided by their root mean square (eps None: as they are) times weight
    [D], then pair j of the first 2 len(freq) values of each head turned by positions freq[j]:
    values j and j + len(freq), or 2 j and 2 j + 1 (adjacent).  Rows at negative positions
    come back as NaN: nothing is written there."""
    x, out = np.asarray(x, np.float64), np.full(np.shape(x), np.nan)
    h = len(freq)
    for r, p in enumerate(positions):
        if p < 0:
            continue
        for i in range(x.shape[1]):
            y = x[r, i].copy()
            if eps is not None:
                y /= math.sqrt(float(y @ y) / y.size + eps)
                if weight is not None:
                    y *= weight
            out[r, i] = y
            for j, f in enumerate(freq):
                a, b = (2 * j, 2 * j + 1) if adjacent else (j, j + h)
                c, s = math.cos(p * f), math.sin(p * f)
                out[r, i, a], out[r, i, b] = y[a] * c - y[b] * s, y[b] * c + y[a] * s
    return out


def fork(source, length, lens, table, free, n_free, P):
    """Row b of the table becomes the first length[b] positions (length None or length[b] < 0:
    all) of row source[b] as it was (source None: b; negative: nothing).  Returns (table',
    lens', free', n_free', copies {b: (src, dst, rows)}), or None where it does not fit."""
    lens, table, free = [int(x) for x in lens], np.array(table), list(free)
    B, M = table.shape
    num = len(free)
    new, rows = [], []
    for b in range(B):
        s = b if source is None else int(source[b])
        n = 0
        if s >= B or not 0 <= lens[b] <= M * P:
            return None
        if s >= 0:
            n = lens[s] if length is None or length[b] < 0 else int(length[b])
            if n > lens[s]:
                return None
        new.append(n)
        rows.append([int(p) for p in table[s, :-(-n // P)]] if n else [])
    whole, begun = set(), {}                   # pages held whole, and the first row that has begun one
    for b in range(B):
        for j, p in enumerate(rows[b]):
            if (j + 1) * P <= new[b]:
                whole.add(p)
            else:
                begun.setdefault(p, b)
    there = lambda p: 0 <= p < num  # noqa: E731
    end, seen = n_free, set()
    for b in range(B):
        for p in table[b, :-(-lens[b] // P)]:
            p = int(p)
            if there(p) and p not in whole and p not in begun and p not in seen:
                if end >= num:
                    return None
                seen.add(p)
                free[end] = p
                end += 1
    copies = {}
    for b in range(B):
        if new[b] % P and there(rows[b][-1]) and (rows[b][-1] in whole or begun[rows[b][-1]] != b):
            if end == 0:
                return None
            end -= 1
            copies[b] = (rows[b][-1], int(free[end]), new[b] % P)
    for b in range(B):
        if b in copies:
            rows[b][-1] = copies[b][1]
        table[b] = rows[b] + [-1] * (M - len(rows[b]))
    return table, new, free, end, copies


def compact(lens, table, num, P):
    """Pages that a row holds, moved to the lowest numbers: the i-th (ascending) held page of at
    least n_live goes to the i-th page below n_live that none holds.  Returns (table', n_live,
    moves [(src, dst)]); everything from n_live on is free, the last page first in the list."""
    table = np.array(table)
    used = [[int(p) for p in table[b, :-(-int(n) // P)]] for b, n in enumerate(lens)]
    held = {p for row in used for p in row if 0 <= p < num}
    live = sorted(held)
    holes = [p for p in range(len(live)) if p not in held]
    to = dict(zip([p for p in live if p >= len(live)], holes))
    for b, row in enumerate(used):
        table[b] = [to.get(p, p) for p in row] + [-1] * (table.shape[1] - len(row))
    return table, len(live), list(to.items())


def copy_pages(codes, scale, src, dst, rows=None):
    """The first rows[i] rows (None: all) of every head of page src[i], and its scale, put in
    page dst[i]: codes [blocks, N, P, D] and scale [blocks, N] change in place."""
    for i, (a, b) in enumerate(zip(src, dst)):
        if a >= 0 and b >= 0:
            r = codes.shape[2] if rows is None else rows[i]
            codes[b, :, :r] = codes[a, :, :r]
            scale[b] = scale[a]


def gather(codes, scale, table, lens, P):
    """The stored rows of all sequences, packed: [sum lens, N, D] (codes as float64 values)."""
    out = [np.zeros((0, codes.shape[1], codes.shape[3]))]
    for b, n in enumerate(lens):
        for p in range(n):
            i = int(table[b][p // P])
            out.append((codes[i, :, p % P] * scale[i][:, None])[None])
    return np.concatenate(out)
