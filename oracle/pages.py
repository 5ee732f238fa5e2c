"""Full-attention layers written out in float64: the plan of a step's pages, K/V rows in
8-bit pages, the decode attention over them and the causal attention of packed prompts.

Test infrastructure, like the rest of ``oracle/``; it shares no code with the CUDA library.
Everything is the operators' definitions, one element, page or row at a time.
"""
from __future__ import annotations

import math

import numpy as np

__all__ = ["plan", "release", "scale_of", "e4m3_round", "append", "page_attention", "prompt_attention"]


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
