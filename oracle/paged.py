"""The key/value cache in pages, from its definitions: tables and slots one
sequence after another, bounds of a page's keys, the pages a query selects,
attention over what it sees (fp64, whole numbers exact).

    sequence b of n tokens: the first ceil(n / page) entries of its table row;
        token i lies in slot table[b, i // page] * page + i % page
    resize: pages no longer needed go back first (in order of the sequences,
        then of their rows), to the places before ``used``; then pages are taken
        from there on, all that a sequence needs or none, and after one
        that has to wait no later one takes any
    bounds: m = max|k|, e = max(floor(log2 m) - 7, -100), every channel's
        largest and smallest key rounded up and down to multiples of 2^e;
        infinite where m is not below 2^100 (or not a number)
    selection: qc = round_half_even(q / 2^f), f = max(floor(log2 max|q|) - 6, -100)
        over the group (0 where max|q| is not below 2^100); score = max over
        the heads of sum_d max(qc_d hi_d, qc_d lo_d), infinite where that is
        not finite; the first and last pages, then by score, ties to the lower page
"""
from __future__ import annotations

from typing import Optional

import numpy as np


def resize(table: np.ndarray, free: np.ndarray, used: int, lens, new_lens, page: int, T: int):
    """Changes table and free in place; -> (lens, used, slots)."""
    B, M = table.shape
    out = list(lens)
    slots = np.full((B, T), -1, dtype=np.int32)
    fits = [0 <= n <= M * page and 0 <= w <= M * page and w - n <= T for n, w in zip(lens, new_lens)]
    pages_of = lambda n: -(-n // page)  # noqa: E731
    back = [p for b in range(B) if fits[b] for p in table[b, pages_of(new_lens[b]):pages_of(lens[b])].tolist()]
    if not 0 <= used <= len(free) or len(back) > used:
        return out, used, slots
    used -= len(back)
    free[used:used + len(back)] = back
    waiting = False
    for b in range(B):
        if not fits[b]:
            continue
        have, more = pages_of(lens[b]), pages_of(new_lens[b]) - pages_of(lens[b])
        if more > 0:
            if waiting or used + more > len(free):
                waiting = True
                continue
            table[b, have:have + more] = free[used:used + more]
            used += more
        out[b] = new_lens[b]
        for i in range(max(0, new_lens[b] - lens[b])):
            at = lens[b] + i
            p = table[b, at // page]
            slots[b, i] = p * page + at % page if 0 <= p < len(free) else -1
    return out, used, slots


def _unit(top: float, bits: int) -> float:
    """2^max(floor(log2 top) - bits, -100)."""
    return 2.0 ** max(int(np.frexp(top)[1]) - 1 - bits, -100) if top > 0 else 2.0 ** -100


def bounds(k: np.ndarray) -> np.ndarray:
    """[2, D] of keys [n, D]."""
    top = np.abs(k).max()
    if not top < 2.0 ** 100:
        return np.stack((np.full(k.shape[1], np.inf), np.full(k.shape[1], -np.inf)))
    s = _unit(top, 7)
    return np.stack((np.ceil(k.max(0) / s) * s, np.floor(k.min(0) / s) * s))


def scores(q: np.ndarray, b: np.ndarray) -> np.ndarray:
    """[pages] of a group's q [G, D] and bounds [pages, 2, D]."""
    top = np.abs(q).max()
    qc = np.rint(q / _unit(top, 6)) if top < 2.0 ** 100 else np.zeros_like(q)
    out = np.empty(len(b))
    with np.errstate(invalid="ignore"):
        for j, (hi, lo) in enumerate(b):
            s = np.maximum(qc * hi, qc * lo).sum(1) if np.isfinite(hi).all() else np.full(len(q), np.inf)
            out[j] = s.max()
    return out


def select(q: np.ndarray, b: np.ndarray, keep: int, first: int, recent: int) -> np.ndarray:
    """int32 [keep]: the pages of a query that sees the pages whose bounds are b [pages, 2, D]."""
    n = len(b)
    out = np.full(keep, -1, dtype=np.int32)
    if n == 0:
        return out
    s = scores(q, b)
    always = [j < first or j >= n - recent for j in range(n)]
    order = sorted(range(n), key=lambda j: (not always[j], -s[j], j))[:keep]
    out[:len(order)] = sorted(order)
    return out


def first_key(pos: int, left: Optional[int] = None, chunk: Optional[int] = None) -> int:
    if left is not None and left >= 0:
        return max(0, pos - left)
    return pos // chunk * chunk if chunk else 0


def attend(q: np.ndarray, k: np.ndarray, v: np.ndarray, scale: float, cap: float = 0.0, sinks=None):
    """One row over the keys it sees [n, D]: (o [D], lse, sum p |v| [D], max scale sum|q k|)."""
    D = len(q)
    z = np.zeros(0) if sinks is None else np.asarray(sinks, np.float64)
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        s = k @ q * scale
        size = float((np.abs(k) @ np.abs(q)).max() * abs(scale)) if len(k) else 0.0
        if cap:
            s = cap * np.tanh(s / cap)
        a = np.concatenate((s, z))
        if not len(a):
            return np.zeros(D), -np.inf, np.zeros(D), 0.0
        m = a.max()
        lse = m + np.log(np.exp(a - m).sum())
        if not len(k):
            return np.zeros(D), lse, np.zeros(D), 0.0
        p = np.exp(s - lse)
        return p @ v, lse, p @ np.abs(v), size
