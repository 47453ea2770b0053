"""The 4-bit key/value cache in fp64: quantisation, row order, attention over
it, accumulated weights and eviction, from their definitions.

    a row of D elements is D/32 groups of 32 consecutive ones; per group
        s = bf16(max|x| / 7),  code = round_half_even(x / s), kept in -7..7, + 8  (8 if s = 0),
        value = s * (code - 8);  a group with an infinity or a NaN: s = NaN
    K row: element d is nibble d % 8 of 32-bit word (d % 32 // 8) * (D // 32) + d // 32
    V row: element d is nibble d % 4 of 16-bit word (d % 32 // 4) * (D // 32) + d // 32;
        D = 128: byte i of the row is stored at i ^ 32 in slots with bit 1 set

    attention: new token t < n of a sequence holding `len` slots sees slots
        0 .. len - n + t;  p = exp(s - lse),  o = sum p v
    weights: w[j] += sum of p over the rows of key head h's group
    eviction: the `keep` slots of largest weight, positions >= seen - recent
        before all others, ties to the lower slot, NaN above every number
"""
from __future__ import annotations

from typing import Optional

import numpy as np


def bf16(x: np.ndarray) -> np.ndarray:
    """fp64 values of x (fp64) rounded to bf16, to nearest even."""
    f = np.asarray(x, np.float64)
    with np.errstate(invalid="ignore"):
        m, e = np.frexp(f)
    # 8 significant bits; below 2^-126 the step stays at 2^-133
    step = np.ldexp(1.0, np.maximum(e - 8, -133))
    out = np.rint(f / step) * step
    return np.where(np.isfinite(f), out, f)


def quantise(x: np.ndarray):
    """codes uint8 [.., D], scales fp64 [.., D/32] (bf16 values) of rows x."""
    g = np.asarray(x, np.float64).reshape(*x.shape[:-1], -1, 32)
    with np.errstate(invalid="ignore"):
        top = np.abs(g).max(-1)
        bad = ~np.isfinite(g).all(-1)
        s = np.where(bad, np.nan, bf16(np.where(bad, 0.0, top) / 7))
        safe = np.where(np.isnan(s) | (s == 0), 1.0, s)[..., None]
        q = np.where((np.isnan(s) | (s == 0))[..., None], 0.0, np.clip(np.rint(g / safe), -7, 7))
    return (q + 8).astype(np.uint8).reshape(x.shape), s


def _places(D: int, name: str):
    """(byte, shift) of every element of a row (V rows not exchanged)."""
    d = np.arange(D)
    if name == "k":
        return 4 * (d % 32 // 8 * (D // 32) + d // 32) + d % 8 // 2, 4 * (d % 2)
    return 2 * (d % 32 // 4 * (D // 32) + d // 32) + d % 4 // 2, 4 * (d % 2)


def _row_bytes(D: int, name: str, slots: np.ndarray) -> np.ndarray:
    byte, _ = _places(D, name)
    byte = np.broadcast_to(byte, (len(slots), D)).copy()
    if name == "v" and D == 128:
        byte ^= np.where(slots & 2, 32, 0)[:, None]
    return byte


def pack(codes: np.ndarray, name: str, slots: np.ndarray) -> np.ndarray:
    """uint8 [.., n, D/2] of codes [.., n, D] for the given slots."""
    D = codes.shape[-1]
    byte, shift = _row_bytes(D, name, slots), _places(D, name)[1]
    out = np.zeros(codes.shape[:-1] + (D // 2,), np.uint8)
    for i in range(len(slots)):
        for d in range(D):
            out[..., i, byte[i, d]] |= (codes[..., i, d] << shift[d]).astype(np.uint8)
    return out


def unpack(rows: np.ndarray, name: str) -> np.ndarray:
    """codes [.., capacity, D] of a cache's rows [.., capacity, D/2]."""
    n, D = rows.shape[-2], rows.shape[-1] * 2
    byte, shift = _row_bytes(D, name, np.arange(n)), _places(D, name)[1]
    got = np.take_along_axis(rows, np.broadcast_to(byte, rows.shape[:-1] + (D,)), -1)
    return (got >> shift) & 15


def values(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """fp64 [.., D]: what codes stand for."""
    return (codes.astype(np.float64) - 8) * np.repeat(scales, 32, -1)


def forward(q, k, v, lens, q_lens=None, scale: Optional[float] = None, cap: Optional[float] = None, sinks=None):
    """q [B,Hq,T,D], k/v [B,Hkv,n,D] fp64 values of the slots.
    -> o [B,Hq,T,D], lse [B,Hq,T], weights [B,Hkv,n] (the sums of p), and
    abs_pv [B,Hq,T,1] = sum_j p_j max_d |v_jd|, abs_qk [B,Hq,T] = max over the seen keys of scale * sum |q||k|
    (what the error bounds of lower precision are made of)."""
    B, Hq, T, D = q.shape
    Hkv, n = k.shape[1:3]
    G = Hq // Hkv
    scale = D ** -0.5 if scale is None else scale
    o, apv = np.zeros((B, Hq, T, D)), np.zeros((B, Hq, T, 1))
    lse, aqk = np.full((B, Hq, T), -np.inf), np.zeros((B, Hq, T))
    w = np.zeros((B, Hkv, n))
    for b in range(B):
        ln = min(max(int(lens[b]), 0), n)
        nq = T if q_lens is None else min(max(int(q_lens[b]), 0), T)
        for h in range(Hq):
            g = h // G
            z = np.zeros(0) if sinks is None else np.asarray(sinks[g] if np.ndim(sinks) == 2 else sinks, np.float64)
            for t in range(T):
                end = max(0, ln - nq + t + 1) if t < nq else 0
                s = scale * (k[b, g, :end] @ q[b, h, t])
                if end:
                    aqk[b, h, t] = abs(scale) * (np.abs(k[b, g, :end]) @ np.abs(q[b, h, t])).max()
                if cap:
                    s = cap * np.tanh(s / cap)
                every = np.concatenate([s, z])
                if every.size == 0:
                    continue
                m = every.max()
                lse[b, h, t] = m + np.log(np.exp(every - m).sum())
                p = np.exp(s - lse[b, h, t])
                o[b, h, t] = p @ v[b, g, :end]
                apv[b, h, t] = (p * np.abs(v[b, g, :end]).max(-1)).sum()
                w[b, g, :end] += p
    return o, lse, w, apv, aqk


def evict(weights, positions, lens, keep: int, recent: int = 0, seen=None, in_place: bool = False):
    """index [B,Hkv,keep] (-1 past the new length) and the new lengths."""
    B, H, n = weights.shape
    index = np.full((B, H, keep), -1, np.int64)
    new = np.zeros(B, np.int64)
    for b in range(B):
        ln = min(max(int(lens[b]), 0), n)
        first = int(lens[b] if seen is None else seen[b]) - recent
        new[b] = min(ln, keep)
        for h in range(H):
            def rank(i):
                late = recent > 0 and (i if positions is None else positions[b, h, i]) >= first
                w = float(weights[b, h, i])
                return (not late, 0 if late else (0 if np.isnan(w) else 1), 0.0 if late or np.isnan(w) else -w, i)
            kept = sorted(sorted(range(ln), key=rank)[:keep])
            if not in_place:
                index[b, h, :len(kept)] = kept
                continue
            low = [i for i in kept if i < keep]
            holes = sorted(set(range(min(keep, ln))) - set(low))
            for i in low:
                index[b, h, i] = i
            for hole, i in zip(holes, [i for i in kept if i >= keep]):
                index[b, h, hole] = i
    return index, new
