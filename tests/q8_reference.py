"""64-bit references of the 8-bit cache formats, the attention over such a
cache and the verification of drafted tokens, written from the definitions in
include/dflash_attn.h (numpy, one value at a time where that is the plainest)."""
from __future__ import annotations

import math
from fractions import Fraction

import numpy as np

QMAX = {"int8": 127.0, "e4m3": 448.0}


def scale_exponent(amax: float, fmt: str) -> int:
    """Smallest e >= -117 with amax <= qmax * 2^e."""
    e = -117
    if amax > 0:
        e = max(e, math.frexp(amax)[1] - 12)
    while amax > math.ldexp(QMAX[fmt], e):
        e += 1
    return e


def round_code(y: np.ndarray, fmt: str) -> np.ndarray:
    if fmt == "int8":
        return np.round(y)  # ties to even
    a = np.maximum(np.abs(y), 2.0 ** -6)
    step = 2.0 ** (np.floor(np.log2(a)) - 3)
    return np.round(y / step) * step


def stored_values(x: np.ndarray, fmt: str) -> np.ndarray:
    """What rows x [..., 128] read back as."""
    x = np.asarray(x, dtype=np.float64)
    out = np.empty_like(x).reshape(-1, 32)
    for i, g in enumerate(x.reshape(-1, 32)):
        if not np.all(np.isfinite(g)):
            out[i] = np.nan
            continue
        g = np.clip(g, -(2.0 ** 126), 2.0 ** 126)
        e = scale_exponent(float(np.max(np.abs(g))), fmt)
        out[i] = np.ldexp(round_code(np.ldexp(g, -e), fmt), e)
    return out.reshape(x.shape)


def seen_keys(length: int, q_len: int, t: int, window: int, causal: bool):
    """Key range [lo, hi) that block row t sees."""
    at = length - q_len + t
    lo, hi = 0, length
    if window > 0:
        lo, hi = max(lo, at - window + 1), min(hi, at + window)
    if causal:
        hi = min(hi, at + 1)
    return lo, max(lo, hi)


def attend(q, k, v, window=0, causal=False):
    """One sequence: q [T, nq, d], k and v [len, nkv, d] -> (out, lse, A, Q):
    A = sum p |v| / sum p and Q = the largest sum_c |q_c k_c| / sqrt(d) of the
    row, what the error bounds of an fp32/bf16 evaluation are made of."""
    T, nq, d = q.shape
    length, nkv = k.shape[0], k.shape[1]
    out, lse = np.zeros((T, nq, d)), np.full((T, nq), -np.inf)
    A, Q = np.zeros((T, nq, d)), np.zeros((T, nq))
    for t in range(T):
        lo, hi = seen_keys(length, T, t, window, causal)
        if hi <= lo:
            continue
        for h in range(nq):
            kh, vh = k[lo:hi, h // (nq // nkv)], v[lo:hi, h // (nq // nkv)]
            s = kh @ q[t, h] / math.sqrt(d)
            m = np.max(s)
            p = np.exp(s - m)
            out[t, h] = p @ vh / p.sum()
            lse[t, h] = m + math.log(p.sum())
            A[t, h] = p @ np.abs(vh) / p.sum()
            Q[t, h] = np.max(np.abs(kh) @ np.abs(q[t, h])) / math.sqrt(d)
    return out, lse, A, Q


def fixed(p: np.ndarray) -> list:
    """floor(min(max(p, 0), 1) * 2^44), NaN as 0, in Python integers."""
    res = []
    for x in np.asarray(p, dtype=np.float64):
        x = min(float(x), 1.0) if x > 0 else 0.0
        res.append(int(Fraction(x) * (1 << 44) // 1))
    return res


def verify(drafts, draft, target, u_accept, u_sample, n):
    """One sequence (drafts [D], draft [D, V] or None, target [D + 1, V], n of
    the D drafts in use) -> (accepted, tokens [D + 1])."""
    D, V = len(drafts), target.shape[1]
    n = min(max(int(n), 0), D)
    a = 0
    while a < n:
        x = int(drafts[a])
        if not 0 <= x < V:
            break
        q = 1.0 if draft is None else float(draft[a, x])
        p, u = float(target[a, x]), float(u_accept[a])
        if any(math.isnan(z) for z in (p, q, u)):
            break
        if any(math.isinf(z) for z in (p, q, u)):
            if not u * q < p:
                break
        elif not Fraction(u) * Fraction(q) < Fraction(p):
            break
        a += 1
    w = p_row = fixed(target[a])
    if a < n:
        if draft is None:
            w = [0 if v == int(drafts[a]) else x for v, x in enumerate(p_row)]
        else:
            w = [max(x - y, 0) for x, y in zip(p_row, fixed(draft[a]))]
        if sum(w) == 0:
            w = p_row
    total, token = sum(w), -1
    if total > 0:
        u = float(u_sample)
        u = min(u, 1.0) if u > 0 else 0.0
        t = min(math.floor(u * float(total)), total - 1)
        c = 0
        for v, x in enumerate(w):
            c += x
            if c > t:
                token = v
                break
    tokens = [int(x) for x in drafts[:a]] + [token]
    return a, tokens + [-1] * (D + 1 - len(tokens))
