"""Oracle of the language streams' operators: 8-bit tails, attention over the
shared store and such a tail, and the verification of drafted tokens.

Written from the definitions in fp64 NumPy; stores and queries are arrays of
float64 holding bf16 or e4m3 values.
"""
from __future__ import annotations

import numpy as np


def e4m3_values() -> np.ndarray:
    """The values of codes 0..126 (sign 0; code 127 is NaN), increasing."""
    c = np.arange(127)
    e, m = c >> 3, c & 7
    return np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10))


def e4m3_encode(x: np.ndarray) -> np.ndarray:
    """Nearest code of each value (|x| <= 448), ties to the even code."""
    t = e4m3_values()
    mag = np.abs(x)
    hi = np.clip(np.searchsorted(t, mag), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dh, dl = t[hi] - mag, mag - t[lo]
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    return (code | np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def e4m3_decode(code: np.ndarray) -> np.ndarray:
    t = np.append(e4m3_values(), np.nan)
    return np.where(code >= 128, -1.0, 1.0) * t[code & 127]


def quantise(x: np.ndarray):
    """x [..., D] -> (codes [..., D], exponent bytes [...])."""
    codes = np.zeros(x.shape, np.uint8)
    byte = np.zeros(x.shape[:-1], np.uint8)
    for i in np.ndindex(*x.shape[:-1]):
        v = x[i]
        top = np.max(np.abs(v))
        if not np.isfinite(top):
            byte[i] = 255
            continue
        e = -127
        while top > 448.0 * 2.0 ** e:
            e += 1
        byte[i] = e + 127
        codes[i] = e4m3_encode(v * 2.0 ** -e)
    return codes, byte


def dequantise(codes: np.ndarray, byte: np.ndarray) -> np.ndarray:
    s = np.where(byte == 255, np.nan, 2.0 ** (byte.astype(np.float64) - 127))
    return e4m3_decode(codes) * s[..., None]


def stream_attention(q, k_shared, v_shared, k_tail, v_tail):
    """q [n][Hq][D]: the newest n tokens of a tail k_tail, v_tail [len][Hkv][D];
    shared keys [K][Hkv][D].  Returns (out, spread): spread[t][h][d] =
    sum_j alpha_j |v_jd|, what a relative error of every weight may move."""
    n, Hq, D = q.shape
    Hkv = k_tail.shape[1]
    G = Hq // Hkv
    out = np.zeros((n, Hq, D))
    spread = np.zeros((n, Hq, D))
    for t in range(n):
        seen = max(0, len(k_tail) - n + t + 1)
        for h in range(Hq):
            g = h // G
            k = np.concatenate([k_shared[:, g], k_tail[:seen, g]])
            v = np.concatenate([v_shared[:, g], v_tail[:seen, g]])
            if len(k) == 0:
                continue
            s = k @ q[t, h] / np.sqrt(D)
            a = np.exp(s - np.max(s))
            a /= np.sum(a)
            out[t, h] = a @ v
            spread[t, h] = a @ np.abs(v)
    return out, spread


def verify(p, q, draft, u, r, n):
    """One stream: p [T+1][V], q [T][V] or None -> (tokens, accepted)."""
    V = p.shape[1]
    a = 0
    while a < n:
        x = draft[a]
        if not 0 <= x < V or not u[a] * (1.0 if q is None else q[a, x]) < p[a, x]:
            break
        a += 1
    w = p[a].copy()
    if a < n:
        if q is not None:
            with np.errstate(invalid="ignore"):
                w = w - q[a]
        elif 0 <= draft[a] < V:
            w[draft[a]] = 0.0

    def weights(w):
        return np.where(np.isfinite(w) & (w > 0), w, 0.0)

    w = weights(w)
    if not np.any(w > 0):
        w = weights(p[a])
    nxt = -1
    if np.any(w > 0):
        c = np.cumsum(w)
        over = np.flatnonzero((c > r * c[-1]) & (w > 0))
        nxt = int(over[0]) if len(over) else int(np.flatnonzero(w > 0)[-1])
    return [int(x) for x in draft[:a]] + [nxt], a
