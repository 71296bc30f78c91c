"""Oracle of the paged language streams' operators: norm and rotation of heads,
attention of new tokens over places of a stream, the weight that keys gather,
and eviction by that weight.

Written from the definitions in fp64 NumPy; arrays of float64 hold bf16 values.
"""
from __future__ import annotations

import numpy as np


def rotate(x, weight, eps, pos, freq, sections, adjacent):
    """x [N][heads][D] -> normed (weight [D] or None) and rotated."""
    x = np.array(x, np.float64)
    if weight is not None:
        x = x / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps) * weight
    R2 = sum(sections)
    out = x.copy()
    axis = [a for a, n in enumerate(sections) for _ in range(n)]
    for i in range(R2):
        one, two = (2 * i, 2 * i + 1) if adjacent else (i, i + R2)
        turn = (np.asarray(pos[axis[i]], np.float64) * float(freq[i]))[:, None]
        out[..., one] = x[..., one] * np.cos(turn) - x[..., two] * np.sin(turn)
        out[..., two] = x[..., two] * np.cos(turn) + x[..., one] * np.sin(turn)
    return out


def seen(t, n, length, prefix):
    """Places that new token t of n sees (a count from place 0)."""
    return max(0, length - n + t + 1, min(max(prefix, 0), length))


def attend(q, k, v, there, prefix, k_shared=None, v_shared=None):
    """q [n][Hq][D]: the new tokens of a stream with places k, v [len][Hkv][D],
    of which those with there [len] count.  Returns out, lse [n][Hq], spread =
    sum_j alpha_j |v_j|, and reach [n][Hq] = max_j sum_i |q_i k_ji| / sqrt(D)."""
    n, Hq, D = q.shape
    length, Hkv = k.shape[:2]
    G = Hq // Hkv
    out, spread = np.zeros((n, Hq, D)), np.zeros((n, Hq, D))
    lse, reach = np.full((n, Hq), -np.inf), np.zeros((n, Hq))
    shared = 0 if k_shared is None else len(k_shared)
    for h in range(Hq):
        g = h // G
        kk = k[:, g] if not shared else np.concatenate([k_shared[:, g], k[:, g]])
        vv = v[:, g] if not shared else np.concatenate([v_shared[:, g], v[:, g]])
        for t in range(n):
            on = np.concatenate([np.ones(shared, bool), there & (np.arange(length) < seen(t, n, length, prefix))])
            if not on.any():
                continue
            s = kk[on] @ q[t, h] / np.sqrt(D)
            reach[t, h] = np.max(np.abs(kk[on]) @ np.abs(q[t, h])) / np.sqrt(D)
            top = np.max(s)
            e = np.exp(s - top)
            lse[t, h] = top + np.log(np.sum(e))
            a = e / np.sum(e)
            out[t, h] = a @ vv[on]
            spread[t, h] = a @ np.abs(vv[on])
    return out, lse, spread, reach


def gather(q, lse, k, there, prefix):
    """[len][Hkv]: the weight that the places gather from the new tokens."""
    n, Hq, D = q.shape
    length, Hkv = k.shape[:2]
    G = Hq // Hkv
    w = np.zeros((length, Hkv))
    for h in range(Hq):
        for t in range(n):
            on = there & (np.arange(length) < seen(t, n, length, prefix))
            if not np.isfinite(lse[t, h]):
                continue
            w[on, h // G] += np.exp(k[on, h // G] @ q[t, h] / np.sqrt(D) - lse[t, h])
    return w


def keep(weight, sink, recent, budget):
    """Old places that one head keeps, in order.  weight [len]; NaN (and a place
    without a page, given as NaN) comes last."""
    n = len(weight)
    if n <= budget:
        return list(range(n))
    middle = range(sink, n - recent)
    order = sorted(middle, key=lambda i: (np.isnan(weight[i]), -weight[i] if not np.isnan(weight[i]) else 0.0, i))
    return list(range(sink)) + sorted(order[:budget - sink - recent]) + list(range(n - recent, n))
