"""Attention of many rows per sequence, drafted trees and the query/key norm with rotation (oracle).

TEST INFRASTRUCTURE ONLY (see the package docstring).

Everything is written from the definitions in float64, one sequence and one head at a time:

* ``attend``: softmax(scale q k^T over the keys a row sees) v, with the logarithm of the sum of
  exponentials, and ``size`` = sum_t p_t |v_t|, the magnitude that the rounding of the softmax
  weights to 16 bits is measured against.  A row that sees nothing has output 0 and lse -inf.
  Keys and values that a row does not see are never touched.
* ``causal_limits``: the number of keys new token i of Lq sees when the last Lq of Lk keys are the
  new tokens' own.
* ``ancestors``: which drafts a draft sees (itself and its chain of parents).
* ``norm_rope``: y = x / sqrt(mean x^2 + eps) w, then the rotation of the first 2 n channels by
  position * inv_freq in pairs half a rotated part apart, or interleaved.
"""
from __future__ import annotations

import numpy as np


def attend(q, k, v, seen, scale):
    """q [R, D], k, v [T, D], seen bool [R, T] -> out [R, D], lse [R], size [R, D], span [R].

    span = max over seen keys of scale * sum_d |q_d k_d|: the scale of a score's rounding error."""
    q, k, v = (np.asarray(x, dtype=np.float64) for x in (q, k, v))
    R, D = q.shape
    out, size = np.zeros((R, D)), np.zeros((R, D))
    lse, span = np.full(R, -np.inf), np.zeros(R)
    for r in range(R):
        at = np.nonzero(seen[r])[0]
        if at.size == 0:
            continue
        s = (k[at] @ q[r]) * scale
        m = s.max()
        p = np.exp(s - m)
        total = p.sum()
        p /= total
        out[r] = p @ v[at]
        size[r] = p @ np.abs(v[at])
        lse[r] = m + np.log(total)
        span[r] = (np.abs(k[at]) @ np.abs(q[r])).max() * scale
    return out, lse, size, span


def causal_limits(lq: int, lk: int) -> np.ndarray:
    return np.clip(np.arange(lq) + lk - lq + 1, 0, lk)


def prompt_attention(q, k, v, cu_q, cu_k, scale):
    """q [TQ, Hq, D], k, v [TK, H, D] -> dict of out, lse, size, span over all rows; rows of no
    sequence are NaN."""
    TQ, Hq, D = q.shape
    G = Hq // k.shape[1]
    r = {"out": np.full((TQ, Hq, D), np.nan), "lse": np.full((TQ, Hq), np.nan),
         "size": np.zeros((TQ, Hq, D)), "span": np.zeros((TQ, Hq))}
    for s in range(len(cu_q) - 1):
        q0, q1, k0, k1 = cu_q[s], cu_q[s + 1], cu_k[s], cu_k[s + 1]
        seen = np.arange(k1 - k0) < causal_limits(q1 - q0, k1 - k0)[:, None]
        for j in range(Hq):
            o, e, a, b = attend(q[q0:q1, j], k[k0:k1, j // G], v[k0:k1, j // G], seen, scale)
            r["out"][q0:q1, j], r["lse"][q0:q1, j] = o, e
            r["size"][q0:q1, j], r["span"][q0:q1, j] = a, b
    return r


def ancestors(parents) -> np.ndarray:
    """parents of one sequence's nodes -> bool [n, n]: row i marks the nodes that node i sees."""
    n = len(parents)
    see = np.zeros((n, n), dtype=bool)
    for i in range(n):
        j = i
        while j >= 0:
            see[i, j] = True
            j = parents[j]
    return see


def tree_attention(q, k_hat, v_hat, length, parents, scale):
    """One sequence: q [n, Hq, D], k_hat, v_hat [length + n, H, D] -> out, size, span."""
    n, Hq, D = q.shape
    G = Hq // k_hat.shape[1]
    seen = np.concatenate([np.ones((n, length), dtype=bool), ancestors(parents)], axis=1)
    out, size, span = np.zeros((n, Hq, D)), np.zeros((n, Hq, D)), np.zeros((n, Hq))
    for j in range(Hq):
        out[:, j], _, size[:, j], span[:, j] = attend(q[:, j], k_hat[:, j // G], v_hat[:, j // G],
                                                      seen, scale)
    return out, size, span


def norm_rope(x, w, positions, inv_freq, eps, interleaved):
    """x [T, H, D] -> float64 [T, H, D]; w [D] or None."""
    y = np.array(x, dtype=np.float64)
    if w is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * np.asarray(w, dtype=np.float64)
    n = len(inv_freq)
    i = np.arange(n)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
    angle = np.asarray(positions, dtype=np.float64)[:, None, None] * np.asarray(inv_freq)
    ya, yb = y[..., a].copy(), y[..., b].copy()
    y[..., a] = ya * np.cos(angle) - yb * np.sin(angle)
    y[..., b] = yb * np.cos(angle) + ya * np.sin(angle)
    return y
