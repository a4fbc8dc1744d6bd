"""Attention of queries over an encoder's states, in float64."""
from __future__ import annotations

import numpy as np


def attend(q, k, v, visible, scale: float):
    """q [B, Lq, Hq, D], k and v [B, Lk, Hkv, D], visible bool [B, Lk] -> (out, mean, size).
    mean: sum p |v| / sum p, which roundings of the weights and sums are relative to; size: the largest
    |scale| sum |q_c k_c| of a row, which the rounding of its scores is relative to [B, Lq, Hq, 1]."""
    B, Lq, Hq, D = q.shape
    g = Hq // k.shape[2]
    out, mean, size = np.zeros(q.shape), np.zeros(q.shape), np.zeros((B, Lq, Hq, 1))
    for b in range(B):
        at = np.nonzero(visible[b])[0]
        for h in range(Hq if len(at) else 0):
            kk, vv = k[b, at, h // g], v[b, at, h // g]
            with np.errstate(invalid="ignore"):
                s = scale * (q[b, :, h] @ kk.T)
                p = np.exp(s - s.max(-1, keepdims=True))
                p /= p.sum(-1, keepdims=True)
                out[b, :, h], mean[b, :, h] = p @ vv, p @ np.abs(vv)
                size[b, :, h, 0] = abs(scale) * (np.abs(q[b, :, h]) @ np.abs(kk).T).max(-1)
    return out, mean, size
