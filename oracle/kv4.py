"""CPU oracle: the MXFP4 key/value cache and causal attention over it.

TEST INFRASTRUCTURE (same import rule as ``oracle.svdquant``).  Parity
status: pinned by ``tests/test_oracle_serving.py``.

The rows are encoded as ``oracle.mxfp4`` states it, 32 consecutive channels
to a block, with one addition: a block that holds an infinity or a NaN stands
for 32 NaNs.  For sequence b of length n, new token i of Q and query head h,

    out[b, i, h] = sum_t p_t v[t] / sum_t p_t,   p_t = exp(scale q . k[t]),

over the tokens t < n - Q + i + 1 of key/value head h // (Hq / Hkv); zero
where there is none.  Everything in float64.
"""
from __future__ import annotations

import numpy as np

from . import mxfp4 as MX


def values(x: np.ndarray) -> np.ndarray:
    """What the cache holds for rows x [..., D]: float64, NaN blocks for non-finite input."""
    x = np.asarray(x, dtype=np.float64)
    flat = x.reshape(-1, x.shape[-1])
    bad = ~np.isfinite(flat).reshape(len(flat), -1, MX.BLOCK).all(-1)
    codes, e = MX.quantize_rows(np.where(np.repeat(bad, MX.BLOCK, 1), 0.0, flat).astype(np.float32))
    v = MX.dequantize(codes, e)
    v[np.repeat(bad, MX.BLOCK, 1)] = np.nan
    return v.reshape(x.shape)


def attend(q: np.ndarray, k: list, v: list, lens, scale: float):
    """q [B, Q, Hq, D]; k[b], v[b] [n_b, Hkv, D] the sequences' values.
    Returns (out, mass) float64 [B, Q, Hq, D] with mass = sum p |v| / sum p,
    the size of the terms that make an output, and (largest, terms): the
    largest scale * sum_d |q_d k_td| of each row and its number of tokens."""
    q = np.asarray(q, dtype=np.float64)
    B, Q, Hq, D = q.shape
    out, mass = np.zeros_like(q), np.zeros_like(q)
    largest, terms = np.zeros((B, Q, Hq, 1)), np.zeros((B, Q, Hq, 1))
    for b in range(B):
        g = Hq // k[b].shape[1]
        for i in range(Q):
            n = int(lens[b]) - Q + i + 1
            for h in range(Hq):
                if n <= 0:
                    continue
                kk, vv = k[b][:n, h // g], v[b][:n, h // g]
                s = scale * (kk @ q[b, i, h])
                p = np.exp(s - s.max())
                p /= p.sum()
                out[b, i, h], mass[b, i, h] = p @ vv, p @ np.abs(vv)
                largest[b, i, h] = abs(scale) * (np.abs(kk) @ np.abs(q[b, i, h])).max()
                terms[b, i, h] = n
    return out, mass, largest, terms
