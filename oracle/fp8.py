"""The linear in 8-bit floating point (e4m3, scales for blocks of 128), in float64."""
from __future__ import annotations

import numpy as np


def e4m3(v: np.ndarray) -> np.ndarray:
    """The nearest e4m3 value of |v| <= 448, ties to even: three bits behind the first, steps of 2^-9 below 2^-6."""
    v = np.asarray(v, np.float64)
    step = np.exp2(np.floor(np.log2(np.maximum(np.abs(v), 2.0 ** -6))) - 3)
    return np.rint(v / step) * step


def decode(codes: np.ndarray) -> np.ndarray:
    """The values of e4m3 bit patterns."""
    c = np.asarray(codes, np.uint8).astype(np.int64)
    e, m = c >> 3 & 15, c & 7
    v = np.where(e == 0, m / 8.0 * 2.0 ** -6, (1 + m / 8.0) * np.exp2(e - 7.0))
    v = np.where(e * 8 + m == 127, np.nan, v)
    return np.where(c & 128, -v, v)


def blocks(K: int) -> int:
    return -(-K // 128)


def quantize_rows(x: np.ndarray):
    """x [M, K] float64 of 16-bit values -> (values of the codes [M, K], scale exponents [M, blocks])."""
    M, K = x.shape
    v, e = np.empty((M, K)), np.empty((M, blocks(K)), np.int64)
    for b in range(blocks(K)):
        part = x[:, 128 * b:128 * (b + 1)]
        top = np.abs(part).max(1) if part.size else np.zeros(M)
        exp = np.full(M, -127)
        for i, t in enumerate(top):
            if not np.isfinite(t):
                exp[i] = 0
                continue
            while t > 448 * 2.0 ** exp[i]:
                exp[i] += 1
        e[:, b] = exp
        with np.errstate(invalid="ignore"):
            v[:, 128 * b:128 * (b + 1)] = np.where(np.isfinite(top)[:, None], e4m3(part / np.exp2(exp.astype(float))[:, None]), np.nan)
    return v, e


def forward(x: np.ndarray, codes: np.ndarray, scales: np.ndarray, bias=None):
    """(x Q8) W^T + bias and the sum of its terms' magnitudes, which its float32 sums round relative to."""
    v, e = quantize_rows(x)
    N, K = codes.shape
    xq = v * np.exp2(np.repeat(e, 128, 1)[:, :K].astype(np.float64))
    w = decode(codes) * np.repeat(np.repeat(scales.astype(np.float64), 128, 0)[:N], 128, 1)[:, :K]
    y, size = xq @ w.T, np.abs(xq) @ np.abs(w).T
    if bias is not None:
        y, size = y + bias, size + np.abs(bias)
    return y, size


def gelu(y: np.ndarray) -> np.ndarray:
    return y / (1 + np.exp(np.minimum(-2 * np.sqrt(2 / np.pi) * (y + 0.044715 * y ** 3), 700)))
