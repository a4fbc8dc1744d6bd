"""Rotary positions with several axes, in float64."""
from __future__ import annotations

import numpy as np


def ladder(widths, theta: float, per_axis: bool):
    """Each pair's frequency (radians a step) and axis."""
    freq, axis = [], []
    for a, w in enumerate(widths):
        for i in range(w // 2):
            freq.append(theta ** (-2.0 * i / w) if per_axis else theta ** (-2.0 * len(freq) / sum(widths)))
            axis.append(a)
    return np.array(freq), np.array(axis)


def turn(x: np.ndarray, positions: np.ndarray, freq, axis, interleaved: bool) -> np.ndarray:
    """Rows x [T, H, D] turned by positions [T, axes]."""
    y = np.array(x, np.float64)
    n = len(freq)
    angle = np.asarray(positions, np.float64)[:, axis] * freq
    cos, sin = np.cos(angle)[:, None], np.sin(angle)[:, None]
    first, second = (np.arange(0, 2 * n, 2), np.arange(1, 2 * n, 2)) if interleaved else (np.arange(n), np.arange(n, 2 * n))
    a, b = y[..., first], y[..., second]
    y[..., first], y[..., second] = a * cos - b * sin, a * sin + b * cos
    return y
