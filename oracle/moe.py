"""CPU oracle: the router and the AWQ W4A16 expert layer of a mixture of experts.

TEST INFRASTRUCTURE (same import rule as ``oracle.svdquant``).  Parity
status: pinned by ``tests/test_oracle_serving.py``.

    logits = x w^T;  score = softmax over the experts, or sigmoid
    ids    = the top_k largest of score + bias (of the logits without a bias),
             the lower index first among equals
    weight = score of the choice (/ the sum of the choices' scores)
    y_t    = sum_j weight_tj Down_e (act(Gate_e x_t) * (Up_e x_t)),  e = ids_tj

Everything in float64; expert matrices are ``oracle.awq`` weights.
"""
from __future__ import annotations

import math

import numpy as np

from . import awq


def route(x, w, top_k, bias=None, score="softmax", normalize=True):
    logits = np.asarray(x, np.float64) @ np.asarray(w, np.float64).T
    if score == "softmax":
        s = np.exp(logits - logits.max(1, keepdims=True))
        s /= s.sum(1, keepdims=True)
    else:
        s = 1.0 / (1.0 + np.exp(-logits))
    key = logits if bias is None else s + np.asarray(bias, np.float64)
    ids = np.argsort(-key, axis=1, kind="stable")[:, :top_k]
    wt = np.take_along_axis(s, ids, 1)
    if normalize:
        wt = wt / wt.sum(1, keepdims=True)
    return ids.astype(np.int32), wt


def activate(g, act):
    if act == "silu":
        return g / (1.0 + np.exp(-g))
    return 0.5 * g * (1.0 + np.tanh(math.sqrt(2.0 / math.pi) * (g + 0.044715 * g ** 3)))


def _magnitude(x, s, z):
    """sum_g s sum_{k in g} |x| (128 + 15 + 128 + z): the size of the terms of
    a product formed as sum x (128 + code) - (128 + z) sum x."""
    a = np.abs(x).reshape(len(x), -1, awq.GROUP).sum(2)
    return a @ (np.abs(s.astype(np.float64)) * (271.0 + z.astype(np.float64))).T


def layer(x, gate_up, down, ids, weights, act="silu"):
    """x [T, K]; gate_up, down: lists over the experts of (q [N, K] codes, s,
    z).  Returns (y, bound) float64 [T, K]: bound is what float32 sums in any
    order, the terms' sizes as in ``_magnitude``, and h kept to 2^-17, can
    move y by."""
    x = np.asarray(x, np.float64)
    T, K = x.shape
    u = 2.0 ** -24
    y, bound = np.zeros((T, K)), np.zeros((T, K))
    for t in range(T):
        for j, e in enumerate(ids[t]):
            if not 0 <= e < len(gate_up):
                continue
            qg, sg, zg = gate_up[e]
            I = qg.shape[0] // 2
            gu = awq.forward(x[t:t + 1], qg, sg, zg)[0]
            err = (64 + K // 64 + 8) * u * _magnitude(x[t:t + 1], sg, zg)[0]
            g, up = gu[:I], gu[I:]
            a = activate(g, act)
            h = a * up
            # |act'| <= 1.2 for both; the device's exponential and division are good to 2^-20
            herr = (1.2 * err[:I] + 2.0 ** -20 * np.abs(a)) * (np.abs(up) + err[I:]) + np.abs(a) * err[I:] \
                + 2.0 ** -16 * np.abs(h)
            qd, sd, zd = down[e]
            d = awq.forward(h[None], qd, sd, zd)[0]
            w = float(weights[t][j])
            y[t] += w * d
            spread = np.abs(awq.dequantize(qd, sd, zd)) @ herr
            bound[t] += abs(w) * (spread + (128 + I // 64 + 8) * u * _magnitude(h[None], sd, zd)[0]
                                  + (len(ids[t]) + 2) * u * np.abs(d))
    return y, bound
