"""Plain 64-bit forms of the gated feed-forward operators, for their tests (CPU, NumPy).

Weights come from the CPU oracle's exact dequantisation; everything here is the definition written out.
"""
from __future__ import annotations

import math

import numpy as np

ACTS = ("silu", "gelu_tanh", "gelu")

_erf = np.vectorize(math.erf, otypes=[np.float64])


def act(g: np.ndarray, kind: str):
    """act(g) and act'(g) in float64."""
    if kind == "silu":
        p = 0.5 * (1 + np.tanh(0.5 * g))
        return g * p, p * (1 + g * (1 - p))
    if kind == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = np.tanh(c * (g + 0.044715 * g ** 3))
        return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * c * (1 + 3 * 0.044715 * g ** 2)
    p = 0.5 * (1 + _erf(g / math.sqrt(2)))
    return g * p, p + g * np.exp(-0.5 * g * g) / math.sqrt(2 * math.pi)


def save8(v: np.ndarray):
    """float64 [rows][cols] -> (codes int8 [rows][cp], exponents uint8 [rows][cp / 16])."""
    rows, cols = v.shape
    cp = -(-cols // 16) * 16
    p = np.zeros((rows, cp))
    p[:, :cols] = v
    p = p.reshape(rows, cp // 16, 16)
    top = np.abs(p).max(-1)
    bad = ~np.isfinite(top) | (top >= 2.0 ** 128 * (1 - 2.0 ** -8))
    q = np.where(bad[..., None], 0.0, p)
    top = np.where(bad, 0.0, top)
    e = np.where(top > 0, np.floor(np.log2(np.where(top > 0, top, 1.0))), -1000).astype(np.int64)
    e = e - (2.0 ** np.clip(e, -1022, 1023) > top)  # log2 may round up at a power of two
    E = np.maximum(e - 6 + 127, 1)
    E = E + (np.rint(np.ldexp(top, 127 - E)) > 127)
    codes = np.rint(np.ldexp(q, 127 - E[..., None])).astype(np.int8)
    return codes.reshape(rows, cp), np.where(bad, 255, E).astype(np.uint8)


def restore8(codes: np.ndarray, exps: np.ndarray, cols: int) -> np.ndarray:
    rows = codes.shape[0]
    v = np.ldexp(codes.reshape(rows, -1, 16).astype(np.float64), exps.astype(np.int64)[..., None] - 127)
    v = np.where((exps == 255)[..., None], np.nan, v)
    return v.reshape(rows, -1)[:, :cols]


def gated_backward(g, u, dh, kind: str):
    """(dg | du) in float64."""
    a, d = act(g, kind)
    return np.concatenate((dh * u * d, dh * a), 1)
