"""Plain 64-bit forms of the 8-bit integer lane (numpy): row quantisation, the product with
token and channel scales, and the mixture-of-experts layer over int8 experts."""
from __future__ import annotations

from fractions import Fraction

import numpy as np

from .q4k import bf16_to_f64, route_topk


def quantize_rows(x_bits: np.ndarray):
    """bf16 bit patterns [M][K] -> (codes int8 [M][K], scales fp32 [M]); finite rows.

    The code is 127 x / amax rounded to nearest, ties to even. In 64 bits the quotient of a
    15-bit by an 8-bit number is close enough to tell a tie, and exact where there is one."""
    x = bf16_to_f64(x_bits)
    amax = np.abs(x).max(axis=1, keepdims=True)
    q = np.rint(np.divide(127.0 * x, amax, out=np.zeros_like(x), where=amax > 0))
    return q.astype(np.int8), (amax[:, 0] / 127.0).astype(np.float32)


def code_exact(x: float, amax: float) -> int:
    """One code by rational arithmetic."""
    return round(Fraction(127) * Fraction(x) / Fraction(amax))


def matmul_ref(W, w_scale, X, x_scale):
    """(64-bit value, the three fp32 roundings of the definition) of X W^T with scales."""
    acc = X.astype(np.int64) @ W.astype(np.int64).T
    y = acc * np.asarray(x_scale, np.float64)[:, None] * np.asarray(w_scale, np.float64)
    y32 = acc.astype(np.float32) * np.asarray(x_scale, np.float32)[:, None] * np.asarray(w_scale, np.float32)
    return y, y32


def silu(g):
    return g / (1.0 + np.exp(-g))


def moe_layer_ref(logits, topk, W_gate_up, s_gate_up, W_down, s_down, x_bits, residual=None):
    """The layer in 64 bits, token by token."""
    ids, _ = route_topk(logits, topk)
    x = bf16_to_f64(x_bits)
    F = W_down.shape[2]
    y = np.zeros((x.shape[0], W_down.shape[1])) if residual is None else residual.astype(np.float64)
    for t in range(x.shape[0]):
        v = logits[t, ids[t]].astype(np.float64)
        p = np.exp(v - v.max())
        p /= p.sum()
        for e, pe in zip(ids[t], p):
            gu = (W_gate_up[e].astype(np.float64) @ x[t]) * s_gate_up[e]
            h = silu(gu[:F]) * gu[F:]
            y[t] += pe * (W_down[e].astype(np.float64) @ h) * s_down[e]
    return y
