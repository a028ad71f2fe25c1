"""Oracle of the operators around the expert layer (test infrastructure only),
NumPy in float64 from their definitions:

* add_rmsnorm: h = x + residual, n = h / sqrt(mean(h^2) + eps) * weight;
* the activations and the epilogue of the fused linear;
* routing of rows that are MXFP8 already: route_ref's permutation applied to
  the payload and scale rows.

Nothing is rounded here: the tests round, or bound the rounding, themselves.
"""

import math

import numpy as np

from .moe_ref import route_ref, route_ref_fast
from .mx_ref import BLOCK, block_scale_exponent


def add_rmsnorm_ref(x, residual, weight, eps):
    """x, residual (or None): float64 [T, K]; weight float64 [K].  Returns (h, n)."""
    h = x if residual is None else x + residual
    ms = np.array([math.fsum(row * row) / row.size for row in h]) if h.size < 1 << 20 else np.mean(h * h, axis=1)
    return h, h / np.sqrt(ms + eps)[:, None] * weight


def activate_ref(z, act):
    """none, relu, silu, gelu (z * Phi(z)) or gelu_tanh (its tanh form)."""
    if act == "none":
        return z
    if act == "relu":
        return np.maximum(z, 0.0)
    with np.errstate(over="ignore"):
        if act == "silu":
            return z / (1.0 + np.exp(-z))
        if act == "gelu":
            return z * 0.5 * np.vectorize(math.erfc, otypes=[np.float64])(-z / math.sqrt(2.0))
        assert act == "gelu_tanh", act
        return z * 0.5 * (1.0 + np.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3)))


def linear_fused_ref(x, w, bias, act, residual):
    """act(x . w^T + bias) + residual on float64 values."""
    z = x @ w.T
    if bias is not None:
        z = z + bias
    z = activate_ref(z, act)
    return z if residual is None else z + residual


def route_mx_ref(q, s, topk_ids, E):
    """(xq, xs, sorted_row, expanded_row_idx, counts): MXFP8 rows [T, K] and
    their scales sent to the experts' rows, each row as it is."""
    T, k = topk_ids.shape
    counts, sorted_row, eri = (route_ref if T * k <= 4096 else route_ref_fast)(topk_ids, E)
    token = sorted_row.astype(np.int64) // k
    return q[token], s[token], sorted_row, eri, counts


def block_exponents(n):
    """Shared exponents and largest magnitudes of the 32-element blocks of
    float64 rows [R, K]: (exponent [R, nb], amax [R, nb])."""
    R, K = n.shape
    nb = -(-K // BLOCK)
    pad = np.zeros((R, nb * BLOCK))
    pad[:, :K] = np.abs(n)
    amax = pad.reshape(R, nb, BLOCK).max(axis=2)
    return block_scale_exponent(amax), amax
