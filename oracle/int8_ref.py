"""Oracle of the INT8 path and of the expert sort with its gradients (test
infrastructure only), NumPy from their definitions:

* int8_quantize: every code and scale, in the fp32 steps that define them;
* the products of int8 rows with scales per token and channel, dense and by
  expert, in float64 (the integer sums are exact there);
* moe_permute, moe_unpermute and its gradients, in float64.

Nothing but the quantiser rounds: the tests bound the rounding themselves.
"""

import numpy as np

F32 = np.float32


def int8_quantize_ref(x):
    """x: float64 [R, K] holding fp32 values.  Returns (q int8, s fp32)."""
    x = x.astype(F32)
    s = np.maximum(np.abs(x).max(axis=1) * (F32(1) / F32(127)), F32(2.0 ** -126))   # (a NaN stays one)
    r = F32(1) / s
    with np.errstate(invalid="ignore"):
        q = np.rint(x * r[:, None])
    return np.where(np.isnan(q), F32(0), q).astype(np.int8), s


def int8_product_ref(xq, xs, wq, ws):
    """(sum xq wq) xs ws, float64 [T, N]."""
    return (xq.astype(np.float64) @ wq.astype(np.float64).T) * xs.astype(np.float64)[:, None] * ws.astype(np.float64)


def group_counts(group_list, kind, M):
    """Rows per expert of a count (1) or cumulative (0) list, clamped to M rows together."""
    n = np.asarray(group_list, np.int64)
    if kind == 0:
        n = np.diff(n, prepend=0)
    end = np.minimum(np.cumsum(np.clip(n, 0, M)), M)
    return np.diff(end, prepend=0)


def gmm_int8_ref(a, a_s, w, w_s, counts, swiglu):
    """(y float64 [M, N] (zeros in rows no expert owns), (gate, up) or None)."""
    M = a.shape[0]
    rows = w.shape[1]
    z = np.zeros((M, rows))
    at = 0
    for e, n in enumerate(counts):
        z[at:at + n] = int8_product_ref(a[at:at + n], a_s[at:at + n], w[e], w_s[e])
        at += n
    if not swiglu:
        return z, None
    g, u = z[:, :rows // 2], z[:, rows // 2:]
    with np.errstate(over="ignore"):
        return g / (1 + np.exp(-g)) * u, (g, u)


def permute_ref(x, topk_ids, E):
    """(rows of x by expert, sorted_row, expanded_row_idx, counts); ids outside
    [0, E) are dropped (expanded_row_idx -1)."""
    k = topk_ids.shape[1]
    ids = topk_ids.reshape(-1).astype(np.int64)
    valid = (ids >= 0) & (ids < E)
    counts = np.bincount(ids[valid], minlength=E)
    sorted_row = np.argsort(np.where(valid, ids, E), kind="stable")[:int(valid.sum())]
    eri = np.full(ids.size, -1, np.int32)
    eri[sorted_row] = np.arange(sorted_row.size, dtype=np.int32)
    return x[sorted_row // k], sorted_row.astype(np.int32), eri, counts


def unpermute_ref(y, eri, k, w=None):
    """out [T, K] float64."""
    T = eri.size // k
    out = np.zeros((T, y.shape[1]))
    for t in range(T):
        for j in range(k):
            p = int(eri.reshape(-1)[t * k + j])
            if 0 <= p < y.shape[0]:
                out[t] += (1.0 if w is None else float(w[t, j])) * y[p]
    return out


def unpermute_backward_ref(dout, eri, k, M, w=None, y=None):
    """(dy [M, K] with NaN in rows that no entry names, dw [T, k] or None), float64."""
    T = eri.size // k
    dy = np.full((M, dout.shape[1]), np.nan)
    dw = np.zeros((T, k)) if y is not None else None
    for t in range(T):
        for j in range(k):
            p = int(eri.reshape(-1)[t * k + j])
            if not 0 <= p < M:
                continue
            dy[p] = (1.0 if w is None else float(w[t, j])) * dout[t]
            if y is not None:
                dw[t, j] = np.dot(dout[t], y[p])
    return dy, dw
