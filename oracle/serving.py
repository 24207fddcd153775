"""References of the token-serving operators in fp64: the weight-only linear layer and
the attention of one new token over a paged cache, each with the magnitudes that an
error bound needs.

    wlinear:  Y[m, n] = t * sum_k X[m, k] (E*D)_w[n, k] + bias[n]
    attention of sequence b, query head h (kv head h // G) over its visible tokens j:
        s_j = scale * q . k_j,  lse = log sum_j exp s_j,  out = sum_j exp(s_j - lse) v_j
        visible: max(0, L - window) <= j < L (window 0: all below L), j in a page of
        the table whose id names a page of the cache.  None visible: out 0, lse -inf.

Appending to a cache is ``nvfp4.quantize`` of the rows under the cache's tensor scale.
"""
from __future__ import annotations

import numpy as np

from . import mxfp4
from .nvfp4 import dequantize
from .qlinear import operand_exact


def wlinear_ref64(x, data, scales, t=None, bias=None, rows=None):
    """x [M, K] fp64; a record blocked along K (t None: MXFP4), or its rows ``rows``.
    Returns (Y, S) with S[m, n] = |t| sum_k |x w| + |bias|."""
    w = (mxfp4.operand_exact(data, scales, rows) if t is None
         else operand_exact(data, scales, rows) * float(t))
    y, s = x @ w.T, np.abs(x) @ np.abs(w).T
    if bias is not None:
        y, s = y + bias, s + np.abs(bias)
    return y, s


def cache_rows_f64(values, scales=None, t=None):
    """Rows of a cache as fp64 [..., dim]: fp values as they are, or NVFP4 rows."""
    if scales is None:
        return np.asarray(values, dtype=np.float64)
    shape = values.shape[:-1] + (2 * values.shape[-1],)
    return dequantize(values.reshape(-1, values.shape[-1]), scales.reshape(-1, scales.shape[-1]),
                      t).astype(np.float64).reshape(shape)


def visible(length, table_row, page_size, num_pages, window=0):
    """(page id, row of the page) of every visible token, ascending."""
    first = max(0, int(length) - window) if window else 0
    j = np.arange(first, max(first, min(int(length), len(table_row) * page_size)))
    ids = np.asarray(table_row, dtype=np.int64)[j // page_size] if len(j) else np.zeros(0, np.int64)
    ok = (ids >= 0) & (ids < num_pages)
    return ids[ok], (j % page_size)[ok]


def attend_ref64(q, k, v, scale):
    """q [Hq, D], k and v [n, Hkv, D] (visible tokens), fp64.  Returns out [Hq, D], lse
    [Hq], and for the bounds: A[h] = max_j scale sum_d |q_d k_jd| (the scores'
    magnitude), V[h, d] = sum_j p_j |v_jd| and E[h] = sum_j exp(s_j - max s)."""
    Hq, D = q.shape
    n, Hkv = k.shape[:2]
    G = Hq // Hkv
    out, lse = np.zeros((Hq, D)), np.full(Hq, -np.inf)
    A, V, E = np.zeros(Hq), np.zeros((Hq, D)), np.ones(Hq)
    if n == 0:
        return out, lse, A, V, E
    for h in range(Hq):
        kk, vv = k[:, h // G], v[:, h // G]
        s = scale * (kk @ q[h])
        top = s.max()
        e = np.exp(s - top)
        lse[h] = top + np.log(e.sum())
        p = e / e.sum()
        out[h] = p @ vv
        A[h] = abs(scale) * (np.abs(kk) @ np.abs(q[h])).max()
        V[h] = p @ np.abs(vv)
        E[h] = e.sum()
    return out, lse, A, V, E
