"""Gradients of the routed-expert layer's steps (test infrastructure; see the
package docstring): the token permutation, the weighted combine, the grouped
matmul's input and the SiLU-gated activation, each the plain derivative of the
forward definition in this package, in float64.
"""

import numpy as np

from .gmm import dense_weights


def _pairs(pair_row, T, k, rows):
    pr = np.asarray(pair_row, dtype=np.int64).reshape(T, k)
    return pr, (pr >= 0) & (pr < rows)


def dispatch(x, pair_row, rows, fill=np.nan):
    """xs[pair_row[t*k + j]] = x[t]; rows no pair names hold `fill`."""
    x = np.asarray(x, dtype=np.float64)
    T = x.shape[0]
    pr, ok = _pairs(pair_row, T, len(pair_row) // T, rows)
    xs = np.full((rows, x.shape[1]), fill)
    for j in range(pr.shape[1]):
        xs[pr[ok[:, j], j]] = x[ok[:, j]]
    return xs


def dispatch_bwd(dxs, pair_row, k):
    """dx[t] = sum_j dxs[pair_row[t*k + j]]."""
    dxs = np.asarray(dxs, dtype=np.float64)
    T = len(pair_row) // k
    pr, ok = _pairs(pair_row, T, k, dxs.shape[0])
    dx = np.zeros((T, dxs.shape[1]))
    for j in range(k):
        dx[ok[:, j]] += dxs[pr[ok[:, j], j]]
    return dx


def combine_bwd(dout, y, topk_weights, pair_row, fill=np.nan):
    """(dy [rows, N], dweights [T, k]); rows of dy no pair names hold `fill`."""
    dout = np.asarray(dout, dtype=np.float64)
    y = np.asarray(y, dtype=np.float64)
    w = np.asarray(topk_weights, dtype=np.float64)
    T, k = w.shape
    pr, ok = _pairs(pair_row, T, k, y.shape[0])
    dy = np.full(y.shape, fill)
    dw = np.zeros((T, k))
    for j in range(k):
        o = ok[:, j]
        dy[pr[o, j]] = w[o, j, None] * dout[o]
        dw[o, j] = (dout[o] * y[pr[o, j]]).sum(axis=1)
    return dy, dw


def gmm_dgrad(dy, group_offsets, w, absolute=False):
    """dX[r, :] = dY[r, :] @ W[e] for every row r of band e; rows of no band
    NaN.  absolute: the same with |dY| and |W| (the scale of its rounding)."""
    dy = np.asarray(dy, dtype=np.float64)
    off = np.asarray(group_offsets, dtype=np.int64)
    out = None
    for e in range(off.size - 1):
        lo, hi = int(off[e]), int(off[e + 1])
        if hi > lo or out is None:
            W = dense_weights(w, e)                  # [N, K]
            if out is None:
                out = np.full((dy.shape[0], W.shape[1]), np.nan)
            if absolute:
                out[lo:hi] = np.abs(dy[lo:hi]) @ np.abs(W)
            else:
                out[lo:hi] = dy[lo:hi] @ W
    return out


def silu_mul_bwd(preact, dh):
    """Gradient of act.silu_mul's input: [M, 2K] from preact [M, 2K] and dh
    [M, K]."""
    p = np.asarray(preact, dtype=np.float64)
    dh = np.asarray(dh, dtype=np.float64)
    h = p.shape[1] // 2
    g, u = p[:, :h], p[:, h:]
    with np.errstate(over="ignore"):
        s = 1.0 / (1.0 + np.exp(-g))
    return np.concatenate([dh * u * s * (1.0 + g * (1.0 - s)), dh * g * s], axis=1)
