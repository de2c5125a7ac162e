"""The dense half of the layer (test infrastructure; see the package
docstring): 4-bit integer weights with group scales, and the gated block with
its gradients, each the plain definition in float64.
"""

import numpy as np

from .act import silu_mul
from .grad import silu_mul_bwd


def w4_weights(codes, scales, zeros=None):
    """[N, K] float64 weights of codes [N, K/2] (the even k in the low nibble),
    scales [N, K/G] and zero points [N, K/G] (8 everywhere without them)."""
    codes = np.asarray(codes)
    scales = np.asarray(scales, dtype=np.float64)
    n, half = codes.shape
    c = np.empty((n, 2 * half))
    c[:, 0::2] = codes & 15
    c[:, 1::2] = codes >> 4
    group = 2 * half // scales.shape[1]
    z = np.full(scales.shape, 8.0) if zeros is None else np.asarray(zeros, dtype=np.float64)
    return (c - np.repeat(z, group, axis=1)) * np.repeat(scales, group, axis=1)


def w4_gemv(codes, scales, x, zeros=None, topk_ids=None, topk_weights=None, act=False):
    """y[t] = W x[t]; with ids [T, k] and codes [E, N, K/2] a row per pair (x has
    T or T*k rows), or with weights [T, k] too a token's rows summed.  Pairs of
    ids outside [0, E) give zeros."""
    x = np.asarray(x, dtype=np.float64)
    if topk_ids is None:
        y = x @ w4_weights(codes, scales, zeros).T
        return silu_mul(y) if act else y
    ids = np.asarray(topk_ids)
    T, k = ids.shape
    E, N = np.asarray(codes).shape[:2]
    y = np.zeros((T * k, N))
    for t in range(T):
        for j in range(k):
            e = int(ids[t, j])
            if 0 <= e < E:
                p = t * k + j
                w = w4_weights(codes[e], scales[e], None if zeros is None else zeros[e])
                y[p] = w @ x[t if x.shape[0] == T else p]
    if topk_weights is not None:
        live = (ids >= 0) & (ids < E)
        w = np.where(live, np.asarray(topk_weights, dtype=np.float64), 0.0)
        return (y.reshape(T, k, N) * w[:, :, None]).sum(axis=1)
    return silu_mul(y) if act else y


def gate_up(x, w13):
    """(h [M, N/2], sums [M, N]) of x [M, K] and w13 [N, K]."""
    y = np.asarray(x, dtype=np.float64) @ np.asarray(w13, dtype=np.float64).T
    return silu_mul(y), y


def gate_up_bwd(dh, x, w13, preact):
    """(dx [M, K], dw13 [N, K], d [M, N])."""
    d = silu_mul_bwd(preact, dh)
    return d @ np.asarray(w13, dtype=np.float64), d.T @ np.asarray(x, dtype=np.float64), d
