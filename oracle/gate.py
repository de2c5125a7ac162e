"""Router choice, its weights and their gradient (test infrastructure; see the
package docstring).

The pages start from given top-k ids and weights; this is the usual
definition of what produces them.  s = softmax or sigmoid of a token's
logits; the k experts with the largest s (s + bias where a bias is given) in
descending order, ties to the lower index; weights scale * s_j, divided by the
sum of the chosen s with renorm.  Logits of -inf or NaN mask their expert;
slots left without an expert have id -1 and weight 0.  All in float64.
"""

import numpy as np


def _scores(logits, score):
    x = np.asarray(logits, dtype=np.float64)
    masked = np.isnan(x) | (x == -np.inf)
    x = np.where(masked, -np.inf, x)
    if score == "softmax":
        top = x.max(axis=1, keepdims=True)
        d = np.where(x == top, 0.0, x - np.where(np.isfinite(top), top, 0.0))
        d = np.where((top == np.inf) & (x < np.inf), -np.inf, d)
        e = np.where(masked, 0.0, np.exp(d))
        z = e.sum(axis=1, keepdims=True)
        s = e / np.where(z > 0, z, 1.0)
    elif score == "sigmoid":
        with np.errstate(over="ignore"):
            s = np.where(masked, 0.0, 1.0 / (1.0 + np.exp(-np.where(masked, 0.0, x))))
    else:
        raise ValueError("score must be 'softmax' or 'sigmoid'")
    return x, masked, s


def topk_gate(logits, k, score="softmax", bias=None, renorm=True, scale=1.0):
    """(ids [T, k] int32, weights [T, k] float64)."""
    x, masked, s = _scores(logits, score)
    key = x if bias is None else s + np.asarray(bias, dtype=np.float64)
    key = np.where(masked | np.isnan(key), -np.inf, key)
    order = np.argsort(-key, axis=1, kind="stable")[:, :k]
    picked = np.take_along_axis(key, order, axis=1)
    ids = np.where(picked > -np.inf, order, -1).astype(np.int32)
    return ids, slot_weights(logits, ids, score, renorm) * scale


def slot_weights(logits, ids, score, renorm):
    """Unscaled weights of given ids: s, or s over the sum of the chosen s."""
    x, masked, s = _scores(logits, score)
    ids = np.asarray(ids, dtype=np.int64)
    idx = np.clip(ids, 0, x.shape[1] - 1)
    live = (ids >= 0) & (ids < x.shape[1]) & ~np.take_along_axis(masked, idx, axis=1)
    if not renorm:
        return np.where(live, np.take_along_axis(s, idx, axis=1), 0.0)
    # log of the scores up to a common factor, so that none underflows
    l = np.take_along_axis(x, idx, axis=1)
    l = np.where(live, l, 0.0)
    log_s = l if score == "softmax" else np.minimum(l, 0.0) - np.log1p(np.exp(-np.abs(l)))
    log_s = np.where(live, log_s, -np.inf)
    top = log_s.max(axis=1, keepdims=True)
    top = np.where(top > -np.inf, top, 0.0)
    with np.errstate(invalid="ignore"):                 # two logits at +inf: set to 1 below
        e = np.where(live, np.exp(np.where(live, log_s, top) - top), 0.0)
    e = np.where(live & (log_s == top), 1.0, e)
    z = e.sum(axis=1, keepdims=True)
    return e / np.where(z > 0, z, 1.0)


def topk_gate_bwd(logits, ids, dweights, score="softmax", renorm=True, scale=1.0):
    """Gradient of sum(weights * dweights) with respect to the logits, the ids
    held fixed.  [T, E] float64."""
    x, masked, s = _scores(logits, score)
    T, E = x.shape
    ids = np.asarray(ids, dtype=np.int64)
    w = slot_weights(logits, ids, score, renorm)
    idx = np.clip(ids, 0, E - 1)
    live = (ids >= 0) & (ids < E) & ~np.take_along_axis(masked, idx, axis=1)
    g = np.where(live, np.asarray(dweights, dtype=np.float64) * scale, 0.0)
    mean = (g * w).sum(axis=1, keepdims=True)
    out = np.zeros((T, E))
    if score == "softmax":
        if renorm:
            d = w * (g - mean)
        else:
            out -= mean * s
            d = w * g
    else:
        p = np.take_along_axis(s, idx, axis=1)
        d = w * (g - (mean if renorm else 0.0)) * (1.0 - p)
    for t in range(T):
        for j in range(ids.shape[1]):
            if live[t, j]:
                out[t, ids[t, j]] += d[t, j]
    return out
