"""The oracle's router and gradients against closed forms and central
differences (float64, no GPU)."""

import itertools

import numpy as np
import pytest

import oracle


def _difference(f, x, h=1e-6):
    """Central differences of the scalar f over every entry of x."""
    g = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        a = x.copy()
        a[i] += h
        b = x.copy()
        b[i] -= h
        g[i] = (f(a) - f(b)) / (2 * h)
    return g


def test_gate_closed_forms():
    ids, w = oracle.topk_gate(np.log([[1.0, 2.0, 4.0, 1.0]]), 2, "softmax", renorm=False)
    assert ids.tolist() == [[2, 1]]
    assert np.allclose(w, [[0.5, 0.25]], atol=1e-15)
    ids, w = oracle.topk_gate(np.log([[1.0, 2.0, 4.0, 1.0]]), 2, "softmax", renorm=True, scale=3.0)
    assert np.allclose(w, [[2.0, 1.0]], atol=1e-14)
    ids, w = oracle.topk_gate(np.array([[0.0, np.log(3.0)]]), 2, "sigmoid", renorm=False)
    assert ids.tolist() == [[1, 0]] and np.allclose(w, [[0.75, 0.5]], atol=1e-15)


def test_gate_ties_masks_and_bias():
    ids, _ = oracle.topk_gate(np.zeros((1, 5)), 3)
    assert ids.tolist() == [[0, 1, 2]]                       # ties: the lowest index
    x = np.array([[-np.inf, np.nan, 1.0, -np.inf], [-np.inf] * 4, [np.inf, 0.0, 0.0, 0.0]])
    ids, w = oracle.topk_gate(x, 2)
    assert ids.tolist() == [[2, -1], [-1, -1], [0, 1]]
    assert w.tolist() == [[1.0, 0.0], [0.0, 0.0], [1.0, 0.0]]
    # the bias steers the choice, not the weights
    ids, w = oracle.topk_gate(np.array([[0.0, 0.0, 0.0]]), 1, "sigmoid", bias=[0.0, 0.0, 1.0], renorm=False)
    assert ids.tolist() == [[2]] and w.tolist() == [[0.5]]
    # renormalised weights keep their ratio where the scores underflow
    _, w = oracle.topk_gate(np.array([[-2000.0, -2000.0 + np.log(3.0)]]), 2, "sigmoid")
    assert np.allclose(w, [[0.75, 0.25]], rtol=1e-9)


@pytest.mark.parametrize("score,renorm", itertools.product(["softmax", "sigmoid"], [False, True]))
def test_gate_gradient_is_the_difference(score, renorm):
    rng = np.random.default_rng(401)
    T, E, k = 4, 7, 3
    x = rng.standard_normal((T, E)) * 1.5
    x[1, 2] = -np.inf
    ids, _ = oracle.topk_gate(x, k, score)
    ids[2, 1] = -1
    g = rng.standard_normal((T, k))
    got = oracle.topk_gate_bwd(x, ids, g, score, renorm, scale=1.7)
    f = lambda a: float((oracle.slot_weights(a, ids, score, renorm) * 1.7 * np.where(ids >= 0, g, 0)).sum())  # noqa: E731
    ref = _difference(f, np.where(np.isfinite(x), x, -1e9))
    assert np.abs(got - ref).max() < 1e-8


def test_permutation_gradients_are_adjoint_and_differences():
    rng = np.random.default_rng(402)
    T, k, E, N = 5, 2, 3, 4
    ids = rng.integers(0, E, size=(T, k))
    ids[3, 1] = -1
    r = oracle.route_sort(ids, E)
    pr, M = r["pair_row"], T * k
    x, y, dxs = rng.standard_normal((T, N)), rng.standard_normal((M, N)), rng.standard_normal((M, N))
    w, dout = rng.standard_normal((T, k)), rng.standard_normal((T, N))
    xs = oracle.dispatch(x, pr, M)
    assert np.isnan(xs).any(axis=1).sum() == 1                 # the dropped pair's row
    f = lambda a: float(np.nansum(oracle.dispatch(a, pr, M) * dxs))  # noqa: E731
    assert np.abs(oracle.dispatch_bwd(dxs, pr, k) - _difference(f, x)).max() < 1e-8
    dy, dw = oracle.combine_bwd(dout, y, w, pr, fill=0.0)
    fy = lambda a: float((oracle.combine(a, w, pr) * dout).sum())  # noqa: E731
    fw = lambda a: float((oracle.combine(y, a, pr) * dout).sum())  # noqa: E731
    assert np.abs(dy - _difference(fy, y)).max() < 1e-8
    assert np.abs(dw - _difference(fw, w)).max() < 1e-8


def test_product_and_activation_gradients_are_differences():
    rng = np.random.default_rng(403)
    E, N, K = 2, 4, 32
    w = {"fmt": "mxfp4", "codes": rng.integers(0, 256, size=(E, N, K // 2), dtype=np.uint8),
         "scales": rng.integers(125, 129, size=(E, N, 1)).astype(np.uint8)}
    off = np.array([0, 2, 3])
    from oracle.gmm import gmm_dense_x
    x, dy = rng.standard_normal((3, K)), rng.standard_normal((3, N))
    f = lambda a: float((gmm_dense_x(a, None, off, w) * dy).sum())  # noqa: E731
    assert np.abs(oracle.gmm_dgrad(dy, off, w) - _difference(f, x)).max() < 1e-7
    assert (oracle.gmm_dgrad(dy, off, w, absolute=True) >= np.abs(oracle.gmm_dgrad(dy, off, w))).all()
    pre, dh = rng.standard_normal((3, 8)) * 2, rng.standard_normal((3, 4))
    h = lambda a: float((oracle.silu_mul(a) * dh).sum())  # noqa: E731
    assert np.abs(oracle.silu_mul_bwd(pre, dh) - _difference(h, pre)).max() < 1e-8
