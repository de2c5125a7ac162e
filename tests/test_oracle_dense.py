"""The oracle's 4-bit integer products and dense gated block, pinned to closed
forms, loops and differences."""

import numpy as np

import oracle


def test_w4_weights_by_hand():
    codes = np.array([[0x10, 0x32], [0xFE, 0x88]], dtype=np.uint8)
    assert np.array_equal(oracle.w4_weights(codes, [[2.0], [0.5]]),
                          [[-16, -14, -12, -10], [3, 3.5, 0, 0]])
    assert np.array_equal(oracle.w4_weights(codes, [[1, 10], [1, 1]], [[0, 1], [14, 8]]),
                          [[0, 1, 10, 20], [0, 1, 0, 0]])


def test_w4_forms_agree():
    rng = np.random.default_rng(1)
    E, N, K, G, T, k = 4, 6, 64, 32, 5, 2
    codes = rng.integers(0, 256, (E, N, K // 2), dtype=np.uint8)
    scales, zeros = rng.random((E, N, K // G)), rng.integers(0, 16, (E, N, K // G))
    x = rng.standard_normal((T, K))
    ids = rng.integers(0, E, (T, k))
    ids[1, 0], ids[3, 1] = -1, E
    w = rng.random((T, k))
    y = oracle.w4_gemv(codes, scales, x, zeros, ids)
    for t in range(T):
        for j in range(k):
            want = np.zeros(N)
            if 0 <= ids[t, j] < E:
                e = ids[t, j]
                for n in range(N):
                    for i in range(K):
                        c = (codes[e, n, i // 2] >> (4 * (i % 2))) & 15
                        want[n] += scales[e, n, i // G] * (int(c) - zeros[e, n, i // G]) * x[t, i]
            assert np.allclose(y[t * k + j], want, rtol=1e-12, atol=1e-12)
    s = oracle.w4_gemv(codes, scales, x, zeros, ids, w)
    assert np.allclose(s, (y.reshape(T, k, N) * w[:, :, None]).sum(1), rtol=1e-12, atol=1e-12)
    per = oracle.w4_gemv(codes, scales, np.repeat(x, k, axis=0), zeros, ids)
    assert np.array_equal(per, y)
    d = oracle.w4_gemv(codes[0], scales[0], x, zeros[0], act=True)
    full = oracle.w4_gemv(codes[0], scales[0], x, zeros[0])
    assert np.allclose(d, full[:, :3] / (1 + np.exp(-full[:, :3])) * full[:, 3:], rtol=1e-12)


def test_gate_up_gradients_against_differences():
    rng = np.random.default_rng(2)
    M, N, K = 3, 8, 5
    x, w, v = rng.standard_normal((M, K)), rng.standard_normal((N, K)), rng.standard_normal((M, N // 2))
    _, pre = oracle.gate_up(x, w)
    dx, dw, d = oracle.gate_up_bwd(v, x, w, pre)
    assert d.shape == (M, N)
    for base, grad in ((x, dx), (w, dw)):
        for i in range(base.shape[0]):
            for j in range(base.shape[1]):
                ends = []
                for step in (-1e-5, 1e-5):
                    old = base[i, j]
                    base[i, j] = old + step
                    ends.append((v * oracle.gate_up(x, w)[0]).sum())
                    base[i, j] = old
                assert abs((ends[1] - ends[0]) / 2e-5 - grad[i, j]) < 1e-7
