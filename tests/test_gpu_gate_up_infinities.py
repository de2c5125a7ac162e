"""f32 gradients of the dense block with infinities and NaN in w13 (dx) and in x
(dw13), whose d is kept as three bf16 values: every result must be the infinity
or the NaN that the sum of the whole values' products is, and the others are
untouched.

Finite results: small integers are exact (bit for bit the oracle's); random ones
to the suite's max|delta| / max|ref| <= 1e-5.
"""

import numpy as np
import pytest
import torch

import moe_grouped_gemm_route_amd as moe
import oracle
from tests.gpu_util import DEV, REL_TOL

pytestmark = pytest.mark.gpu

F, B = moe.F32, moe.BF16
INF, NAN = float("inf"), float("nan")


def product(a, b):
    """a @ b in float64; columns of b that are not finite by plain sums of
    products (a BLAS may leave out a zero's)."""
    out = a @ np.where(np.isfinite(b), b, 0.0)
    with np.errstate(invalid="ignore"):
        for j in np.nonzero(~np.isfinite(b).all(axis=0))[0]:
            out[:, j] = (a * b[:, j]).sum(axis=1)
    return out


def same(got, want, exact):
    got = got.double().cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(want))
    over = np.isinf(want)
    assert np.array_equal(np.isinf(got), over) and np.array_equal(got[over], want[over])
    finite = np.isfinite(want)
    assert finite.any()
    if exact:
        assert np.array_equal(got[finite], want[finite])
    else:
        assert np.max(np.abs(got[finite] - want[finite])) <= REL_TOL * np.max(np.abs(want[finite]))


def inputs(seed, M, N, K, exact):
    """dh, x, w13, preact.  exact: every d a multiple of 1/2 with few bits, some
    of them zero; else 24 bits that the three values share out, in both signs."""
    g = torch.Generator().manual_seed(seed)
    if exact:
        ints = lambda shape, lo=-3: torch.randint(lo, 4, shape, generator=g).float()  # noqa: E731
        gate = torch.where(torch.rand((M, N // 2), generator=g) > 0.5, 64.0, 0.0)
        return ints((M, N // 2)), ints((M, K)), ints((N, K)), torch.cat((gate, ints((M, N // 2))), 1)
    n = lambda shape, std=1.0: torch.randn(shape, generator=g) * std  # noqa: E731
    return n((M, N // 2), 0.1), n((M, K)), n((N, K), K ** -0.5), n((M, N), 1.5)


def spoil(t, seed):
    """Infinities of both signs, two of them in one column, and a NaN."""
    rows, cols = t.shape
    g = torch.Generator().manual_seed(seed)
    at = lambda: (int(torch.randint(0, rows, (1,), generator=g)), int(torch.randint(0, cols // 2, (1,), generator=g)))  # noqa: E731
    for v in (INF, -INF):
        i, j = at()
        t[i, j] = v
    t[0, cols - 1], t[rows - 1, cols - 1] = INF, -INF
    t[rows // 2, cols - 2], t[rows // 3, cols - 3] = INF, NAN
    return t


# ends inside tiles and stages, one tile and many, one share of a sum and several
# (dx in 128 x 256, 64 x 256 and 64 x 128 tiles, dw13 in 128 x 256)
SHAPES = [(1, 16, 8), (1, 480, 4112), (33, 144, 64), (40, 512, 640), (66, 2544, 4112), (129, 272, 200),
          (240, 16, 8), (969, 16, 8), (8406, 16, 160), (8497, 16, 264)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("exact", [True, False])
def test_infinities_of_the_weights_and_of_the_rows(shape, exact):
    M, N, K = shape
    dh, x, w, pre = inputs(1, M, N, K, exact)
    x, w = spoil(x.bfloat16(), 2), spoil(w.bfloat16(), 3)
    f64 = lambda t: t.double().numpy()  # noqa: E731
    d = oracle.silu_mul_bwd(f64(pre), f64(dh))
    dx, dw = moe.gate_up_bwd(dh.to(DEV), x.to(DEV), w.to(DEV), pre.to(DEV))
    same(dx, product(d, f64(w)), exact)
    same(dw, product(d.T, f64(x)), exact)
    # mixed types: the same f32 bits beside a bf16 result
    assert torch.equal(moe.gate_up_bwd(dh.to(DEV), x.to(DEV), w.to(DEV), pre.to(DEV), dx_dtype=B)[1].nan_to_num(7.0),
                       dw.nan_to_num(7.0))


@pytest.mark.parametrize("shape", [(40, 512, 640), (300, 272, 1416)])
def test_infinities_of_both_factors(shape):
    """d of an infinite row of dh, and an infinity of the other factor behind it."""
    M, N, K = shape
    dh, x, w, pre = inputs(4, M, N, K, True)
    pre[:, N // 2:][pre[:, N // 2:] == 0] = 1.0
    dh[5, 3], dh[M - 1, N // 2 - 1] = INF, -INF
    x[5, 2] = x[M - 1, K - 1] = -INF
    w[3, 2] = w[N // 2 - 1, K - 1] = w[3, 9] = INF
    f64 = lambda t: t.double().numpy()  # noqa: E731
    with np.errstate(invalid="ignore"):
        g, u = f64(pre)[:, :N // 2], f64(pre)[:, N // 2:]
        on = g > 0
        d = np.concatenate((np.where(on, f64(dh) * u, f64(dh) * u / 2), f64(dh) * np.where(on, 64.0, 0.0)), axis=1)
        want_x = np.stack([(d * f64(w)[:, j]).sum(axis=1) for j in range(K)], axis=1)
        want_w = np.stack([(d.T * f64(x)[:, j]).sum(axis=1) for j in range(K)], axis=1)
    dx, dw = moe.gate_up_bwd(dh.to(DEV), x.bfloat16().to(DEV), w.bfloat16().to(DEV), pre.to(DEV))
    same(dx, want_x, True)
    same(dw, want_w, True)


def test_captured_and_replayed():
    """The second walk depends on the data alone: one graph, finite inputs and
    others in turn."""
    M, N, K = 66, 2544, 1160
    dh, x, w, pre = (t.to(DEV) for t in inputs(5, M, N, K, True))
    x, w = x.bfloat16(), w.bfloat16()
    bad_x, bad_w = spoil(x.cpu().clone(), 6).to(DEV), spoil(w.cpu().clone(), 7).to(DEV)
    good_x, good_w = x.clone(), w.clone()
    ws = torch.empty(moe.gate_up_bwd_workspace_bytes(M, N, K), dtype=torch.uint8, device=DEV)
    dx, dw = torch.empty((M, K), device=DEV), torch.empty((N, K), device=DEV)
    step = lambda: moe.gate_up_bwd(dh, x, w, pre, dx=dx, dw13=dw, ws=ws)  # noqa: E731
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(6):
        x.copy_(bad_x if i & 1 else good_x)
        w.copy_(bad_w if i & 1 else good_w)
        dx.fill_(7)
        dw.fill_(7)
        graph.replay()
        got = dx.clone(), dw.clone()
        torch.cuda.synchronize()
        want = moe.gate_up_bwd(dh, x, w, pre)
        assert bool(got[0].isnan().any()) == bool(i & 1)
        for a, b in zip(got, want):
            assert torch.equal(a.isnan(), b.isnan()) and torch.equal(a.nan_to_num(7.0), b.nan_to_num(7.0))
