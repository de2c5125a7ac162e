"""moe_gate_up and moe_gate_up_bwd against the float64 oracle.

Exact cases: small integers make every sum exact in f32 whatever the order, so
kept sums and f32 gradients must equal the oracle's bit for bit (the gradients
with gate values 0 and 64, where the sigmoid is 1/2 and 1).

Others: f32 results to the suite's max|delta| / max|ref| <= 1e-5.  A bf16 h or
sum is rounded once: half a step, 2^-8 of the value, beside that.  A bf16
gradient is rounded once, and so is each d it sums: 2^-8 |ref| + 2^-8 sum |d||w|
at most (the second part times 1 + 2^-8 for both), and over all values the
2-norm of the difference stays below 2^-8 of the result's (two independent
roundings, each at most 2^-8 / sqrt(3) in the mean square).
"""

import numpy as np
import pytest
import torch

import moe_grouped_gemm_route_amd as moe
import oracle
from tests.gpu_util import DEV, REL_TOL

pytestmark = pytest.mark.gpu

F, B = moe.F32, moe.BF16
DT = {F: torch.float32, B: torch.bfloat16}


def f64(t):
    return t.double().cpu().numpy()


def ints(seed, shape, lo=-3, hi=4):
    return torch.randint(lo, hi, shape, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16).to(DEV)


def normal(seed, shape, std=1.0, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * std).to(dtype).to(DEV)


def near(got, want, out):
    slack = REL_TOL * np.max(np.abs(want))
    half = 2.0 ** -8 * np.abs(want) if out == B else 0.0
    assert np.all(np.abs(f64(got) - want) <= half + slack)


# M, N, K: one row, few rows (streamed), rows and columns that end inside every
# tile, depths of one segment, inside a stage, odd stages
SHAPES = [(1, 16, 8), (1, 32, 64), (2, 48, 136), (15, 64, 520), (16, 80, 72), (17, 96, 128), (32, 16, 1000),
          (33, 16, 8), (33, 144, 64), (64, 128, 192), (65, 272, 72), (100, 160, 584), (127, 400, 264),
          (129, 64, 128), (200, 1008, 80), (257, 272, 200), (300, 96, 456)]


@pytest.mark.parametrize("shape", SHAPES)
def test_sums_exact(shape):
    M, N, K = shape
    x, w = ints(1, (M, K)), ints(2, (N, K))
    h, y = moe.gate_up(x, w, preact_dtype=F)
    _, want = oracle.gate_up(f64(x), f64(w))
    assert np.array_equal(f64(y), want)
    assert tuple(h.shape) == (M, N // 2)
    assert torch.equal(h, moe.gate_up(x, w))                      # with and without the sums
    w = (w.float() / 64).to(torch.bfloat16)
    hw, _ = oracle.gate_up(f64(x), f64(w))
    near(moe.gate_up(x, w), hw, F)


# every tile of the forward kernel with ragged edges
@pytest.mark.parametrize("shape", [(2050, 4112, 72), (4000, 4096, 136), (1000, 2064, 328), (513, 4096, 64)])
def test_large_tiles_exact(shape):
    M, N, K = shape
    x, w = ints(3, (M, K)), ints(4, (N, K))
    h, y = moe.gate_up(x, w, out_dtype=B, preact_dtype=B)
    want = x.float() @ w.float().t()                              # integers below 2^24: exact
    assert torch.equal(y, want.to(torch.bfloat16))
    h2, y2 = moe.gate_up(x, w, preact_dtype=F)
    assert torch.equal(y2, want)
    g, u = want.double().chunk(2, dim=1)
    hw = g / (1 + (-g).exp()) * u
    assert float((h2.double() - hw).abs().max()) <= REL_TOL * float(hw.abs().max())
    assert bool(((h.double() - hw).abs() <= 2.0 ** -8 * hw.abs() + REL_TOL * float(hw.abs().max())).all())


@pytest.mark.parametrize("out", [F, B])
@pytest.mark.parametrize("keep", [None, F, B])
@pytest.mark.parametrize("shape", [(1, 512, 1024), (24, 256, 512), (70, 320, 1416), (300, 272, 640)])
def test_forward_random(shape, keep, out):
    M, N, K = shape
    x, w = normal(5, (M, K)), normal(6, (N, K), K ** -0.5)
    r = moe.gate_up(x, w, out_dtype=out, preact_dtype=keep)
    hw, yw = oracle.gate_up(f64(x), f64(w))
    near(r if keep is None else r[0], hw, out)
    if keep is not None:
        assert r[1].dtype == DT[keep]
        near(r[1], yw, keep)


def exact_back(seed, M, N, K, keep, grad):
    """Inputs whose d are multiples of 1/2 with few bits."""
    g = torch.where(ints(seed, (M, N // 2), 0, 2) > 0, 64.0, 0.0)
    pre = torch.cat((g, ints(seed + 1, (M, N // 2)).float()), 1).to(DT[keep])
    return ints(seed + 2, (M, N // 2)).to(DT[grad]), ints(seed + 3, (M, K)), ints(seed + 4, (N, K)), pre


@pytest.mark.parametrize("shape", SHAPES + [(513, 272, 520), (40, 2064, 136), (700, 16, 8)])
@pytest.mark.parametrize("types", [(F, F), (B, B)])
def test_gradients_exact(shape, types):
    M, N, K = shape
    dh, x, w, pre = exact_back(11, M, N, K, *types)
    dx, dw = moe.gate_up_bwd(dh, x, w, pre)
    dxw, dww, _ = oracle.gate_up_bwd(f64(dh), f64(x), f64(w), f64(pre))
    assert np.array_equal(f64(dx), dxw) and np.array_equal(f64(dw), dww)
    # bf16 results are the same sums rounded once; one without the other the same bits
    bx, bw = moe.gate_up_bwd(dh, x, w, pre, dx_dtype=B, dw_dtype=B)
    assert torch.equal(bx, dx.to(torch.bfloat16)) and torch.equal(bw, dw.to(torch.bfloat16))
    only, none = moe.gate_up_bwd(dh, x, w, pre, dx_dtype=B, dw_dtype=None)
    assert none is None and torch.equal(only, bx)
    none, only = moe.gate_up_bwd(dh, x, w, pre, dx_dtype=None, dw_dtype=B)
    assert none is None and torch.equal(only, bw)
    mx, mw = moe.gate_up_bwd(dh, x, w, pre, dx_dtype=B, dw_dtype=F)
    assert torch.equal(mx, bx) and torch.equal(mw, dw)


@pytest.mark.parametrize("shape", [(2050, 4112, 264), (4000, 528, 4104), (300, 4096, 4096)])
def test_large_gradients_exact(shape):
    M, N, K = shape
    dh, x, w, pre = exact_back(21, M, N, K, B, B)
    dx, dw = moe.gate_up_bwd(dh, x, w, pre)
    g, u, e = pre[:, :N // 2].float(), pre[:, N // 2:].float(), dh.float()
    on = g > 0
    d = torch.cat((torch.where(on, e * u, e * u / 2), torch.where(on, e * 64, 0.0)), 1)
    assert torch.equal(dx, d @ w.float()) and torch.equal(dw, d.t() @ x.float())
    bx, bw = moe.gate_up_bwd(dh, x, w, pre, dx_dtype=B, dw_dtype=B)
    assert torch.equal(bx, dx.to(torch.bfloat16)) and torch.equal(bw, dw.to(torch.bfloat16))


@pytest.mark.parametrize("shape", [(1, 256, 512), (64, 512, 320), (300, 272, 1416), (1237, 528, 136)])
@pytest.mark.parametrize("keep,grad", [(F, F), (B, F), (F, B), (B, B)])
def test_gradients_random(shape, keep, grad):
    M, N, K = shape
    x, w = normal(31, (M, K)), normal(32, (N, K), K ** -0.5)
    pre = normal(33, (M, N), 1.5, DT[keep])
    dh = normal(34, (M, N // 2), 0.1, DT[grad])
    dxw, dww, d = oracle.gate_up_bwd(f64(dh), f64(x), f64(w), f64(pre))
    dx, dw = moe.gate_up_bwd(dh, x, w, pre)
    near(dx, dxw, F)
    near(dw, dww, F)
    bx, bw = moe.gate_up_bwd(dh, x, w, pre, dx_dtype=B, dw_dtype=B)
    for got, want, size in ((bx, dxw, np.abs(d) @ np.abs(f64(w))), (bw, dww, np.abs(d).T @ np.abs(f64(x)))):
        diff = np.abs(f64(got) - want)
        assert np.all(diff <= 2.0 ** -8 * (np.abs(want) + size * (1 + 2.0 ** -8)) + REL_TOL * np.max(np.abs(want)))
        if M > 1:
            assert np.linalg.norm(diff) <= 2.0 ** -8 * np.linalg.norm(want)


def test_gradient_against_differences():
    """Entries against central differences of sum(v * h) in f64.  With a step of
    1e-4 the differences are off by step^2 / 6 of a third derivative (|v| |w|^3
    and its like, under 1e2 here: 2e-7) and by 2^-52 of the loss over the step
    (under 1e-9): 1e-5 of the largest gradient covers both."""
    M, N, K = 40, 96, 64
    x, w = normal(41, (M, K)), normal(42, (N, K), K ** -0.5)
    v = normal(43, (M, N // 2), 1.0, torch.float32)
    _, pre = moe.gate_up(x, w, preact_dtype=F)
    dx, dw = moe.gate_up_bwd(v, x, w, pre)
    v64, x64, w64 = f64(v), f64(x), f64(w)
    for which, grad in (("x", dx), ("w", dw)):
        grad = f64(grad)
        for i, j in ((0, 0), (grad.shape[0] - 1, K - 1), (grad.shape[0] // 2, 7), (3, 31)):
            ends = []
            for step in (-1e-4, 1e-4):
                a, b = x64.copy(), w64.copy()
                (a if which == "x" else b)[i, j] += step
                ends.append(float((v64 * oracle.gate_up(a, b)[0]).sum()))
            assert abs((ends[1] - ends[0]) / 2e-4 - grad[i, j]) <= 2 * REL_TOL * np.max(np.abs(grad))


def test_values_that_are_not_finite_stay_in_their_rows():
    M, N, K = 70, 96, 136
    x, w = ints(51, (M, K)), ints(52, (N, K))
    clean = moe.gate_up(x, w, preact_dtype=F)[1]
    bad = x.clone()
    bad[3, 5], bad[69, 135] = float("inf"), float("nan")
    y = moe.gate_up(bad, w, preact_dtype=F)[1]
    keep = torch.ones(M, dtype=torch.bool)
    keep[[3, 69]] = False
    assert torch.equal(y.cpu()[keep], clean.cpu()[keep]) and bool(y[69].isnan().all())
    # a depth that ends inside a stage: what lies behind the row does not enter
    far = torch.full((2 * M, K), float("nan"), dtype=torch.bfloat16, device=DEV)
    far[:M] = x
    assert torch.equal(moe.gate_up(far[:M], w, preact_dtype=F)[1], clean)


@pytest.mark.parametrize("M", [1, 40])
def test_extreme_gates(M):
    """Gates where e^-g overflows or vanishes: no NaN, the limits of the formulas."""
    N, K = 64, 32
    g = torch.tensor([-200.0, -100.0, -88.0, 88.0, 200.0, 0.0, -0.0, 1e4]).repeat(M, N // 16).to(DEV)
    pre = torch.cat((g, torch.ones_like(g)), 1).contiguous()
    dh = torch.ones((M, N // 2), device=DEV)
    x, w = ints(61, (M, K)), ints(62, (N, K))
    dx, dw = moe.gate_up_bwd(dh, x, w, pre)
    dxw, dww, _ = oracle.gate_up_bwd(f64(dh), f64(x), f64(w), f64(pre))
    near(dx, dxw, F)
    near(dw, dww, F)


def test_rows_behind_and_given_outputs():
    M, N, K = 50, 80, 72
    dh, x, w, pre = exact_back(71, M, N, K, F, B)
    want = moe.gate_up_bwd(dh, x, w, pre)
    big_x = torch.full((M + 3, K), 9.0, device=DEV)
    big_w = torch.full((N + 3, K), 9.0, device=DEV)
    ws = torch.empty(moe.gate_up_bwd_workspace_bytes(M, N, K) + 512, dtype=torch.uint8, device=DEV)
    dx, dw = moe.gate_up_bwd(dh, x, w, pre, dx=big_x[:M], dw13=big_w[:N], ws=ws)
    assert torch.equal(dx, want[0]) and torch.equal(dw, want[1])
    assert bool((big_x[M:] == 9).all()) and bool((big_w[N:] == 9).all())
    big_h = torch.full((M + 3, N // 2), 9.0, device=DEV)
    big_p = torch.full((M + 3, N), 9.0, device=DEV)
    h, y = moe.gate_up(x, w, out=big_h[:M], preact=big_p[:M])
    hw, yw = moe.gate_up(x, w, preact_dtype=F)
    assert torch.equal(h, hw) and torch.equal(y, yw)
    assert bool((big_h[M:] == 9).all()) and bool((big_p[M:] == 9).all())
