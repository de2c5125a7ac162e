"""GPU parity of the router, the permutation's gradients, the unfused
activation and the product's input gradient against the float64 oracle.

Tolerances count roundings.  EPS = 2^-24 is half a step of f32, H[dt] half a
step of the output type; a sum of n f32 terms is off by at most n EPS times the
sum of the magnitudes, a product of bf16 values is exact in f32.  expf and the
hardware exponential are within 2 ulp of the exponential of their argument, and
an argument a is formed within 2 EPS |a|, so an exponential is off by at most
EPS (2 |a| + 4) relative."""

import itertools

import numpy as np
import pytest
import torch

import moe_grouped_gemm_route_amd as moe
import oracle
from moe_grouped_gemm_route_amd.synth import f32_to_bf16_bits, make_problem
from tests.gpu_util import DEV, bf16_bits_to_f64, to_dev

pytestmark = pytest.mark.gpu

EPS = 2.0 ** -24
H = {torch.float32: EPS, torch.bfloat16: 2.0 ** -8}
ENUM = {torch.float32: moe.F32, torch.bfloat16: moe.BF16}
BOTH = [torch.float32, torch.bfloat16]


def f64(t):
    return t.double().cpu().numpy()


def dev(a, dtype):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV).to(dtype)


def close(got, ref, bound, dtype):
    """|got - ref| <= bound (computed in f32 or better), then one rounding to
    dtype (2^-126 covers flushed and subnormal results)."""
    got, ref = np.asarray(got), np.asarray(ref)
    tol = bound + H[dtype] * (np.abs(ref) + bound) + 2.0 ** -126
    worst = np.max(np.abs(got - ref) - tol)
    assert np.isfinite(got).all() and worst <= 0, "off by %g over the bound" % worst


# ----------------------------------------------------------- the router ---

def gate_bound(x, ids, w):
    """Rounding of a weight: two exponentials whose arguments are differences
    of the row's finite logits, a sum of up to 1024 of them in 16 + 6 steps, a
    division, the scale."""
    fin = np.where(np.isfinite(x), x, 0.0)
    spread = np.abs(fin).max(axis=1, keepdims=True) * 2
    return np.abs(w) * EPS * (2 * (2 * spread + 4) + 26)


GATES = [(1, 1, 1), (1, 256, 6), (3, 7, 7), (64, 256, 6), (5, 64, 64), (33, 65, 8), (17, 128, 3), (9, 500, 16),
         (6, 1000, 10), (4, 1024, 64), (257, 96, 2)]


@pytest.mark.parametrize("T,E,k", GATES)
@pytest.mark.parametrize("dtype", BOTH)
def test_gate_matches_oracle(T, E, k, dtype):
    rng = np.random.default_rng(1000 * T + E + k)
    x = dev(rng.standard_normal((T, E)) * 2, dtype)
    b = dev(rng.standard_normal(E) * 0.2, torch.float32)
    for score, renorm, bias in itertools.product(["softmax", "sigmoid"], [True, False], [None, b]):
        code = moe.GATE_SOFTMAX if score == "softmax" else moe.GATE_SIGMOID
        ids, w = moe.topk_gate(x, k, score=code, bias=bias, renormalize=renorm, scale=2.5)
        rid, rw = oracle.topk_gate(f64(x), k, score, None if bias is None else f64(bias), renorm, 2.5)
        assert np.array_equal(ids.cpu().numpy(), rid), (score, renorm, bias is None)
        close(f64(w), rw, gate_bound(f64(x), rid, rw), torch.float32)


def edge_logits():
    inf, nan = np.inf, np.nan
    rows = np.zeros((10, 70))
    rows[1] = -inf
    rows[2] = nan
    rows[3, 5:] = -inf                            # five experts left
    rows[4, ::2] = nan
    rows[5, [3, 69]] = inf                        # two at +inf
    rows[6] = -3.0e38
    rows[7] = -np.arange(70) * 1000.0             # scores underflow
    rows[8] = -1.0e4 + np.arange(70)
    rows[9] = np.finfo(np.float32).min
    return rows


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_gate_masked_infinite_and_tied_logits(score, renorm):
    x = torch.from_numpy(edge_logits()).float().to(DEV)
    code = moe.GATE_SOFTMAX if score == "softmax" else moe.GATE_SIGMOID
    ids, w = moe.topk_gate(x, 8, score=code, renormalize=renorm)
    rid, rw = oracle.topk_gate(f64(x), 8, score, None, renorm)
    assert np.array_equal(ids.cpu().numpy(), rid)
    # arguments of magnitude up to 2 * 7e4 matter (larger ones give 0 exactly)
    close(f64(w), rw, EPS * (2 * (2 * 2 * 7.0e4 + 4) + 26) * rw, torch.float32)
    # with a bias: masked experts stay unchosen, a NaN bias masks its expert
    b = torch.linspace(0.5, -0.5, 70, device=DEV)
    b[2] = float("nan")
    ids, _ = moe.topk_gate(x, 8, score=code, bias=b, renormalize=renorm)
    rid, _ = oracle.topk_gate(f64(x), 8, score, f64(b), renorm)
    assert np.array_equal(ids.cpu().numpy(), rid)
    # the dropped slots go through the sort as dropped pairs
    r = moe.route_sort(ids, 70)
    assert int(r["err_count"]) == int((rid < 0).sum())
    assert np.array_equal(r["pair_row"].cpu().numpy() < 0, rid.reshape(-1) < 0)


@pytest.mark.parametrize("T,E,k", GATES)
@pytest.mark.parametrize("dtype", BOTH)
def test_gate_gradient_matches_oracle(T, E, k, dtype):
    rng = np.random.default_rng(7 * T + E + k)
    x = dev(rng.standard_normal((T, E)) * 2, dtype)
    for score, renorm in itertools.product(["softmax", "sigmoid"], [True, False]):
        code = moe.GATE_SOFTMAX if score == "softmax" else moe.GATE_SIGMOID
        ids, _ = moe.topk_gate(x, k, score=code)
        if T > 2:
            ids[1, 0] = -1                         # a dropped slot
            ids[2, k - 1] = E + 3                  # an id out of range
            ids[0, k - 1] = ids[0, 0]              # (where k > 1) the same expert twice
        g = torch.randn(ids.shape, device=DEV, generator=torch.Generator(DEV).manual_seed(T + E))
        got = moe.topk_gate_bwd(x, ids, g, score=code, renormalize=renorm, scale=1.5)
        assert got.dtype == dtype
        ref = oracle.topk_gate_bwd(f64(x), ids.cpu().numpy(), f64(g), score, renorm, 1.5)
        # every term is at most (1 + k) weights' worth of 1.5 |g|, each off as
        # a weight is; the mean sums k terms; a repeated id adds its terms
        spread = 2 * np.abs(f64(x)).max(axis=1, keepdims=True)
        size = 1.5 * np.abs(f64(g)).max(axis=1, keepdims=True) * (1 + min(k, 2))
        close(f64(got), ref, EPS * (4 * (2 * spread + 4) + 32 + 2 * k) * size, dtype)


def test_gate_gradient_of_masked_rows_is_zero_or_finite():
    x = torch.from_numpy(edge_logits()).float().to(DEV)
    for code, renorm in itertools.product([moe.GATE_SOFTMAX, moe.GATE_SIGMOID], [True, False]):
        ids, _ = moe.topk_gate(x, 8, score=code)
        g = torch.ones((10, 8), device=DEV)
        g[ids < 0] = float("nan")                  # never looked at
        d = moe.topk_gate_bwd(x, ids, g, score=code, renormalize=renorm)
        assert bool(torch.isfinite(d).all())
        assert not bool(d[1:3].any())
        # a masked expert gets no gradient even where an id names it
        ids[3] = torch.arange(60, 68, device=DEV, dtype=torch.int32)
        d = moe.topk_gate_bwd(x, ids, torch.full_like(g, 3.0), score=code, renormalize=renorm)
        assert not bool(d[3].any())


# (the differences of this test are of the oracle's float64 weights;
# test_gpu_gate_difference takes those of the weights that the GPU returns)
def test_gate_gradient_is_the_difference():
    # differences of the GPU's own weights (f32: a step of 2^-5 keeps their
    # rounding, 2^-20, and the third-order term, h^2/6 times a third derivative
    # of at most 1, under 4e-4)
    T, E, k, h = 8, 12, 3, 2.0 ** -5
    x = torch.randn((T, E), device=DEV, generator=torch.Generator(DEV).manual_seed(5))
    g = torch.rand((T, k), device=DEV) - 0.5
    for code, renorm in itertools.product([moe.GATE_SOFTMAX, moe.GATE_SIGMOID], [True, False]):
        ids, _ = moe.topk_gate(x, k, score=code, renormalize=renorm)
        d = f64(moe.topk_gate_bwd(x, ids, g, score=code, renormalize=renorm))
        name = "softmax" if code == moe.GATE_SOFTMAX else "sigmoid"
        for e in range(E):
            vals = []
            for s in (h, -h):
                xe = x.clone()
                xe[:, e] += s
                vals.append((oracle.slot_weights(f64(xe), ids.cpu().numpy(), name, renorm) * f64(g)).sum(axis=1))
            assert np.abs((vals[0] - vals[1]) / (2 * h) - d[:, e]).max() < 4e-4


# ------------------------------------------------------ the permutation ---

PERMS = [(1, 1, 1, 4), (1, 6, 8, 64), (5, 3, 4, 12), (64, 6, 256, 512), (37, 2, 5, 520), (3, 64, 70, 1028),
         (130, 8, 16, 2560), (300, 7, 9, 100)]


def routed(T, k, E, drop=0.0, seed=0):
    rng = np.random.default_rng(seed + 31 * T + k)
    ids = rng.integers(0, E, size=(T, k), dtype=np.int32)
    ids[rng.random((T, k)) < drop] = -1
    return moe.route_sort(to_dev(ids), E), oracle.route_sort(ids, E)


@pytest.mark.parametrize("T,k,E,N", PERMS)
@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("drop", [0.0, 0.2])
def test_dispatch_and_its_gradient(T, k, E, N, dtype, drop):
    r, rr = routed(T, k, E, drop)
    M = T * k
    gen = torch.Generator(DEV).manual_seed(N)
    x = torch.randn((T, N), device=DEV, generator=gen).to(dtype)
    out = torch.full((M + 3, N), 7.0, device=DEV, dtype=dtype)
    xs = moe.moe_dispatch(x, r["pair_row"], k, out=out)
    ref = oracle.dispatch(f64(x), rr["pair_row"], M + 3, fill=7.0)
    assert np.array_equal(f64(xs), ref)                    # a copy: exact, other rows untouched
    if drop == 0.0:
        assert torch.equal(moe.moe_dispatch(x, r["pair_row"], k), xs[:M])
    for odt in BOTH:
        dxs = torch.randn((M, N), device=DEV, generator=gen).to(dtype)
        dx = moe.moe_dispatch_bwd(dxs, r["pair_row"], k, out_dtype=ENUM[odt])
        a = oracle.dispatch_bwd(np.abs(f64(dxs)), rr["pair_row"], k)
        close(f64(dx), oracle.dispatch_bwd(f64(dxs), rr["pair_row"], k), k * EPS * a, odt)


@pytest.mark.parametrize("T,k,E,N", PERMS)
@pytest.mark.parametrize("drop", [0.0, 0.2])
@pytest.mark.parametrize("types", list(itertools.product(BOTH, BOTH, BOTH)))
def test_combine_gradient(T, k, E, N, drop, types):
    gdt, ydt, odt = types
    r, rr = routed(T, k, E, drop, seed=3)
    M = T * k
    gen = torch.Generator(DEV).manual_seed(N + 1)
    dout = torch.randn((T, N), device=DEV, generator=gen).to(gdt)
    y = torch.randn((M, N), device=DEV, generator=gen).to(ydt)
    y[int(r["group_offsets"][-1]):] = float("nan")          # rows behind the last band are not read
    w = torch.rand((T, k), device=DEV, generator=gen)
    out = torch.full((M, N), 5.0, device=DEV, dtype=odt)
    dy, dw = moe.moe_combine_bwd(dout, y, w, r["pair_row"], out_dtype=ENUM[odt], out=out)
    yz = np.nan_to_num(f64(y))
    rdy, rdw = oracle.combine_bwd(f64(dout), yz, f64(w), rr["pair_row"], fill=5.0)
    close(f64(dy), rdy, EPS * np.abs(rdy), odt)
    off = int(rr["group_offsets"][-1])
    assert bool((dy[off:] == 5.0).all())                    # and not written
    _, size = oracle.combine_bwd(np.abs(f64(dout)), np.abs(yz), f64(w), rr["pair_row"])
    close(f64(dw), rdw, N * EPS * size, torch.float32)


def test_permutation_ignores_rows_out_of_range():
    # entries past the last row are dropped pairs, like negative ones
    x = torch.randn((2, 8), device=DEV)
    pr = torch.tensor([1, 4, -5, 1 << 30], dtype=torch.int32, device=DEV)
    out = torch.zeros((4, 8), device=DEV)
    moe.moe_dispatch(x, pr, 2, out=out)
    assert torch.equal(out[1], x[0]) and not bool(out[[0, 2, 3]].any())
    dx = moe.moe_dispatch_bwd(out, pr, 2)
    assert torch.equal(dx[0], x[0]) and not bool(dx[1].any())
    w = torch.ones((2, 2), device=DEV)
    dy, dw = moe.moe_combine_bwd(x, out, w, pr, out=torch.zeros((4, 8), device=DEV))
    assert torch.equal(dy[1], x[0]) and not bool(dy[[0, 2, 3]].any())
    assert not bool(dw.reshape(-1)[1:].any()) and float(dw[0, 0]) > 0


# -------------------------------------------------------- the activation ---

def silu_rel(g):
    """Relative rounding of s = 1 / (1 + e^-g): the exponential's, an add and
    a division."""
    return EPS * (2 * np.abs(g) + 4 + 3)


@pytest.mark.parametrize("M,N", [(1, 8), (3, 16), (5, 1416), (64, 4096), (257, 1032), (1000, 24)])
@pytest.mark.parametrize("types", list(itertools.product(BOTH, BOTH)))
def test_silu_mul(M, N, types):
    idt, odt = types
    y = (torch.randn((M, N), device=DEV, generator=torch.Generator(DEV).manual_seed(M)) * 4).to(idt)
    h = moe.silu_mul(y, out_dtype=ENUM[odt])
    ref = oracle.silu_mul(f64(y))
    g = f64(y)[:, : N // 2]
    close(f64(h), ref, np.abs(ref) * (silu_rel(g) + 2 * EPS), odt)
    # with band offsets only the bands' rows are read and written
    live = M // 2
    off = torch.tensor([0, live // 2, live], dtype=torch.int32, device=DEV)
    out = torch.full((M, N // 2), 3.0, device=DEV, dtype=odt)
    moe.silu_mul(y, group_offsets=off, out_dtype=ENUM[odt], out=out)
    assert torch.equal(out[:live], h[:live]) and bool((out[live:] == 3.0).all())


def test_silu_mul_extremes():
    g = torch.tensor([[0.0, -0.0, 200.0, -200.0, float("nan"), float("inf"), 1e-30, -88.0]], device=DEV)
    y = torch.cat((g, torch.full_like(g, 2.0)), 1)
    h = moe.silu_mul(y)[0].tolist()
    assert h[0] == 0 and h[1] == 0 and h[2] == 400.0 and h[3] == 0 and np.isnan(h[4]) and h[5] == np.inf
    assert abs(h[6] - 1e-30) < 1e-36


# ------------------------------------------------ the product's gradient ---

def bands(counts, extra=0):
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    return off, int(off[-1]) + extra


def make_weights(E, N, K, fmt, seed):
    """Canonical weights and the pack.  fmt: mxfp4, nvfp4 (general scales,
    negative and subnormal ones among them), nvfp4_pow2, nvfp4_mixed (one
    expert general)."""
    rng = np.random.default_rng(seed)
    codes = rng.integers(0, 256, size=(E, N, K // 2), dtype=np.uint8)
    if fmt == "mxfp4":
        s = rng.integers(110, 140, size=(E, N, K // 32)).astype(np.uint8)
        return {"fmt": "mxfp4", "codes": codes, "scales": s}, moe.mxfp4_encode(to_dev(codes), to_dev(s))
    s = rng.integers(0, 15, size=(E, N, K // 16)).astype(np.uint8) << 3
    s[s == 0] = 8
    if fmt != "nvfp4_pow2":
        general = rng.integers(0, 256, size=s.shape).astype(np.uint8)
        general[(general & 0x7F) == 0x7F] = 0x01
        if fmt == "nvfp4":
            s = general
        else:
            s[E // 2] = general[E // 2]
    ts = rng.uniform(0.01, 2.0, size=E).astype(np.float32)
    w = {"fmt": "nvfp4", "codes": codes, "block_scales": s, "tensor_scale": ts}
    return w, moe.mxfp4_encode(to_dev(codes), to_dev(s), to_dev(ts), moe.NVFP4)


def random_dy(M, N, seed):
    rng = np.random.default_rng(seed)
    return f32_to_bf16_bits(rng.standard_normal((M, N), dtype=np.float32))


def dgrad_bound(dy, off, w, N):
    """N products exact in f32, their f32 sum (the matrix unit's own order),
    and the NVFP4 tensor scale's product: (N + 2) EPS of the magnitudes, twice
    that for a unit that truncates."""
    return 2 * (N + 2) * EPS * oracle.gmm_dgrad(dy, off, w, absolute=True)


FMTS = ["mxfp4", "nvfp4", "nvfp4_pow2", "nvfp4_mixed"]
DGRADS = [
    ([1], 64, 128), ([1, 0, 2], 64, 128), ([5, 0, 17], 192, 384), ([16, 15, 33, 0, 1], 64, 256),
    ([127, 128, 129, 0, 3], 128, 256), ([0, 0, 260], 320, 640), ([3] * 40, 64, 128),
]


@pytest.mark.parametrize("counts,N,K", DGRADS)
@pytest.mark.parametrize("fmt", FMTS)
def test_dgrad_full_oracle(counts, N, K, fmt):
    E = len(counts)
    fe = 2 if E > 2 else 0
    off, M = bands(counts, extra=2)
    w, packed = make_weights(E, N, K, fmt, seed=N + K + E + fe)
    bits = random_dy(M, N, seed=M)
    dy64 = bf16_bits_to_f64(bits)
    ref, tol = oracle.gmm_dgrad(dy64, off, w), dgrad_bound(dy64, off, w, N)
    live = off[-1]
    enum = moe.MXFP4 if fmt == "mxfp4" else moe.NVFP4
    for odt in BOTH:
        out = torch.full((M, K), 9.0, device=DEV, dtype=odt)
        got = moe.moe_gmm_dgrad(packed, enum, E, N, K, to_dev(bits), to_dev(off), M, out_dtype=ENUM[odt], out=out)
        close(f64(got)[:live], ref[:live], tol[:live], odt)
        assert bool((out[live:] == 9.0).all())             # rows of no band left as they were


def act_bound(dh_tol, dh, pre):
    """Rounding of dg = dh u f(g), f = s (1 + g (1 - s)), and du = dh g s: the
    rounding of dh, and of f: s moves s by silu_rel, and f by at most
    s (1 + 2 |g|) times that, plus four products and sums of size s (1 + |g|)."""
    K = dh.shape[1]
    g, u = pre[:, :K], pre[:, K:]
    s = 1 / (1 + np.exp(-g))
    f = np.abs(s * (1 + g * (1 - s)))
    df = s * (1 + 2 * np.abs(g)) * silu_rel(g) + 6 * EPS * s * (1 + np.abs(g))
    dg = np.abs(u) * (dh_tol * (f + df) + np.abs(dh) * df) + 4 * EPS * np.abs(dh * u) * (f + df)
    du = np.abs(g * s) * (dh_tol + (np.abs(dh) + dh_tol) * (silu_rel(g) + 4 * EPS))
    return np.concatenate([dg, du], axis=1)


@pytest.mark.parametrize("counts,N,K", DGRADS)
@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("pdt", BOTH)
def test_dgrad_through_the_activation(counts, N, K, fmt, pdt):
    E = len(counts)
    off, M = bands(counts, extra=1)
    w, packed = make_weights(E, N, K, fmt, seed=N + K)
    bits = random_dy(M, N, seed=M + 5)
    dy64 = bf16_bits_to_f64(bits)
    pre = (torch.randn((M, 2 * K), device=DEV, generator=torch.Generator(DEV).manual_seed(M)) * 2).to(pdt)
    live = int(off[-1])
    dh, tol = oracle.gmm_dgrad(dy64, off, w)[:live], dgrad_bound(dy64, off, w, N)[:live]
    p64 = f64(pre)[:live]
    ref, bound = oracle.silu_mul_bwd(p64, dh), act_bound(tol, dh, p64)
    enum = moe.MXFP4 if fmt == "mxfp4" else moe.NVFP4
    for odt in BOTH:
        out = torch.full((M, 2 * K), 9.0, device=DEV, dtype=odt)
        got = moe.moe_gmm_dgrad(packed, enum, E, N, K, to_dev(bits), to_dev(off), M, out_dtype=ENUM[odt],
                                act=moe.ACT_SILU_MUL, preact=pre, out=out)
        close(f64(got)[:live], ref, bound, odt)
        assert bool((out[live:] == 9.0).all())


@pytest.mark.parametrize("E", [1, 63, 64, 65, 1000, 1024])
def test_dgrad_many_experts(E):
    N, K = 64, 128
    rng = np.random.default_rng(E)
    counts = rng.integers(0, 4, size=E)
    counts[E - 1] = 1
    counts[0] = 140 if E < 100 else 2
    off, M = bands(counts)
    w, packed = make_weights(E, N, K, "mxfp4", seed=E)
    bits = random_dy(M, N, seed=E)
    dy64 = bf16_bits_to_f64(bits)
    got = moe.moe_gmm_dgrad(packed, moe.MXFP4, E, N, K, to_dev(bits), to_dev(off), M)
    close(f64(got), oracle.gmm_dgrad(dy64, off, w), dgrad_bound(dy64, off, w, N), torch.float32)


@pytest.mark.parametrize("rows", [1, 15, 16, 17, 31, 32, 33, 47, 48, 49, 63, 64, 65, 80, 95, 96, 97, 112, 113, 127,
                                  128, 129, 255, 257])
def test_dgrad_every_band_size(rows):
    N, K = 128, 384
    off, M = bands([2, rows, 0, 1])
    w, packed = make_weights(4, N, K, "nvfp4_pow2", seed=rows)
    bits = random_dy(M, N, seed=rows)
    dy64 = bf16_bits_to_f64(bits)
    got = moe.moe_gmm_dgrad(packed, moe.NVFP4, 4, N, K, to_dev(bits), to_dev(off), M)
    close(f64(got), oracle.gmm_dgrad(dy64, off, w), dgrad_bound(dy64, off, w, N), torch.float32)


# grids that take each way of sharing the work: 128- and 256-column
# workgroups, n walked by four, two or one group of waves, and
# 32-, 64- and 128-row tiles; n of one stage, of fewer stages than groups, and
# of a number no group count divides
@pytest.mark.parametrize("E,K,rows", [(6, 896, 2), (40, 1024, 1), (100, 1024, 1), (210, 1024, 1), (30, 896, 7),
                                      (12, 640, 40), (5, 640, 100)])
@pytest.mark.parametrize("N", [64, 192, 1088])
@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4", "nvfp4_pow2"])
def test_dgrad_every_grid(E, K, rows, N, fmt):
    rng = np.random.default_rng(E + K + N)
    counts = np.maximum(0, rows + rng.integers(-rows, rows + 1, size=E))
    counts[0] = 3 * rows + 30
    off, M = bands(counts, extra=1)
    w, packed = make_weights(E, N, K, fmt, seed=E + N)
    bits = random_dy(M, N, seed=K)
    dy64 = bf16_bits_to_f64(bits)
    live = off[-1]
    out = torch.full((M, K), 9.0, device=DEV)
    enum = moe.MXFP4 if fmt == "mxfp4" else moe.NVFP4
    got = moe.moe_gmm_dgrad(packed, enum, E, N, K, to_dev(bits), to_dev(off), M, out=out)
    close(f64(got)[:live], oracle.gmm_dgrad(dy64, off, w)[:live], dgrad_bound(dy64, off, w, N)[:live], torch.float32)
    assert bool((out[live:] == 9.0).all())


def test_dgrad_offsets_never_lead_outside():
    # offsets past M, falling and negative ones: bands are cut to the rows that
    # exist; rows of sound bands come out right and nothing else is touched
    E, N, K, M = 5, 128, 256, 40
    w, packed = make_weights(E, N, K, "mxfp4", seed=4)
    bits = random_dy(M, N, seed=4)
    good = np.array([0, 10, 20, 30, 40, 40], dtype=np.int32)
    ref = oracle.gmm_dgrad(bf16_bits_to_f64(bits), good, w)
    tol = dgrad_bound(bf16_bits_to_f64(bits), good, w, N)
    pool = torch.full((M + 64, K), 7.0, device=DEV)
    for bad in ([0, 10, 20, 30, 1 << 30, 1 << 30], [0, 10, 20, 30, 40, 5], [-50, 10, 20, 30, 40, 40]):
        pool.fill_(7.0)
        out = pool[:M]
        moe.moe_gmm_dgrad(packed, moe.MXFP4, E, N, K, to_dev(bits), to_dev(np.array(bad, dtype=np.int32)), M, out=out)
        close(f64(out), ref, tol, torch.float32)
        assert bool((pool[M:] == 7.0).all())


def test_sizes_past_32_bit_offsets():
    # more than 2^31 elements (4 GiB of bf16): the last rows come out right
    T, k, N = 270000, 2, 4096
    M = T * k
    pr = torch.arange(M - 1, -1, -1, dtype=torch.int32, device=DEV)       # pair p at row M - 1 - p
    x = torch.zeros((T, N), dtype=torch.bfloat16, device=DEV)
    x[0], x[-1] = 1.5, -2.5
    xs = moe.moe_dispatch(x, pr, k)
    assert bool((xs[-2:] == 1.5).all()) and bool((xs[:2] == -2.5).all()) and not bool(xs[2:-2].any())
    dx = moe.moe_dispatch_bwd(xs, pr, k, out_dtype=moe.BF16)
    assert bool((dx[0] == 3.0).all()) and bool((dx[-1] == -5.0).all())
    w = torch.full((T, k), 0.5, device=DEV)
    dy, dw = moe.moe_combine_bwd(x, xs, w, pr, out_dtype=moe.BF16)
    assert bool((dy[-1] == 0.75).all()) and bool((dy[0] == -1.25).all())
    assert dw[0].tolist() == [2.25 * N] * 2 and dw[-1].tolist() == [6.25 * N] * 2
    del dy, dw, dx, xs
    y = torch.zeros((M, N), dtype=torch.bfloat16, device=DEV)
    y[-1, : N // 2], y[-1, N // 2:] = 200.0, 0.25
    h = moe.silu_mul(y, out_dtype=moe.BF16)
    assert bool((h[-1] == 50.0).all()) and not bool(h[:-1].any())
    # the product's gradient, through the activation (dx of 2^31 elements)
    E, n, K = 2, 64, 2048
    _, packed = make_weights(E, n, K, "mxfp4", seed=6)
    off = torch.tensor([0, M - 3, M], dtype=torch.int32, device=DEV)
    dyb = torch.zeros((M, n), dtype=torch.bfloat16, device=DEV)
    dyb[-1] = 1.0
    got = moe.moe_gmm_dgrad(packed, moe.MXFP4, E, n, K, dyb, off, M, out_dtype=moe.BF16, act=moe.ACT_SILU_MUL, preact=y)
    few = moe.moe_gmm_dgrad(packed, moe.MXFP4, E, n, K, dyb[-3:], torch.tensor([0, 0, 3], dtype=torch.int32, device=DEV),
                            3, out_dtype=moe.BF16, act=moe.ACT_SILU_MUL, preact=y[-3:])
    assert torch.equal(got[-1], few[-1]) and bool(got[-1].any()) and not bool(got[:-1].any())


def test_dgrad_no_rows_and_bad_rows_stay_apart():
    E, N, K = 4, 128, 256
    _, packed = make_weights(E, N, K, "mxfp4", seed=1)
    # every pair dropped: nothing is written
    out = torch.full((6, K), 4.0, device=DEV)
    z = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    moe.moe_gmm_dgrad(packed, moe.MXFP4, E, N, K, torch.ones((6, N), device=DEV, dtype=torch.bfloat16), z, 6, out=out)
    assert bool((out == 4.0).all())
    # infinities and NaN of a row (and of rows behind the bands) stay in it
    off, M = bands([20, 0, 30, 10], extra=4)
    dy = torch.randn((M, N), device=DEV).bfloat16()
    ref = moe.moe_gmm_dgrad(packed, moe.MXFP4, E, N, K, dy, to_dev(off), M)
    bad = dy.clone()
    bad[7] = float("nan")
    bad[25] = float("inf")
    bad[60:] = float("nan")
    got = moe.moe_gmm_dgrad(packed, moe.MXFP4, E, N, K, bad, to_dev(off), M)
    keep = [i for i in range(60) if i not in (7, 25)]
    assert torch.equal(got[keep], ref[keep])
    assert bool(torch.isnan(got[7]).all()) and not bool(torch.isfinite(got[25]).any())


def test_dgrad_is_the_forward_products_adjoint():
    # <dy, gmm(x)> = <dgrad(dy), x>: the forward kernel against this one, as
    # the difference of a linear map; both sides f32 sums of N (K) products
    E, N, K = 6, 512, 384
    off, M = bands([40, 0, 3, 70, 1, 130])
    w, packed = make_weights(E, N, K, "mxfp4", seed=9)
    x, dyb = random_dy(M, K, 10), random_dy(M, N, 11)
    y = moe.moe_gmm(packed, moe.MXFP4, E, N, K, to_dev(x), to_dev(off), M)
    dx = moe.moe_gmm_dgrad(packed, moe.MXFP4, E, N, K, to_dev(dyb), to_dev(off), M)
    x64, dy64 = bf16_bits_to_f64(x), bf16_bits_to_f64(dyb)
    size = (np.abs(oracle.gmm_dgrad(dy64, off, w, absolute=True)) * np.abs(x64)).sum(axis=1)
    left, right = (f64(y) * dy64).sum(axis=1), (f64(dx) * x64).sum(axis=1)
    assert (np.abs(left - right) <= 2 * (N + K) * EPS * size).all()


def test_dgrad_same_bits_every_call():
    E, N, K = 16, 256, 512
    off, M = bands([9, 140, 0, 33] * 4)
    _, packed = make_weights(E, N, K, "nvfp4", seed=2)
    dy, o = to_dev(random_dy(M, N, 3)), to_dev(off)
    a = moe.moe_gmm_dgrad(packed, moe.NVFP4, E, N, K, dy, o, M)
    for _ in range(5):
        assert torch.equal(moe.moe_gmm_dgrad(packed, moe.NVFP4, E, N, K, dy, o, M), a)


# ----------------------------------------------------------- a whole layer ---

def layer(x, logits, wg, packs, dims, dout, fmt=moe.MXFP4):
    """Forward and backward of a layer on the GPU, as a training step runs it."""
    T, k, E, D, I = dims
    M = T * k
    p13, p2 = packs
    ids, tw = moe.topk_gate(logits, k, score=moe.GATE_SIGMOID, bias=wg, scale=1.5)
    r = moe.route_sort(ids, E)
    off = r["group_offsets"]
    y13 = moe.moe_gmm(p13, fmt, E, 2 * I, D, x, off, M, row_index=r["sorted_token"])
    h = moe.silu_mul(y13, group_offsets=off, out_dtype=moe.BF16)
    y2 = moe.moe_gmm(p2, fmt, E, D, I, h, off, M, out_dtype=moe.BF16)
    out = moe.moe_combine(y2, tw, r["pair_row"])
    dy2, dw = moe.moe_combine_bwd(dout, y2, tw, r["pair_row"], out_dtype=moe.BF16)
    d13 = moe.moe_gmm_dgrad(p2, fmt, E, D, I, dy2, off, M, out_dtype=moe.BF16, act=moe.ACT_SILU_MUL, preact=y13)
    dxs = moe.moe_gmm_dgrad(p13, fmt, E, 2 * I, D, d13, off, M, out_dtype=moe.BF16)
    dx = moe.moe_dispatch_bwd(dxs, r["pair_row"], k)
    dl = moe.topk_gate_bwd(logits, ids, dw, score=moe.GATE_SIGMOID, scale=1.5)
    return ids, tw, out, dx, dl


def layer_inputs(T, k, E, D, I, seed):
    rng = np.random.default_rng(seed)
    w13 = make_problem(T=2, k=1, E=E, K=D, N=2 * I, seed=seed, exp_range=(-6, -4))
    w2 = make_problem(T=2, k=1, E=E, K=I, N=D, seed=seed + 1, exp_range=(-6, -4))
    packs = [moe.mxfp4_encode(to_dev(q["codes"]), to_dev(q["scales"])) for q in (w13, w2)]
    ws = [{"fmt": "mxfp4", "codes": q["codes"], "scales": q["scales"]} for q in (w13, w2)]
    x = dev(rng.standard_normal((T, D)), torch.bfloat16)
    logits = dev(rng.standard_normal((T, E)), torch.float32)
    bias = dev(rng.standard_normal(E) * 0.1, torch.float32)
    dout = dev(rng.standard_normal((T, D)), torch.float32)
    return x, logits, bias, packs, ws, dout


def test_layer_forward_and_backward_against_the_formulas():
    T, k, E, D, I = 50, 3, 8, 256, 128
    x, logits, bias, packs, ws, dout = layer_inputs(T, k, E, D, I, seed=50)
    ids, tw, out, dx, dl = layer(x, logits, bias, packs, (T, k, E, D, I), dout)
    # the same layer in torch's float64 autograd on the CPU, the choice fixed
    rid, _ = oracle.topk_gate(f64(logits), k, "sigmoid", f64(bias))
    assert np.array_equal(ids.cpu().numpy(), rid)
    xt = torch.from_numpy(f64(x)).requires_grad_()
    lt = torch.from_numpy(f64(logits)).requires_grad_()
    s = torch.gather(torch.sigmoid(lt), 1, torch.from_numpy(rid.astype(np.int64)))
    wt = 1.5 * s / s.sum(1, keepdim=True)
    W13 = torch.from_numpy(np.stack([oracle.dense_weights(ws[0], e) for e in range(E)]))
    W2 = torch.from_numpy(np.stack([oracle.dense_weights(ws[1], e) for e in range(E)]))
    rows = []
    for t in range(T):
        acc = 0
        for j in range(k):
            e = int(rid[t, j])
            y13 = W13[e] @ xt[t]
            h = torch.nn.functional.silu(y13[:I]) * y13[I:]
            acc = acc + wt[t, j] * (W2[e] @ h)
        rows.append(acc)
    o = torch.stack(rows)
    (o * torch.from_numpy(f64(dout))).sum().backward()
    # bf16 roundings on the way: h, y2 forward; dy2, d13, dxs (and y2 in dw)
    # backward.  Each is at most 2^-8 of its value and independent of the
    # others' signs; over the tensor their effect adds up to at most the sum of
    # the steps in norm
    rel = lambda a, b: float(np.linalg.norm(f64(a) - b.numpy()) / np.linalg.norm(b.numpy()))  # noqa: E731
    assert rel(tw, wt.detach()) < 1e-6
    assert rel(out, o.detach()) < 2 * 2.0 ** -8
    assert rel(dx, xt.grad) < 4 * 2.0 ** -8
    assert rel(dl, lt.grad) < 4 * 2.0 ** -8


def test_layer_training_step_captured_in_a_graph():
    # forward and backward captured once, replayed on new inputs with eager
    # work and synchronisations between: the eager bits every time
    T, k, E, D, I = 40, 2, 8, 256, 128
    x, logits, bias, packs, _, dout = layer_inputs(T, k, E, D, I, seed=60)
    step = lambda: layer(x, logits, bias, packs, (T, k, E, D, I), dout)  # noqa: E731
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    torch.cuda.synchronize()
    for i in range(4):
        nx, nl, _, _, _, nd = layer_inputs(T, k, E, D, I, seed=70 + i)
        x.copy_(nx)
        logits.copy_(nl)
        dout.copy_(nd)
        ref = step()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, ref):
            assert torch.equal(a, b), i


def test_parameters_and_views_are_taken_and_strided_ones_refused():
    # an nn.Parameter router output, a row range of a larger buffer; a column
    # range or a transposed view is refused, not read wrongly
    x = torch.nn.Parameter(torch.randn((9, 16), device=DEV))
    ids, w = moe.topk_gate(x, 2)
    ids2, w2 = moe.topk_gate(x.detach(), 2)
    assert torch.equal(ids, ids2) and torch.equal(w, w2)
    big = torch.randn((20, 16), device=DEV)
    assert torch.equal(moe.silu_mul(big[4:13]), moe.silu_mul(big[4:13].clone()))
    for bad in (big[:, :8], big.t(), big[::2]):
        with pytest.raises(moe.MoeGmmError):
            moe.silu_mul(bad)
        with pytest.raises(moe.MoeGmmError):
            moe.topk_gate(bad, 2)
    # rows that start off a 16-byte boundary
    flat = torch.randn(4 * 12 + 2, device=DEV)
    with pytest.raises(moe.MoeGmmError):
        moe.moe_dispatch(flat[2:].view(4, 12), torch.arange(4, dtype=torch.int32, device=DEV), 1)


def test_operators_on_another_stream():
    T, k, E, D, I = 30, 2, 8, 128, 128
    x, logits, bias, packs, _, dout = layer_inputs(T, k, E, D, I, seed=80)
    ref = layer(x, logits, bias, packs, (T, k, E, D, I), dout)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = layer(x, logits, bias, packs, (T, k, E, D, I), dout)
    s.synchronize()
    for a, b in zip(got, ref):
        assert torch.equal(a, b)


def test_bf16_rounding_of_every_kind_of_value():
    # dispatch_bwd with k = 1 is a rounding alone: ties to even, the largest
    # finite values, subnormals, infinities and NaN as torch rounds them
    rng = np.random.default_rng(90)
    bits = rng.integers(0, 1 << 32, size=1 << 16, dtype=np.uint64).astype(np.uint32)
    ties = (rng.integers(0, 1 << 16, size=4096, dtype=np.uint32) << 16) | 0x8000
    edge = np.array([0, 0x80000000, 1, 0x7FFF, 0x8000, 0x8001, 0x7F7FFFFF, 0xFF7FFFFF, 0x7F7F7FFF, 0x7F7F8000,
                     0x7F800000, 0xFF800000, 0x7FC00000, 0x7F800001, 0x00800000, 0x007FFFFF], dtype=np.uint32)
    v = np.concatenate([bits, ties, edge])
    v = np.concatenate([v, np.zeros(-len(v) % 64, dtype=np.uint32)]).view(np.float32).reshape(-1, 64)
    x = torch.from_numpy(v.copy()).to(DEV)
    pr = torch.arange(x.shape[0], dtype=torch.int32, device=DEV)
    got, ref = moe.moe_dispatch_bwd(x, pr, 1, out_dtype=moe.BF16), x.bfloat16()
    assert torch.equal(torch.isnan(got), torch.isnan(ref))
    ok = ~torch.isnan(ref)
    # (0 + -0 is 0 in the sum: compare values)
    assert torch.equal(got[ok], ref[ok])


@pytest.mark.parametrize("E", [64, 200, 256, 1000])
def test_gate_gradient_reaches_experts_of_every_lane(E):
    # token t's slots name E - 1 - t, E - 2 - t, ...: an expert's place in the
    # row belongs to another lane than the slot's, each in turn.  Sigmoid
    # scores without renormalisation at logits 0: dl = g / 4, exactly.
    k = 8
    t = torch.arange(E, device=DEV)
    ids = ((E - 1 - t[:, None] - torch.arange(k, device=DEV)[None]) % E).int()
    g = torch.randint(1, 100, (E, k), device=DEV, generator=torch.Generator(DEV).manual_seed(E)).float()
    x = torch.zeros((E, E), device=DEV)
    ref = torch.zeros((E, E), device=DEV).scatter_(1, ids.long(), g / 4)
    got = moe.topk_gate_bwd(x, ids, g, score=moe.GATE_SIGMOID, renormalize=False)
    assert torch.equal(got, ref)


def test_gate_refuses_k_before_it_allocates():
    # 2^32 + 2 would be 2 to the C entry and its outputs would not fit anywhere
    x = torch.zeros((1 << 12, 16), device=DEV)
    for k in (-1, 0, 17, 1 << 30, (1 << 32) + 2):
        with pytest.raises(moe.MoeGmmError):
            moe.topk_gate(x, k)


@pytest.mark.parametrize("E", [257, 300, 512, 513, 1000, 1024])
@pytest.mark.parametrize("biased", [False, True])
def test_gate_chooses_among_ties_of_many_experts(E, biased):
    # few values, so that most choices are ties over lanes and registers; rows
    # with 0, 1, 3 and all experts live.  Sums of different values lie 1e-5 and
    # more apart, far above an ulp of f64: the ids are exact.
    rng = np.random.default_rng(E)
    T, k = 67, 64
    x = rng.choice([-1.0, 0.0, 0.5, 2.0], size=(T, E), p=[0.4, 0.4, 0.19, 0.01])
    x[:4] = -np.inf
    x[1, E - 1] = 0.5
    x[2, [0, E // 2, E - 2]] = 0.5
    x[3] = 0.0
    x = dev(x, torch.float32)
    b = dev(rng.choice([0.0, 0.1, -0.3], size=E), torch.float32) if biased else None
    for score, code in (("softmax", moe.GATE_SOFTMAX), ("sigmoid", moe.GATE_SIGMOID)):
        ids, _ = moe.topk_gate(x, k, score=code, bias=b)
        rid, _ = oracle.topk_gate(f64(x), k, score, None if b is None else f64(b), True, 1.0)
        assert np.array_equal(ids.cpu().numpy(), rid), (score, E)


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("T,k,N,K", [(700, 4, 320, 1024), (1024, 16, 512, 256)])
def test_dgrad_many_thin_tiles_stay_right_call_after_call(T, k, N, K, fmt):
    # 1,024 experts with bands of 0 to 40 rows: short walks, many tiles a CU,
    # operands that arrive late if any do
    E = 1024
    rng = np.random.default_rng(T)
    off, M = bands(rng.multinomial(T * k, rng.dirichlet(np.full(E, 2.0))))
    w, packed = make_weights(E, N, K, fmt, seed=T + K)
    bits = random_dy(M, N, seed=K)
    dy64 = bf16_bits_to_f64(bits)
    enum = moe.MXFP4 if fmt == "mxfp4" else moe.NVFP4
    d, o = to_dev(bits), to_dev(off)
    first = moe.moe_gmm_dgrad(packed, enum, E, N, K, d, o, M)
    close(f64(first), oracle.gmm_dgrad(dy64, off, w), dgrad_bound(dy64, off, w, N), torch.float32)
    other = torch.zeros((), dtype=torch.int64, device=DEV)
    for _ in range(200):
        other += (moe.moe_gmm_dgrad(packed, enum, E, N, K, d, o, M) != first).sum()
    assert int(other) == 0
