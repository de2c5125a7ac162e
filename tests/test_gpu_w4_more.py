"""moe_w4_gemv beyond tests/test_gpu_w4.py: workgroups that walk several blocks
of columns and several units of k, rows past a block, runs of scales that start
anywhere, capture, streams and refusals.  The same exact cases: every sum an
integer multiple of the smallest scale below 2^24 of it.
"""

import numpy as np
import pytest
import torch

import moe_grouped_gemm_route_amd as moe
from tests.gpu_util import DEV
from tests.test_gpu_w4 import BAD, check as near, dev, ids_of, problem, ref, run

pytestmark = pytest.mark.gpu


def check(p, **kw):
    dkw = {n: dev(t) for n, t in kw.items()}
    nkw = {n: t.numpy() for n, t in kw.items()}
    assert np.array_equal(run(p, **dkw).double().cpu().numpy(), ref(p, **nkw))


# T, N, K, G: columns past what the workgroups take at once, in blocks of two
# and of four tiles, and k past what their waves take at once
LONG = [(1, 20011, 96, 32), (1, 16400, 1056, 32), (1, 33, 8224, 32), (1, 70, 9216, 256), (2, 9001, 160, 32),
        (3, 16500, 160, 32), (5, 16403, 64, 64), (16, 16390, 128, 128), (40, 5003, 96, 32), (19, 16401, 128, 64),
        (33, 8195, 256, 128), (2, 40, 8224, 32), (7, 50, 9280, 64), (16, 33, 4736, 128), (20, 64, 4640, 32)]


@pytest.mark.parametrize("case", LONG)
@pytest.mark.parametrize("zeros", [False, True])
def test_long_dense(case, zeros):
    T, N, K, G = case
    check(problem(1, N, K, G, rows=T, zeros=zeros, exact=True, scale=torch.bfloat16 if N % 2 else torch.float32))


@pytest.mark.parametrize("T", range(1, 36))
@pytest.mark.parametrize("G", [32, 64, 128])
def test_every_number_of_rows(T, G):
    check(problem(2, 50, 640, G, rows=T, exact=True, scale=torch.bfloat16))


# the same with 16 rows a block under narrow groups: many rows, or several with
# many columns; k that ends inside a chunk, a group and a unit
MANY = [(9, 8200, 96, 32), (13, 8193, 160, 32), (17, 16390, 320, 64), (29, 40, 8224, 32), (57, 70, 9280, 64),
        (64, 33, 4640, 32), (31, 8207, 64, 64), (12, 16400, 192, 64), (48, 130, 512, 32), (61, 2100, 448, 64),
        (33, 2, 32, 32), (80, 17, 64, 64)]


@pytest.mark.parametrize("case", MANY)
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("scale", [torch.float32, torch.bfloat16])
def test_many_rows_of_narrow_groups(case, zeros, scale):
    T, N, K, G = case
    check(problem(15, N, K, G, rows=T, zeros=zeros, exact=True, scale=scale))


@pytest.mark.parametrize("case", [(31, 66, 576, 32), (60, 34, 1088, 64), (11, 8208, 128, 32)])
@pytest.mark.parametrize("out", [moe.F32, moe.BF16])
def test_activation_of_many_rows_of_narrow_groups(case, out):
    T, N, K, G = case
    p = problem(16, N, K, G, rows=T, scale=torch.bfloat16)
    near(run(p, out_dtype=out, act=moe.ACT_SILU_MUL), ref(p, act=True), out)


@pytest.mark.parametrize("G", [32, 64])
def test_a_row_that_is_not_finite_stays_alone_among_many(G):
    p = problem(17, 40, 704, G, rows=62, exact=True)
    clean = run(p)
    for value in (float("inf"), float("nan")):
        for t in (0, 21, 61):
            x = p["x"].clone()
            x[t, 577] = value
            y = run(dict(p, x=x))
            keep = torch.arange(62, device=y.device) != t
            assert torch.equal(y[keep], clean[keep]) and bool(y[t].isnan().all())
    p["scales"][11] = float("nan")
    y = run(p)
    keep = torch.arange(40, device=y.device) != 11
    assert torch.equal(y[:, keep], clean[:, keep]) and bool(y[:, 11].isnan().all())


@pytest.mark.parametrize("case", [(2, 3, 4, 40, 4640, 32), (1, 7, 5, 600, 4352, 128), (3, 5, 3, 4500, 96, 32)])
def test_long_pairs(case):
    T, k, E, N, K, G = case
    p = problem(3, N, K, G, E=E, rows=T, exact=True)
    ids = ids_of(4, T, k, E, BAD[:2])
    check(p, topk_ids=ids)
    check(p, topk_ids=ids, topk_weights=torch.exp2(torch.arange(T * k).remainder(4) - 2.0).view(T, k))
    # the same expert for every pair of a token, and nobody's
    same = torch.full((T, k), E - 1, dtype=torch.int32)
    check(p, topk_ids=same)
    check(p, topk_ids=torch.full((T, k), -1, dtype=torch.int32), topk_weights=torch.ones((T, k)))


@pytest.mark.parametrize("scale", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("case", [(1, 64, 512, 32), (4, 64, 512, 32), (7, 48, 512, 64), (12, 40, 512, 128),
                                  (30, 40, 512, 32), (58, 40, 512, 64)])
def test_scales_and_zero_points_that_start_anywhere(case, scale):
    T, N, K, G = case
    p = problem(5, N, K, G, rows=T, scale=scale, exact=True)
    want = ref(p)
    for shift in (1, 2, 3, 5):
        def moved(t):
            flat = torch.empty(t.numel() + shift, dtype=t.dtype, device=DEV)
            view = flat[shift:].view(t.shape)
            view.copy_(t)
            return view
        y = moe.w4_gemv(dev(p["codes"]), moved(p["scales"]), dev(p["x"]), zeros=moved(p["zeros"]))
        assert np.array_equal(y.double().cpu().numpy(), want)


def test_columns_and_experts_do_not_mix():
    """Scales of NaN in one column, and in one expert, reach only their own
    outputs (runs of scales that end inside a chunk among them)."""
    p = problem(6, 37, 160, 32, rows=3, exact=True)
    clean = run(p)
    p["scales"][11] = float("nan")
    y = run(p)
    keep = torch.arange(37) != 11
    assert torch.equal(y[:, keep], clean[:, keep]) and bool(y[:, 11].isnan().all())
    p = problem(7, 37, 160, 32, E=3, rows=2, exact=True)
    ids = torch.tensor([[0, 2], [2, 0]], dtype=torch.int32)
    clean = run(p, topk_ids=dev(ids))
    p["scales"][1] = float("nan")
    assert torch.equal(run(p, topk_ids=dev(ids)), clean)


def test_captured_and_replayed():
    """Gate and up of a token's experts, then their down weights summed, in one
    graph, replayed on new inputs with eager work between."""
    E, N, K, T, k = 5, 256, 512, 2, 3
    a = problem(8, N, K, 32, E=E, rows=T, exact=True)
    b = problem(9, K, N // 2, 64, E=E, rows=1, exact=True)
    ca, sa, za = (dev(a[n]) for n in ("codes", "scales", "zeros"))
    cb, sb, zb = (dev(b[n]) for n in ("codes", "scales", "zeros"))
    sa = sa / 64
    x = dev(a["x"])
    ids = dev(ids_of(10, T, k, E, (-1,)))
    w = torch.rand((T, k), device=DEV)
    h = torch.empty((T * k, N // 2), dtype=torch.bfloat16, device=DEV)
    y = torch.empty((T, K), device=DEV)
    d = torch.empty((T, N), device=DEV)

    def layer(h, y, d):
        moe.w4_gemv(ca, sa, x, zeros=za, topk_ids=ids, act=moe.ACT_SILU_MUL, out=h, out_dtype=moe.BF16)
        moe.w4_gemv(cb, sb, h, zeros=zb, topk_ids=ids, topk_weights=w, out=y)
        moe.w4_gemv(ca[0], sa[0], x, out=d)

    layer(h, y, d)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer(h, y, d)
    for seed in range(5):
        x.copy_(torch.randint(-4, 5, x.shape))
        ids.copy_(ids_of(20 + seed, T, k, E, (-1, E)))
        w.copy_(torch.rand((T, k)))
        for t in (h, y, d):
            t.fill_(7)
        graph.replay()
        got = [t.clone() for t in (h, y, d)]
        torch.cuda.synchronize()
        fresh = [torch.empty_like(t) for t in (h, y, d)]
        layer(*fresh)
        assert all(torch.equal(p, q) for p, q in zip(got, fresh))


def test_two_streams_at_once():
    ps = [problem(11, 4100, 2080, 32, rows=1, exact=True), problem(12, 2050, 1088, 64, rows=9, exact=True)]
    on = [[dev(p[n]) for n in ("codes", "scales", "x", "zeros")] for p in ps]
    want = [torch.from_numpy(ref(p)) for p in ps]
    streams = [torch.cuda.Stream() for _ in ps]
    got = [[] for _ in ps]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(8):
        for i, (c, s, x, z) in enumerate(on):
            with torch.cuda.stream(streams[i]):
                got[i].append(moe.w4_gemv(c, s, x, zeros=z))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(y.double().cpu(), want[i]) for y in got[i])


def test_refusals():
    p = problem(13, 32, 128, 32, rows=2)
    q = problem(14, 32, 128, 32, E=2, rows=2)
    c, s, x, z = (dev(p[n]) for n in ("codes", "scales", "x", "zeros"))
    ec, es = dev(q["codes"]), dev(q["scales"])
    ids = torch.zeros((2, 2), dtype=torch.int32, device=DEV)
    w = torch.ones((2, 2), device=DEV)
    bad = [lambda: moe.w4_gemv(c, s[:, :3].contiguous(), x),             # K % groups
           lambda: moe.w4_gemv(c, s[:31], x), lambda: moe.w4_gemv(c, s, x[:, :64].contiguous()),
           lambda: moe.w4_gemv(c, s, x, zeros=z[:, :2].contiguous()), lambda: moe.w4_gemv(c, s, x, zeros=z.int()),
           lambda: moe.w4_gemv(c, s, x.float()), lambda: moe.w4_gemv(c, s.half(), x),
           lambda: moe.w4_gemv(c, s, x[:0]), lambda: moe.w4_gemv(c, s, x.cpu()),
           lambda: moe.w4_gemv(c.t().contiguous().t(), s, x), lambda: moe.w4_gemv(ec, es, x),
           lambda: moe.w4_gemv(c, s, x, topk_ids=ids), lambda: moe.w4_gemv(c, s, x, topk_weights=w),
           lambda: moe.w4_gemv(ec, es, x[:1], topk_ids=ids),
           lambda: moe.w4_gemv(ec, es, x, topk_ids=ids.long()),
           lambda: moe.w4_gemv(ec, es, x, topk_ids=ids, topk_weights=w[:, :1].contiguous()),
           lambda: moe.w4_gemv(ec, es, x, topk_ids=ids, topk_weights=w, act=moe.ACT_SILU_MUL),
           lambda: moe.w4_gemv(c, s, x, act=2), lambda: moe.w4_gemv(c, s, x, out_dtype=torch.float16),
           lambda: moe.w4_gemv(c, s, x, out=torch.empty((2, 16), device=DEV)),
           lambda: moe.w4_gemv(c[:31], s[:31], x, act=moe.ACT_SILU_MUL),
           lambda: moe.w4_gemv(c, torch.ones((32, 8), device=DEV), x),   # groups of 16
           lambda: moe.w4_gemv(torch.empty(32 * 64 + 8, dtype=torch.uint8, device=DEV)[8:].view(32, 64), s, x)]
    for i, f in enumerate(bad):
        with pytest.raises(moe.MoeGmmError):
            f()
            pytest.fail("call %d was taken" % i)


def ones_but(N, K, lead=()):
    """Codes whose weights are 1 (c - 8), the last k of column N - 2 counting
    twice, and scales of 1, of 2 in the last column."""
    codes = torch.empty(lead + (N, K // 2), dtype=torch.uint8, device=DEV).fill_(0x99)
    codes[..., N - 2, K // 2 - 1] = 0xA9
    scales = torch.ones(lead + (N, K // 256), dtype=torch.bfloat16, device=DEV)
    scales[..., N - 1, :] = 2.0
    return codes, scales


def edges(T, K):
    x = torch.zeros((T, K), dtype=torch.bfloat16, device=DEV)
    t = torch.arange(T, device=DEV) % 5 + 1
    x[:, 0], x[:, K - 1] = 1.0, t.bfloat16()
    return x, t.float()


def test_many_pairs_of_a_matrix_past_32_bit_offsets():
    """So many rows that a workgroup would take 4 GiB of codes."""
    N, K, T = 131072, 65536, 600
    codes, scales = ones_but(N, K, (1,))
    x, t = edges(T, K)
    y = moe.w4_gemv(codes, scales, x, topk_ids=torch.zeros((T, 1), dtype=torch.int32, device=DEV))
    assert bool((y[:, : N - 2] == (1 + t)[:, None]).all())
    assert torch.equal(y[:, N - 2], 1 + 2 * t) and torch.equal(y[:, N - 1], 2 + 2 * t)


def test_many_rows_of_a_matrix_past_32_bit_offsets():
    N, K, T = 1 << 20, 32768, 520
    codes, scales = ones_but(N, K)
    x, t = edges(T, K)
    y = moe.w4_gemv(codes, scales, x, out_dtype=moe.BF16).float()
    assert bool((y[:, : N - 2] == (1 + t)[:, None]).all())
    assert torch.equal(y[:, N - 2], 1 + 2 * t) and torch.equal(y[:, N - 1], 2 + 2 * t)
