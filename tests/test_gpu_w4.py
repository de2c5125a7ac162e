"""moe_w4_gemv against the float64 oracle.

Exact cases: integer activations and power-of-two scales make every product and
every sum an integer multiple of the smallest scale below 2^24 of it, so f32
holds them exactly whatever the order, and the results must equal the oracle's
bit for bit.  Others: f32 results to the suite's max|delta| / max|ref| <= 1e-5,
bf16 ones to half a step (2^-8 of the value) beside that.
"""

import numpy as np
import pytest
import torch

import moe_grouped_gemm_route_amd as moe
import oracle
from tests.gpu_util import DEV, REL_TOL

pytestmark = pytest.mark.gpu

DT = {moe.F32: torch.float32, moe.BF16: torch.bfloat16}


def problem(seed, N, K, G, E=0, rows=1, scale=torch.float32, zeros=True, exact=False):
    g = torch.Generator().manual_seed(seed)
    lead = (E, N) if E else (N,)
    p = dict(codes=torch.randint(0, 256, lead + (K // 2,), generator=g, dtype=torch.uint8))
    if exact:
        p["scales"] = torch.exp2(torch.randint(-3, 1, lead + (K // G,), generator=g).float()).to(scale)
        p["x"] = torch.randint(-4, 5, (rows, K), generator=g).to(torch.bfloat16)
    else:
        p["scales"] = ((0.5 + torch.rand(lead + (K // G,), generator=g)) / (8 * K ** 0.5)).to(scale)
        p["x"] = torch.randn((rows, K), generator=g).to(torch.bfloat16)
    hi = 256 if exact and K <= 512 else 16
    p["zeros"] = torch.randint(0, hi, lead + (K // G,), generator=g, dtype=torch.uint8) if zeros else None
    return p


def dev(t):
    return None if t is None else t.to(DEV)


def run(p, **kw):
    return moe.w4_gemv(dev(p["codes"]), dev(p["scales"]), dev(p["x"]), zeros=dev(p["zeros"]), **kw)


def ref(p, **kw):
    f = lambda t: None if t is None else t.double().numpy()  # noqa: E731
    return oracle.w4_gemv(p["codes"].numpy(), f(p["scales"]), f(p["x"]),
                          zeros=None if p["zeros"] is None else p["zeros"].numpy(), **kw)


def check(got, want, out):
    got = got.double().cpu().numpy()
    slack = REL_TOL * np.max(np.abs(want))
    half = 2.0 ** -8 * np.abs(want) if out == moe.BF16 else 0.0
    assert np.all(np.abs(got - want) <= half + slack)


# T, N, K, G: one of everything, lengths that end inside a chunk and a tile,
# groups whose runs start at odd places, more rows than a workgroup takes
DENSE = [(1, 1, 32, 32), (1, 16, 128, 32), (1, 50, 96, 32), (3, 33, 160, 32), (4, 64, 384, 32), (5, 47, 224, 32),
         (8, 130, 1056, 32), (9, 32, 352, 32), (16, 70, 480, 32), (17, 20, 64, 32), (37, 34, 288, 32),
         (1, 17, 64, 64), (8, 66, 192, 64), (9, 48, 448, 64), (16, 100, 1088, 64), (17, 30, 320, 64), (40, 18, 704, 64),
         (1, 40, 128, 128), (2, 258, 4096, 128), (16, 31, 384, 128), (17, 64, 640, 128), (33, 90, 256, 128),
         (64, 40, 1152, 128), (65, 22, 128, 128), (130, 34, 512, 128), (1, 64, 256, 256), (31, 52, 768, 256)]


@pytest.mark.parametrize("case", DENSE)
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("scale", [torch.float32, torch.bfloat16])
def test_dense_exact(case, zeros, scale):
    T, N, K, G = case
    p = problem(1, N, K, G, rows=T, scale=scale, zeros=zeros, exact=True)
    assert np.array_equal(run(p).double().cpu().numpy(), ref(p))


@pytest.mark.parametrize("case", [(1, 64, 512, 32), (6, 96, 1088, 64), (16, 40, 384, 128), (64, 34, 2048, 256),
                                  (5, 2048, 4096, 128)])
@pytest.mark.parametrize("out", [moe.F32, moe.BF16])
@pytest.mark.parametrize("act", [moe.ACT_NONE, moe.ACT_SILU_MUL])
def test_dense_random(case, out, act):
    T, N, K, G = case
    p = problem(2, N, K, G, rows=T, scale=torch.bfloat16)
    y = run(p, out_dtype=out, act=act)
    assert y.dtype == DT[out] and tuple(y.shape) == (T, N // 2 if act else N)
    check(y, ref(p, act=bool(act)), out)


@pytest.mark.parametrize("case", [(1, 2, 32, 32), (4, 34, 128, 32), (9, 66, 416, 32), (8, 30, 320, 64),
                                  (20, 62, 128, 64), (33, 18, 256, 128), (70, 130, 512, 256)])
def test_dense_activation_of_exact_sums(case):
    T, N, K, G = case
    p = problem(3, N, K, G, rows=T, exact=True)
    p["scales"] = p["scales"] / 64
    check(run(p, act=moe.ACT_SILU_MUL), ref(p, act=True), moe.F32)


def ids_of(seed, T, k, E, bad=()):
    g = torch.Generator().manual_seed(seed)
    ids = torch.randint(0, E, (T, k), generator=g, dtype=torch.int32)
    for i, v in enumerate(bad):
        ids.view(-1)[(i * 5 + 1) % (T * k)] = v
    return ids


BAD = (-1, 1 << 20, -(1 << 31), (1 << 31) - 1)


@pytest.mark.parametrize("case", [(1, 1, 1, 16, 32, 32), (1, 6, 8, 40, 416, 32), (3, 2, 5, 33, 192, 64),
                                  (7, 4, 3, 18, 256, 128), (2, 64, 4, 16, 256, 256), (16, 8, 16, 50, 512, 32)])
@pytest.mark.parametrize("per_pair", [False, True])
@pytest.mark.parametrize("zeros", [False, True])
def test_pairs_exact(case, per_pair, zeros):
    T, k, E, N, K, G = case
    p = problem(4, N, K, G, E=E, rows=T * k if per_pair else T, zeros=zeros, exact=True)
    ids = ids_of(5, T, k, E, BAD[:T * k // 2])
    y = run(p, topk_ids=dev(ids))
    assert tuple(y.shape) == (T * k, N)
    assert np.array_equal(y.double().cpu().numpy(), ref(p, topk_ids=ids.numpy()))
    # summed with weights that f32 holds exactly beside the sums
    w = torch.exp2(torch.randint(-2, 2, (T, k), generator=torch.Generator().manual_seed(6)).float())
    y = run(p, topk_ids=dev(ids), topk_weights=dev(w))
    assert tuple(y.shape) == (T, N)
    assert np.array_equal(y.double().cpu().numpy(), ref(p, topk_ids=ids.numpy(), topk_weights=w.numpy()))


@pytest.mark.parametrize("out", [moe.F32, moe.BF16])
@pytest.mark.parametrize("scale", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("G", [32, 64, 128])
def test_pairs_random(out, scale, G):
    T, k, E, N, K = 5, 3, 7, 130, 1152
    p = problem(7, N, K, G, E=E, rows=T, scale=scale)
    ids = ids_of(8, T, k, E, BAD)
    check(run(p, topk_ids=dev(ids), out_dtype=out, act=moe.ACT_SILU_MUL), ref(p, topk_ids=ids.numpy(), act=True), out)
    w = torch.softmax(torch.randn((T, k), generator=torch.Generator().manual_seed(9)), 1)
    p["x"] = torch.randn((T * k, K), generator=torch.Generator().manual_seed(10)).to(torch.bfloat16)
    check(run(p, topk_ids=dev(ids), topk_weights=dev(w), out_dtype=out),
          ref(p, topk_ids=ids.numpy(), topk_weights=w.numpy()), out)


def test_a_dropped_pair_adds_nothing_whatever_its_weight():
    p = problem(11, 32, 256, 32, E=3, rows=2, exact=True)
    ids = torch.tensor([[0, -1], [-1, 7]], dtype=torch.int32)
    w = torch.tensor([[0.5, float("nan")], [float("inf"), float("nan")]])
    y = run(p, topk_ids=dev(ids), topk_weights=dev(w)).double().cpu().numpy()
    want = 0.5 * oracle.w4_weights(p["codes"][0].numpy(), p["scales"][0].double().numpy(), p["zeros"][0].numpy()) @ \
        p["x"][0].double().numpy()
    assert np.array_equal(y[0], want) and not y[1].any()
    y = run(p, topk_ids=dev(ids), act=moe.ACT_SILU_MUL)
    assert not y[1:].any() and bool(torch.isfinite(y).all())


@pytest.mark.parametrize("G", [32, 64, 128])
def test_a_row_that_is_not_finite_stays_alone(G):
    p = problem(12, 48, 256, G, rows=19, exact=True)
    clean = run(p)
    for value in (float("inf"), float("nan")):
        for t in (0, 5, 18):
            x = p["x"].clone()
            x[t, 77] = value
            y = run(dict(p, x=x))
            keep = torch.arange(19) != t
            assert torch.equal(y.cpu()[keep], clean.cpu()[keep])
            assert bool(y[t].isnan().all())


def test_out_streams_and_repeats():
    p = problem(13, 4096, 2048, 64, rows=3, scale=torch.bfloat16)
    codes, scales, x = dev(p["codes"]), dev(p["scales"]), dev(p["x"])
    zeros = dev(p["zeros"])
    a = moe.w4_gemv(codes, scales, x, zeros=zeros)
    out = torch.full((3, 4096), 7.0, device=DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b = moe.w4_gemv(codes, scales, x, zeros=zeros, out=out)
    torch.cuda.current_stream().wait_stream(s)
    assert b is out and torch.equal(a, out)
    for _ in range(5):
        assert torch.equal(a, moe.w4_gemv(codes, scales, x, zeros=zeros))


def test_past_32_bit_offsets():
    """Experts and columns whose codes start past 2^32 bytes, scales past 2^31."""
    E, N, K, G = 3, 65552, 49152, 32
    codes = torch.zeros((E, N, K // 2), dtype=torch.uint8, device=DEV).fill_(0x99)    # c - 8 = 1
    scales = torch.ones((E, N, K // G), dtype=torch.bfloat16, device=DEV)
    scales[2, N - 1] = 2.0
    codes[2, N - 2, K // 2 - 1] = 0xA9                                                # the last k counts twice
    x = torch.zeros((1, K), dtype=torch.bfloat16, device=DEV)
    x[0, 0], x[0, K - 1] = 1.0, 4.0
    ids = torch.tensor([[2]], dtype=torch.int32, device=DEV)
    y = moe.w4_gemv(codes, scales, x, topk_ids=ids)[0].cpu()
    assert bool((y[: N - 2] == 5.0).all()) and y[N - 2] == 9.0 and y[N - 1] == 10.0
