"""Every tile and every number of shares that the dense block's products can
take, on sizes that end inside tiles and stages: small integers, so that sums
are exact in f32 whatever the order and must equal plain f32 products bit for
bit (themselves exact).  And the same calls captured, on other streams and
beside each other.
"""

import pytest
import torch

import moe_grouped_gemm_route_amd as moe
from tests.gpu_util import DEV

pytestmark = pytest.mark.gpu

F, B = moe.F32, moe.BF16


def ints(g, shape, lo=-3, hi=4, dtype=torch.bfloat16):
    return torch.randint(lo, hi, shape, generator=g, device=DEV).to(dtype)


def inputs(seed, M, N, K):
    """dh, x, w13 and kept sums with gates 0 and 64: a sigmoid of 1/2 and 1."""
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    pre = torch.cat((ints(g, (M, N // 2), 0, 2) * 64, ints(g, (M, N // 2))), 1)
    return ints(g, (M, N // 2)), ints(g, (M, K)), ints(g, (N, K)), pre


def plain(dh, x, w, pre):
    g, u = pre.float().chunk(2, dim=1)
    e = dh.float()
    d = torch.cat((torch.where(g > 0, e * u, e * u / 2), torch.where(g > 0, e * 64, 0.0)), 1)
    return d @ w.float(), d.t() @ x.float()


SHAPES = [(17, 2912, 2704), (1414, 4144, 144), (676, 16, 2824), (921, 32, 8), (2028, 16, 8), (725, 16, 24),
          (2947, 16, 2600), (2721, 16, 2192), (2419, 80, 792), (2071, 1888, 136), (2299, 960, 8), (2701, 2848, 664),
          (2798, 2752, 272), (33, 784, 16), (18, 992, 8), (2078, 1712, 136), (2209, 1104, 24), (29, 928, 24),
          (18, 2432, 8), (2354, 16, 1688), (2707, 2640, 672), (2766, 1456, 272), (2339, 2320, 136), (65, 3680, 2104),
          (2482, 16, 3144), (199, 784, 3040), (27, 400, 16), (2476, 3120, 8), (193, 4480, 8), (199, 4192, 72),
          (98, 4336, 8), (16, 4112, 2056), (9, 6000, 264), (1, 4400, 8200), (237, 2832, 200), (250, 4112, 1032),
          (450, 2832, 72), (513, 4112, 520), (774, 4224, 8), (1001, 2080, 8), (2795, 4048, 280), (2103, 3888, 136),
          (1050, 992, 8), (2163, 1616, 152), (1, 976, 2176)]


@pytest.mark.parametrize("shape", SHAPES)
def test_every_plan(shape):
    dh, x, w, pre = inputs(1, *shape)
    assert torch.equal(moe.gate_up(x, w, preact_dtype=F)[1], x.float() @ w.float().t())
    want = plain(dh, x, w, pre)
    for types in ((F, F), (B, B)):
        got = moe.gate_up_bwd(dh, x, w, pre, dx_dtype=types[0], dw_dtype=types[1])
        for a, b in zip(got, want):
            assert torch.equal(a, b.to(a.dtype))


@pytest.mark.parametrize("shape", [(1, 512, 512), (40, 272, 520), (300, 1040, 264), (700, 4112, 72)])
def test_captured_and_replayed(shape):
    """A forward and a backward step in one graph, replayed on new inputs with
    eager work between, each replay against the eager calls."""
    M, N, K = shape
    dh, x, w, pre = inputs(2, M, N, K)
    ws = torch.empty(moe.gate_up_bwd_workspace_bytes(M, N, K, B, F), dtype=torch.uint8, device=DEV)
    h = torch.empty((M, N // 2), device=DEV)
    kept = torch.empty((M, N), device=DEV)
    dx = torch.empty((M, K), dtype=torch.bfloat16, device=DEV)
    dw = torch.empty((N, K), device=DEV)

    def both():
        moe.gate_up(x, w, out=h, preact=kept)
        moe.gate_up_bwd(dh, x, w, pre, dx=dx, dw13=dw, ws=ws)

    both()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for seed in range(3, 8):
        for old, new in zip((dh, x, w, pre), inputs(seed, M, N, K)):
            old.copy_(new)
        ws.fill_(seed)
        for t in (h, kept, dx, dw):
            t.fill_(7)
        graph.replay()
        got = [t.clone() for t in (h, kept, dx, dw)]
        torch.cuda.synchronize()
        eh, ey = moe.gate_up(x, w, preact_dtype=F)
        ex, ew = moe.gate_up_bwd(dh, x, w, pre, dx_dtype=B, dw_dtype=F)
        for a, b in zip(got, (eh, ey, ex, ew)):
            assert torch.equal(a, b)
        assert torch.equal(ey, x.float() @ w.float().t())


def test_two_streams_at_once():
    """Calls with workspaces of their own on two streams."""
    shapes = [(513, 1040, 520), (200, 2064, 136)]
    data = [inputs(11 + i, *s) for i, s in enumerate(shapes)]
    want = [plain(*d) for d in data]
    streams = [torch.cuda.Stream() for _ in shapes]
    got = [[] for _ in shapes]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(6):
        for i, d in enumerate(data):
            with torch.cuda.stream(streams[i]):
                got[i].append(moe.gate_up_bwd(*d))
                got[i].append((moe.gate_up(d[1], d[2], preact_dtype=F)[1],))
    torch.cuda.synchronize()
    for i, d in enumerate(data):
        y = d[1].float() @ d[2].float().t()
        for r in got[i]:
            for a, b in zip(r, want[i] if len(r) == 2 else (y,)):
                assert torch.equal(a, b)


def test_repeats_give_the_same_bits():
    g = torch.Generator(device=DEV)
    g.manual_seed(21)
    M, N, K = 333, 1040, 1160
    x, w = (torch.randn(s, generator=g, device=DEV).bfloat16() for s in ((M, K), (N, K)))
    pre, dh = (torch.randn(s, generator=g, device=DEV) for s in ((M, N), (M, N // 2)))
    first = moe.gate_up(x, w, preact_dtype=F) + moe.gate_up_bwd(dh, x, w, pre)
    for _ in range(5):
        again = moe.gate_up(x, w, preact_dtype=F) + moe.gate_up_bwd(dh, x, w, pre)
        assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_refusals():
    dh, x, w, pre = inputs(31, 8, 32, 64)
    E = moe.MoeGmmError
    with pytest.raises(E):
        moe.gate_up(x.t().contiguous().t(), w)                      # strides
    with pytest.raises(E):
        moe.gate_up(x, w[:31])                                      # an odd number of rows
    with pytest.raises(E):
        moe.gate_up(x, w[:24])                                      # and one of 8 each
    with pytest.raises(E):
        moe.gate_up(x[:, :60].contiguous(), w[:, :60].contiguous())
    with pytest.raises(E):
        moe.gate_up(x[:0], w)
    with pytest.raises(E):
        moe.gate_up(x, w.float())
    with pytest.raises(E):
        moe.gate_up(x, w.cpu())
    with pytest.raises(E):
        moe.gate_up(x, w, out_dtype=torch.float16)
    with pytest.raises(E):
        moe.gate_up(x, w, out=torch.empty((8, 32), device=DEV))
    flat = torch.empty(8 * 64 + 8, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(E):
        moe.gate_up(flat[4:4 + 8 * 64].view(8, 64), w)              # 8-byte aligned only
    with pytest.raises(E):
        moe.gate_up_bwd(dh, x, w, pre, dx_dtype=None, dw_dtype=None)
    with pytest.raises(E):
        moe.gate_up_bwd(dh[:, :8].contiguous(), x, w, pre)
    with pytest.raises(E):
        moe.gate_up_bwd(dh, x, w, pre[:7])
    with pytest.raises(E):
        moe.gate_up_bwd(dh, x, w, pre, ws=torch.empty(16, dtype=torch.uint8, device=DEV))
    big = torch.empty(moe.gate_up_bwd_workspace_bytes(8, 32, 64) + 512, dtype=torch.uint8, device=DEV)
    with pytest.raises(E):
        moe.gate_up_bwd(dh, x, w, pre, ws=big[128:])
    with pytest.raises(E):
        moe.gate_up_bwd(dh, x, w, pre, ws=big.cpu())
    for kw in (dict(out=[]), dict(preact=[]), dict(out=torch.empty((8, 16))), dict(preact=torch.empty((8, 32)))):
        with pytest.raises(E):
            moe.gate_up(x, w, **kw)                                 # no device tensors
    for kw in (dict(dx=[]), dict(dw13=[]), dict(ws=1), dict(dx=torch.empty((8, 64))), dict(dw13=torch.empty((32, 64)))):
        with pytest.raises(E):
            moe.gate_up_bwd(dh, x, w, pre, **kw)


def test_rows_past_32_bit_offsets():
    """x and dx past 2^32 bytes, and the sum over their rows."""
    M, N, K = 270_017, 16, 8200
    dh, x, w, pre = inputs(41, M, N, K)
    assert x.numel() * 2 > 1 << 32
    assert torch.equal(moe.gate_up(x, w, preact_dtype=F)[1], x.float() @ w.float().t())
    dx, dw = moe.gate_up_bwd(dh, x, w, pre, dx_dtype=B, dw_dtype=F)
    want = plain(dh[-4096:], x[-4096:], w, pre[-4096:])[0]
    assert torch.equal(dx[-4096:], want.bfloat16())
    assert torch.equal(dx[:4096], plain(dh[:4096], x[:4096], w, pre[:4096])[0].bfloat16())
    # d is a multiple of 1/2 up to 192, x up to 3: the sums stay below 2^24 halves
    # only block by block, so f64 adds them up and f32 rounding is allowed for
    total = torch.zeros((N, K), dtype=torch.float64, device=DEV)
    size = torch.zeros_like(total)
    for a in range(0, M, 4096):
        b = slice(a, a + 4096)
        total += plain(dh[b], x[b], w, pre[b])[1].double()
        size += plain(dh[b].abs(), x[b].abs(), w, pre[b].abs())[1].double()
    # at most M / 32 additions in a row, each to 2^-23 of the sum of magnitudes
    assert bool(((dw.double() - total).abs() <= (M / 32 + 64) * 2.0 ** -23 * size).all())


def test_weights_past_32_bit_offsets():
    M, N, K = 21, 270_016, 8200
    dh, x, w, pre = inputs(42, M, N, K)
    y = moe.gate_up(x, w, preact_dtype=F)[1]
    for a in (0, N // 2 - 2048, N - 4096):
        assert torch.equal(y[:, a:a + 4096], x.float() @ w[a:a + 4096].float().t())
    one = moe.gate_up(x[:9], w, preact_dtype=F)[1]
    assert torch.equal(one, y[:9])
    dw = moe.gate_up_bwd(dh, x, w, pre, dx_dtype=None, dw_dtype=B)[1]
    g, u = pre.float().chunk(2, dim=1)
    d = torch.cat((torch.where(g > 0, dh * u, dh * u / 2), torch.where(g > 0, dh * 64, 0.0)), 1).float()
    for a in (0, N // 2 - 2048, N - 4096):
        assert torch.equal(dw[a:a + 4096], (d[:, a:a + 4096].t() @ x.float()).bfloat16())
