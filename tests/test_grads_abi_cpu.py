"""Argument checks of the router, the permutation's gradients, the activation
and the product's gradient on the host (no GPU needed): every call here is
rejected before any HIP call."""

import ctypes

import pytest
import torch

import moe_grouped_gemm_route_amd as moe

ERR_NULL, ERR_SHAPE, ERR_FORMAT, ERR_UNSUPPORTED = 1, 2, 3, 4
A = ctypes.c_void_p(1 << 30)            # aligned, never dereferenced
B8 = ctypes.c_void_p((1 << 30) + 8)     # 8-byte aligned only


@pytest.fixture(scope="module")
def lib():
    return moe.library()


def _call(fn, order, base, **kw):
    d = dict(base, **kw)
    return fn(*[d[n] for n in order], None)


def _gate(lib, **kw):
    return _call(lib.moe_topk_gate, "x dt bias T E k score renorm scale ids w".split(),
                 dict(x=A, dt=0, bias=None, T=4, E=8, k=2, score=0, renorm=1, scale=1.0, ids=A, w=A), **kw)


def _gate_bwd(lib, **kw):
    return _call(lib.moe_topk_gate_bwd, "x dt ids dw T E k score renorm scale dx".split(),
                 dict(x=A, dt=0, ids=A, dw=A, T=4, E=8, k=2, score=0, renorm=1, scale=1.0, dx=A), **kw)


def test_gate_validation(lib):
    for call, ptrs in ((_gate, ("x", "ids", "w")), (_gate_bwd, ("x", "ids", "dw", "dx"))):
        for n in ptrs:
            assert call(lib, **{n: None}) == ERR_NULL, n
        for kw in (dict(T=0), dict(T=-1), dict(E=0), dict(E=1025), dict(k=0), dict(k=9), dict(E=128, k=65),
                   dict(T=(1 << 24) // 2 + 1)):
            assert call(lib, **kw) == ERR_SHAPE, kw
        for kw in (dict(dt=2), dict(dt=-1), dict(score=2), dict(score=-1)):
            assert call(lib, **kw) == ERR_FORMAT, kw


def test_permutation_validation(lib):
    d = lambda **kw: _call(lib.moe_dispatch, "x dt pr T k N rows xs".split(),  # noqa: E731
                           dict(x=A, dt=0, pr=A, T=4, k=2, N=8, rows=8, xs=A), **kw)
    b = lambda **kw: _call(lib.moe_dispatch_bwd, "x dt pr T k N rows out odt".split(),  # noqa: E731
                           dict(x=A, dt=0, pr=A, T=4, k=2, N=8, rows=8, out=A, odt=1), **kw)
    c = lambda **kw: _call(lib.moe_combine_bwd, "g dt y ydt w pr T k N rows dy odt dw".split(),  # noqa: E731
                           dict(g=A, dt=0, y=A, ydt=1, w=A, pr=A, T=4, k=2, N=8, rows=8, dy=A, odt=0, dw=A), **kw)
    for call, ptrs in ((d, ("x", "pr", "xs")), (b, ("x", "pr", "out")), (c, ("g", "y", "w", "pr", "dy", "dw"))):
        for n in ptrs:
            assert call(**{n: None}) == ERR_NULL, n
        for kw in (dict(T=0), dict(k=0), dict(k=65), dict(N=0), dict(N=6), dict(N=-4), dict(N=(1 << 30) + 4),
                   dict(rows=0), dict(rows=(1 << 24) + 1), dict(T=1 << 23, k=4), dict(T=1 << 20, N=1 << 20),
                   dict(rows=1 << 20, N=1 << 20)):
            assert call(**kw) == ERR_SHAPE, kw
        assert call(dt=2) == ERR_FORMAT
    assert b(odt=3) == ERR_FORMAT and c(ydt=3) == ERR_FORMAT and c(odt=-1) == ERR_FORMAT
    for call, names in ((d, ("x", "xs")), (b, ("x", "out")), (c, ("g", "y", "dy"))):
        for n in names:
            assert call(**{n: B8}) == ERR_SHAPE, n


def test_silu_mul_validation(lib):
    f = lambda **kw: _call(lib.moe_silu_mul, "y dt M N n h odt".split(),  # noqa: E731
                           dict(y=A, dt=0, M=4, N=16, n=None, h=A, odt=1), **kw)
    assert f(y=None) == ERR_NULL and f(h=None) == ERR_NULL
    for kw in (dict(M=0), dict(M=(1 << 24) + 1), dict(N=0), dict(N=12), dict(N=(1 << 30) + 8),
               dict(M=1 << 20, N=1 << 20), dict(y=B8), dict(h=B8)):
        assert f(**kw) == ERR_SHAPE, kw
    assert f(dt=4) == ERR_FORMAT and f(odt=4) == ERR_FORMAT


def test_dgrad_validation(lib):
    f = lambda **kw: _call(lib.moe_gmm_dgrad, "packed fmt E N K dy off M pre pdt dx odt act".split(),  # noqa: E731
                           dict(packed=A, fmt=0, E=8, N=512, K=256, dy=A, off=A, M=128, pre=None, pdt=0, dx=A, odt=0,
                                act=0), **kw)
    for n in ("packed", "dy", "off", "dx"):
        assert f(**{n: None}) == ERR_NULL, n
    assert f(act=1) == ERR_NULL                             # the activation's gradient needs its sums
    assert f(pre=A) == ERR_FORMAT                           # and the plain gradient takes none
    assert f(act=2) == ERR_FORMAT and f(act=-1) == ERR_FORMAT
    assert f(act=1, pre=A, pdt=2) == ERR_FORMAT
    assert f(act=1, pre=B8) == ERR_SHAPE
    assert f(fmt=2) == ERR_UNSUPPORTED
    assert f(fmt=3) == ERR_FORMAT and f(odt=2) == ERR_FORMAT
    for kw in (dict(E=0), dict(E=1025), dict(N=500), dict(K=200), dict(M=0), dict(M=(1 << 24) + 1), dict(dy=B8),
               dict(dx=B8), dict(packed=ctypes.c_void_p((1 << 30) + 128)),
               dict(E=1, N=1 << 16, K=1 << 16),             # an expert's codes past 2^31 - 64 KiB
               dict(E=1, N=1 << 23, K=128),                 # a tile's dy rows likewise
               dict(E=1, N=64, K=1 << 25, M=1 << 24)):      # a grid past the dispatch limit
        assert f(**kw) == ERR_SHAPE, kw


def test_binding_rejects_host_tensors_and_wrong_types():
    f, i = torch.zeros((4, 8)), torch.zeros(8, dtype=torch.int32)
    calls = [lambda: moe.topk_gate(f, 2), lambda: moe.topk_gate_bwd(f, i.view(4, 2), f),
             lambda: moe.moe_dispatch(f, i, 2), lambda: moe.moe_dispatch_bwd(f, i, 2),
             lambda: moe.moe_combine_bwd(f, f, f, i), lambda: moe.silu_mul(f),
             lambda: moe.moe_gmm_dgrad(f, 0, 1, 64, 128, f, i, 4),
             lambda: moe.topk_gate(f.to(torch.float16), 2), lambda: moe.silu_mul(f.double())]
    for c in calls:
        with pytest.raises(moe.MoeGmmError):
            c()
