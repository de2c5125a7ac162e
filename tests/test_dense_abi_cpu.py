"""Argument checks of the 4-bit integer products and the dense gated block on
the host (no GPU needed): every call here is rejected before any HIP call."""

import ctypes

import pytest
import torch

import moe_grouped_gemm_route_amd as moe
from tests.test_grads_abi_cpu import A, B8, ERR_FORMAT, ERR_NULL, ERR_SHAPE, ERR_UNSUPPORTED, _call

B1 = ctypes.c_void_p((1 << 30) + 1)
B2 = ctypes.c_void_p((1 << 30) + 2)


@pytest.fixture(scope="module")
def lib():
    return moe.library()


def test_w4_validation(lib):
    order = "codes scales sdt zeros group E N K x rows T ids w k y odt act".split()
    dense = dict(codes=A, scales=A, sdt=0, zeros=None, group=32, E=1, N=64, K=256, x=A, rows=4, T=4, ids=None, w=None,
                 k=1, y=A, odt=0, act=0)
    f = lambda **kw: _call(lib.moe_w4_gemv, order, dense, **kw)  # noqa: E731
    r = lambda **kw: _call(lib.moe_w4_gemv, order, dict(dense, E=8, ids=A, k=2), **kw)  # noqa: E731
    for n in ("codes", "scales", "x", "y"):
        assert f(**{n: None}) == ERR_NULL and r(**{n: None}) == ERR_NULL, n
    assert f(w=A) == ERR_NULL                                # weights without ids
    assert r(w=A, act=1) == ERR_UNSUPPORTED
    for kw in (dict(sdt=2), dict(sdt=-1), dict(odt=2), dict(act=2), dict(act=-1)):
        assert f(**kw) == ERR_FORMAT and r(**kw) == ERR_FORMAT, kw
    for kw in (dict(group=0), dict(group=16), dict(group=48), dict(group=512), dict(group=-32), dict(K=0), dict(K=240),
               dict(K=-256), dict(N=0), dict(N=-64), dict(N=(1 << 30) + 1), dict(K=(1 << 23) + 32), dict(T=0, rows=0),
               dict(T=-1, rows=-1), dict(N=65, act=1), dict(codes=B8), dict(x=B8), dict(scales=B2), dict(y=B2),
               dict(scales=B1, sdt=1), dict(y=B1, odt=1), dict(T=(1 << 24) + 1, rows=(1 << 24) + 1),
               dict(N=1 << 30, K=1 << 12), dict(N=1 << 18, K=1 << 23)):
        assert f(**kw) == ERR_SHAPE, kw
    for kw in (dict(E=2), dict(E=0), dict(k=2), dict(k=0), dict(rows=5), dict(rows=8), dict(rows=0)):
        assert f(**kw) == ERR_SHAPE, kw                      # dense: one matrix, a row each
    for kw in (dict(E=0), dict(E=-1), dict(k=0), dict(k=65), dict(rows=5), dict(rows=0), dict(T=1 << 23, rows=1 << 23, k=4),
               dict(E=1 << 30, N=1 << 12)):
        assert r(**kw) == ERR_SHAPE, kw
    # a grid past the dispatch limit
    assert f(T=1 << 20, rows=1 << 20, N=1 << 20, K=32) == ERR_SHAPE
    assert r(T=1 << 20, rows=1 << 20, N=1 << 10, K=32) == ERR_SHAPE


def test_gate_up_validation(lib):
    order = "x w M N K h odt pre pdt".split()
    f = lambda **kw: _call(lib.moe_gate_up, order, dict(x=A, w=A, M=4, N=32, K=64, h=A, odt=0, pre=None, pdt=0), **kw)  # noqa: E731
    for n in ("x", "w", "h"):
        assert f(**{n: None}) == ERR_NULL, n
    for kw in (dict(odt=2), dict(odt=-1), dict(pre=A, pdt=2)):
        assert f(**kw) == ERR_FORMAT, kw
    for kw in SIZES + [dict(x=B8), dict(w=B8), dict(h=B8), dict(pre=B8)]:
        assert f(**kw) == ERR_SHAPE, kw


SIZES = [dict(M=0), dict(M=-1), dict(M=(1 << 24) + 1), dict(N=0), dict(N=8), dict(N=24), dict(N=-32), dict(K=0),
         dict(K=12), dict(K=-64), dict(N=1 << 22), dict(K=1 << 22), dict(M=1 << 24, N=1 << 16),
         dict(M=1 << 24, K=1 << 16), dict(M=1 << 24, N=1 << 11), dict(N=1 << 21, K=1 << 21)]


def test_gate_up_bwd_validation(lib):
    order = "dh hdt x w pre pdt M N K dx xdt dw wdt ws ws_bytes".split()
    base = dict(dh=A, hdt=0, x=A, w=A, pre=A, pdt=0, M=4, N=32, K=64, dx=A, xdt=0, dw=A, wdt=0, ws=A,
                ws_bytes=ctypes.c_size_t(1 << 60))
    f = lambda **kw: _call(lib.moe_gate_up_bwd, order, base, **kw)  # noqa: E731
    for kw in (dict(dh=None), dict(pre=None), dict(ws=None), dict(dx=None, dw=None), dict(x=None), dict(w=None),
               dict(dx=None, x=None), dict(dw=None, w=None)):
        assert f(**kw) == ERR_NULL, kw
    for kw in (dict(hdt=2), dict(pdt=2), dict(xdt=2), dict(wdt=-1)):
        assert f(**kw) == ERR_FORMAT, kw
    for kw in SIZES + [dict([(n, B8)]) for n in ("dh", "x", "w", "pre", "dx", "dw")]:
        assert f(**kw) == ERR_SHAPE, kw
    # the types of gradients that are not wanted do not matter, their sizes do
    assert f(dx=None, xdt=9, M=0) == ERR_SHAPE
    need = moe.gate_up_bwd_workspace_bytes(4, 32, 64)
    assert need >= 3 * 4 * 32 * 2
    assert f(ws_bytes=ctypes.c_size_t(need - 1)) == ERR_SHAPE
    assert f(ws=ctypes.c_void_p((1 << 30) + 128)) == ERR_SHAPE


def test_workspace_sizes():
    f = moe.gate_up_bwd_workspace_bytes
    for kw in SIZES:
        s = dict(dict(M=4, N=32, K=64), **kw)
        assert f(s["M"], s["N"], s["K"]) == 0, kw
    assert f(4, 32, 64, None, None) == 0 and f(4, 32, 64, 3, None) == 0
    assert f((1 << 32) + 4, 32, 64) == 0
    # d in bf16 where every wanted gradient is bf16, in three parts where one is
    # f32; behind it the shares of a sum, where few tiles have a long one
    assert f(256, 512, 128, None, moe.BF16) >= 256 * 512 * 2
    assert f(256, 512, 128, None, moe.F32) >= 3 * 256 * 512 * 2
    assert f(256, 512, 128, moe.BF16, moe.F32) >= 3 * 256 * 512 * 2
    assert f(4096, 4096, 4096, moe.BF16, moe.BF16) == 4096 * 4096 * 2
    assert f(4096, 4096, 4096, moe.F32, None) == 3 * 4096 * 4096 * 2
    assert f(16, 4096, 4096, moe.BF16, None) >= 16 * 4096 * 2 + 2 * 16 * 4096 * 4


def test_binding_rejects_host_tensors_and_wrong_types():
    u, f, i = torch.zeros((4, 32), dtype=torch.uint8), torch.zeros((4, 2)), torch.zeros((4, 2), dtype=torch.int32)
    b = torch.zeros((4, 64), dtype=torch.bfloat16)
    w = torch.zeros((16, 64), dtype=torch.bfloat16)
    h, p = torch.zeros((4, 8)), torch.zeros((4, 16))
    calls = [lambda: moe.w4_gemv(u, f, b), lambda: moe.w4_gemv(u, f.half(), b), lambda: moe.w4_gemv(u.int(), f, b),
             lambda: moe.w4_gemv(u[None], f[None], b, topk_ids=i), lambda: moe.gate_up(b, w),
             lambda: moe.gate_up(b.float(), w), lambda: moe.gate_up_bwd(h, b, w, p),
             lambda: moe.gate_up_bwd(h.double(), b, w, p)]
    for c in calls:
        with pytest.raises(moe.MoeGmmError):
            c()
