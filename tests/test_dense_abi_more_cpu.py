"""Argument checks of the dense operators beside tests/test_dense_abi_cpu.py (no
GPU needed: every call here is rejected before any HIP call)."""

import ctypes

import pytest
import torch

import moe_grouped_gemm_route_amd as moe
from tests.test_grads_abi_cpu import A, ERR_SHAPE, _call


@pytest.mark.parametrize("off", [1, 2, 3])
def test_w4_ids_and_weights_lie_at_whole_words(off):
    """They are read by scalar loads, which leave out the low two bits of an
    address: a call with others would take the entries before."""
    order = "codes scales sdt zeros group E N K x rows T ids w k y odt act".split()
    base = dict(codes=A, scales=A, sdt=0, zeros=None, group=32, E=8, N=64, K=256, x=A, rows=4, T=4, ids=A, w=A, k=2,
                y=A, odt=0, act=0)
    odd = ctypes.c_void_p((1 << 30) + off)
    f = moe.library().moe_w4_gemv
    assert _call(f, order, base, ids=odd) == ERR_SHAPE
    assert _call(f, order, base, w=odd) == ERR_SHAPE
    assert _call(f, order, base, ids=odd, w=None) == ERR_SHAPE


def test_workspace_bytes_take_the_types_that_the_gradients_take():
    """F32 and BF16 or their torch types, as gate_up_bwd's dx_dtype and dw_dtype."""
    f = moe.gate_up_bwd_workspace_bytes
    both = {moe.F32: torch.float32, moe.BF16: torch.bfloat16, None: None}
    for x in both:
        for w in both:
            assert f(100, 512, 256, both[x], both[w]) == f(100, 512, 256, x, w)
            assert f(100, 512, 256, both[x], w) == f(100, 512, 256, x, w)
    assert f(100, 512, 256, torch.bfloat16, None) > 0
    assert f(100, 512, 256, torch.float16, None) == 0 and f(100, 512, 256, None, torch.int32) == 0
    assert f(100, 512, 256, torch.float16, moe.F32) == 0
