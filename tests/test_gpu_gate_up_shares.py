"""Gradients of the dense block in the instances and shares of a sum that
tests/test_gpu_gate_up_plans.py leaves out (tests/test_dense_plans_cpu.py holds
both files against what the library chooses): the same exact cases.

And its sum over rows past 2^32 bytes, bit for bit.
"""

import pytest
import torch

import moe_grouped_gemm_route_amd as moe
from tests.gpu_util import DEV
from tests.test_gpu_gate_up_plans import inputs, plain

pytestmark = pytest.mark.gpu

F, B = moe.F32, moe.BF16

SHAPES = [(10364, 17680, 136), (6909, 8352, 144), (14843, 144, 4368), (28286, 144, 2088), (2384, 16736, 8),
          (17324, 8160, 144), (8361, 7056, 136), (4449, 11264, 144), (2110, 22320, 136), (72, 3952, 16416),
          (67, 9104, 2064), (8307, 2960, 8), (1117, 5104, 144), (1, 5248, 16488), (1, 480, 4472), (17, 4096, 5120),
          (607, 6528, 3440), (64, 14336, 5120)]


@pytest.mark.parametrize("shape", SHAPES)
def test_every_plan_of_the_gradients(shape):
    dh, x, w, pre = inputs(1, *shape)
    want = plain(dh, x, w, pre)
    for types in ((F, F), (B, B)):
        got = moe.gate_up_bwd(dh, x, w, pre, dx_dtype=types[0], dw_dtype=types[1])
        for a, b in zip(got, want):
            assert torch.equal(a, b.to(a.dtype))


@pytest.mark.parametrize("dw", [F, B])
def test_a_sum_over_rows_past_32_bit_offsets(dw):
    """Exact outright: a gate column's d is a multiple of 1/2 of at most 9, x at
    most 3, so every partial sum is a multiple of 1/2 of at most 27 * 270,017, or
    14.6e6 halves; an up column's d is a multiple of 64 of at most 192, or 2.4e6
    sixty-fours: both below 2^24 of their unit, which f32 holds.  The bf16 result is
    that sum rounded once (every d has at most five bits)."""
    M, N, K = 270_017, 16, 8200
    dh, x, w, pre = inputs(41, M, N, K)
    assert x.numel() * 2 > 1 << 32
    got = moe.gate_up_bwd(dh, x, w, pre, dx_dtype=None, dw_dtype=dw)[1]
    total = torch.zeros((N, K), dtype=torch.float64, device=DEV)
    for a in range(0, M, 4096):
        b = slice(a, a + 4096)
        total += plain(dh[b], x[b], w, pre[b])[1].double()
    assert torch.equal(got, total.float().to(got.dtype)) and torch.equal(total.float().double(), total)
