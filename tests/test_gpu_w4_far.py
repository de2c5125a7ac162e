"""moe_w4_gemv where scales and zero points lie past 2^32 bytes and 2^31 entries:
the weights there are told apart from all others."""

import pytest
import torch

import moe_grouped_gemm_route_amd as moe
from tests.gpu_util import DEV

pytestmark = pytest.mark.gpu


def far(E, N, K, G, scale):
    """Codes of 9, zero points of 8 and scales of 1 (weights of 1); in column N - 1
    of the last expert scales of 2, in column N - 2 zero points of 6 (weights of 3),
    in column N - 3 the last group alone: scale 4 and zero point 1 (weights of 32)."""
    codes = torch.empty((E, N, K // 2), dtype=torch.uint8, device=DEV).fill_(0x99)
    scales = torch.ones((E, N, K // G), dtype=scale, device=DEV)
    zeros = torch.empty((E, N, K // G), dtype=torch.uint8, device=DEV).fill_(8)
    scales[E - 1, N - 1] = 2.0
    zeros[E - 1, N - 2] = 6
    scales[E - 1, N - 3, -1] = 4.0
    zeros[E - 1, N - 3, -1] = 1
    return codes, scales, zeros


def rows(T, K):
    """1 at the first k, t + 1 at the last: 2 + t of weights of 1."""
    x = torch.zeros((T, K), dtype=torch.bfloat16, device=DEV)
    t = torch.arange(1, T + 1, device=DEV).float()
    x[:, 0], x[:, K - 1] = 1.0, t.bfloat16()
    return x, t


def check(y, t):
    N = y.shape[-1]
    assert bool((y[:, :N - 3] == (1 + t)[:, None]).all())
    assert torch.equal(y[:, N - 1], 2 + 2 * t) and torch.equal(y[:, N - 2], 3 + 3 * t)
    assert torch.equal(y[:, N - 3], 1 + 32 * t)


@pytest.mark.parametrize("scale", [torch.float32, torch.bfloat16])
def test_scales_and_zero_points_past_32_bits_of_experts(scale):
    E, N, K, G = 3, 262_152, 90_112, 32
    codes, scales, zeros = far(E, N, K, G, scale)
    # the last expert's begin past 2^30 zero points and its columns end past 2^31; its
    # scales begin past 2^31 and end past 2^32 bytes
    assert zeros.numel() > 1 << 31 and scales.numel() * scales.element_size() > 1 << 32
    x, t = rows(2, K)
    ids = torch.full((2, 1), E - 1, dtype=torch.int32, device=DEV)
    check(moe.w4_gemv(codes, scales, x, zeros=zeros, topk_ids=ids), t)
    other = moe.w4_gemv(codes, scales, x, zeros=zeros, topk_ids=ids - 1)
    assert bool((other == (1 + t)[:, None]).all())
    both = torch.tensor([[0, E - 1], [E - 1, 1]], dtype=torch.int32, device=DEV)
    y = moe.w4_gemv(codes, scales, x, zeros=zeros, topk_ids=both, topk_weights=torch.ones((2, 2), device=DEV))
    check(y - (1 + t)[:, None], t)


@pytest.mark.parametrize("T", [1, 3, 9])
def test_scales_and_zero_points_past_32_bits_of_a_matrix(T):
    N, K, G = 1 << 20, 69_632, 32
    codes, scales, zeros = (v[0] for v in far(1, N, K, G, torch.float32))
    assert zeros.numel() > 1 << 31 and scales.numel() * 4 > 1 << 33
    x, t = rows(T, K)
    check(moe.w4_gemv(codes, scales, x, zeros=zeros), t)
