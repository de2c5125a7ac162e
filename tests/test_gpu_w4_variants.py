"""moe_w4_gemv with the activation and with weighted sums in every kernel that
such calls take: with and without zero points, both scale types, blocks of two
and of four tiles, 16 rows a block under narrow groups, workgroups that walk
several blocks of columns and several units of k.  Against the float64 oracle:
f32 results to the suite's max|delta| / max|ref| <= 1e-5, bf16 ones to half a
step (2^-8 of the value) beside that.
"""

import numpy as np
import pytest
import torch

import moe_grouped_gemm_route_amd as moe
from tests.test_gpu_w4 import BAD, check as near, dev, ids_of, problem, ref, run

pytestmark = pytest.mark.gpu

KINDS = [(zeros, scale) for zeros in (False, True) for scale in (torch.float32, torch.bfloat16)]


# T, N, K, G of dense products.  Row blocks are 16 G / 128 rows (at most 16): four
# tiles a block from N / 64 * row blocks = 256 on, several blocks a workgroup past
# 256 blocks of 32 columns of y (of 16 with two tiles).
DENSE = [(1, 48, 160, 32), (1, 64, 512, 128), (1, 16500, 96, 32), (1, 98, 4672, 64),           # one row
         (2, 66, 160, 32), (7, 50, 320, 64), (16, 34, 384, 128), (30, 40, 256, 256),           # two tiles
         (3, 9002, 64, 64), (2, 70, 4736, 128),                                                # longer
         (2, 33002, 96, 32), (5, 33010, 160, 32), (3, 34002, 192, 64), (4, 33000, 128, 128),   # four tiles
         (70, 4102, 256, 128), (33, 8194, 256, 256), (2, 16386, 4736, 128),
         (20, 8200, 96, 32), (61, 66, 4640, 32),                                               # 16 rows, G 32
         (60, 1026, 448, 64), (40, 8202, 192, 64), (33, 40, 4352, 64)]                         # 16 rows, G 64


@pytest.mark.parametrize("case", DENSE)
@pytest.mark.parametrize("zeros,scale", KINDS)
def test_activation_of_dense_products(case, zeros, scale):
    T, N, K, G = case
    p = problem(1, N, K, G, rows=T, scale=scale, zeros=zeros)
    want = ref(p, act=True)
    assert want.shape == (T, N // 2)
    near(run(p, act=moe.ACT_SILU_MUL), want, moe.F32)
    near(run(p, act=moe.ACT_SILU_MUL, out_dtype=moe.BF16), want, moe.BF16)


# Every kernel of two rows and more: 1, 2 and 4 scale groups a chunk, two and four
# tiles a block, rows of the operand apart or 16 a block, and runs of scales that
# are whole chunks (K a multiple of 128, G below) or end inside one.
EVERY = [(2, 66, 384, 128), (2, 16450, 256, 128),
         (5, 70, 256, 64), (5, 70, 192, 64), (4, 16402, 128, 64), (4, 16402, 192, 64),
         (60, 70, 256, 64), (60, 70, 192, 64), (40, 8202, 128, 64), (40, 8202, 192, 64),
         (3, 66, 256, 32), (3, 66, 160, 32), (3, 16402, 128, 32), (3, 16402, 96, 32),
         (30, 66, 256, 32), (30, 66, 160, 32)]


@pytest.mark.parametrize("case", EVERY)
@pytest.mark.parametrize("zeros,scale", KINDS)
def test_every_kernel_of_dense_rows(case, zeros, scale):
    """Without the activation exactly: integers times powers of two."""
    T, N, K, G = case
    p = problem(10, N, K, G, rows=T, scale=scale, zeros=zeros, exact=True)
    assert np.array_equal(run(p).double().cpu().numpy(), ref(p))
    p = problem(11, N, K, G, rows=T, scale=scale, zeros=zeros)
    near(run(p, act=moe.ACT_SILU_MUL), ref(p, act=True), moe.F32)


# T, k, E, N, K, G of routed ones: several blocks a workgroup where 16 columns of y
# times pairs pass 512 (summed: 32 columns times tokens)
ROUTED = [(1, 6, 8, 96, 416, 32), (8, 6, 5, 2100, 96, 32), (3, 4, 4, 1500, 4352, 64), (6, 2, 3, 5000, 256, 128),
          (2, 3, 4, 70, 8704, 256)]


@pytest.mark.parametrize("case", ROUTED)
@pytest.mark.parametrize("zeros,scale", KINDS)
def test_activation_of_chosen_experts(case, zeros, scale):
    T, k, E, N, K, G = case
    p = problem(2, N, K, G, E=E, rows=T, scale=scale, zeros=zeros)
    ids = ids_of(3, T, k, E, BAD[:2])
    want = ref(p, topk_ids=ids.numpy(), act=True)
    assert want.shape == (T * k, N // 2)
    near(run(p, topk_ids=dev(ids), act=moe.ACT_SILU_MUL), want, moe.F32)


SUMMED = [(1, 6, 8, 50, 416, 32), (8, 6, 5, 2100, 96, 32), (5, 3, 4, 3400, 4352, 128), (9, 4, 3, 2050, 192, 64),
          (2, 40, 4, 70, 768, 256)]


@pytest.mark.parametrize("case", SUMMED)
@pytest.mark.parametrize("zeros,scale", KINDS)
@pytest.mark.parametrize("per_pair", [False, True])
def test_weighted_sums_of_chosen_experts(case, zeros, scale, per_pair):
    T, k, E, N, K, G = case
    p = problem(4, N, K, G, E=E, rows=T * k if per_pair else T, scale=scale, zeros=zeros)
    ids = ids_of(5, T, k, E, BAD[:2])
    w = torch.softmax(torch.randn((T, k), generator=torch.Generator().manual_seed(6)), 1)
    want = ref(p, topk_ids=ids.numpy(), topk_weights=w.numpy())
    near(run(p, topk_ids=dev(ids), topk_weights=dev(w)), want, moe.F32)
    if not per_pair:
        near(run(p, topk_ids=dev(ids), topk_weights=dev(w), out_dtype=moe.BF16), want, moe.BF16)


def test_equal_calls_give_equal_bits():
    p = problem(7, 16386, 1056, 32, rows=3, scale=torch.bfloat16)
    first = run(p, act=moe.ACT_SILU_MUL)
    assert all(torch.equal(first, run(p, act=moe.ACT_SILU_MUL)) for _ in range(4))
    p = problem(8, 2100, 1056, 32, E=5, rows=8)
    ids, w = dev(ids_of(9, 8, 6, 5)), torch.rand((8, 6), device="cuda")
    first = run(p, topk_ids=ids, topk_weights=w)
    assert np.isfinite(first.cpu().numpy()).all()
    assert all(torch.equal(first, run(p, topk_ids=ids, topk_weights=w)) for _ in range(4))
