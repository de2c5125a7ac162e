"""Calls of the router, the permutation, the activation and the product's
gradient that the binding refuses on the host, before anything is launched."""

import pytest
import torch

import moe_grouped_gemm_route_amd as moe
from tests.gpu_util import DEV

pytestmark = pytest.mark.gpu


def test_output_types_other_than_f32_and_bf16_are_refused():
    x, pr = torch.zeros((4, 8), device=DEV), torch.arange(4, dtype=torch.int32, device=DEV)
    w = torch.ones((4, 1), device=DEV)
    codes = torch.zeros((1, 64, 64), dtype=torch.uint8, device=DEV)
    packed = moe.mxfp4_encode(codes, torch.full((1, 64, 4), 127, dtype=torch.uint8, device=DEV))
    dy, off = torch.zeros((4, 64), dtype=torch.bfloat16, device=DEV), torch.tensor([0, 4], dtype=torch.int32, device=DEV)
    for dtype in (torch.float16, torch.float64, torch.int32, 2, None):
        for call in (lambda: moe.silu_mul(x, out_dtype=dtype), lambda: moe.moe_dispatch_bwd(x, pr, 1, out_dtype=dtype),
                     lambda: moe.moe_combine_bwd(x, x, w, pr, out_dtype=dtype),
                     lambda: moe.moe_gmm_dgrad(packed, moe.MXFP4, 1, 64, 128, dy, off, 4, out_dtype=dtype)):
            with pytest.raises(moe.MoeGmmError):
                call()
    with pytest.raises(moe.MoeGmmError):
        moe.silu_mul(x, out_dtype=torch.float16, out=torch.zeros((4, 4), dtype=torch.float16, device=DEV))
    assert moe.silu_mul(x, out_dtype=torch.bfloat16).dtype == torch.bfloat16


def test_sizes_past_32_bits_are_refused():
    # 2^32 + 8 columns (8 GiB, never touched) are not 8 columns, and 2^32 is not enum 0
    N = (1 << 32) + 8
    x = torch.empty((1, N), dtype=torch.bfloat16, device=DEV)
    pr = torch.zeros(1, dtype=torch.int32, device=DEV)
    w = torch.ones((1, 1), device=DEV)
    logits = torch.zeros((2, 8), device=DEV)
    ids, lw = moe.topk_gate(logits, 2)
    for call in (lambda: moe.moe_dispatch(x, pr, 1), lambda: moe.moe_dispatch_bwd(x, pr, 1, out_dtype=moe.BF16),
                 lambda: moe.moe_combine_bwd(x, x, w, pr, out_dtype=moe.BF16),
                 lambda: moe.silu_mul(x, out_dtype=moe.BF16), lambda: moe.topk_gate(logits, 2, score=1 << 32),
                 lambda: moe.topk_gate_bwd(logits, ids, lw, score=(1 << 32) + 1)):
        with pytest.raises(moe.MoeGmmError):
            call()
