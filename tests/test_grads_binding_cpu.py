"""Refusals of the Python binding's newer entry points that need no GPU."""

import pytest
import torch

import moe_grouped_gemm_route_amd as moe


def test_output_types_other_than_f32_and_bf16_are_refused():
    # (called directly: the entry points refuse the host tensors before)
    like = torch.zeros(4)
    for dtype in (torch.float16, torch.float64, torch.int32, 2, -1, "bf16", None):
        with pytest.raises(moe.MoeGmmError):
            moe._out(None, (4,), dtype, "out", like)
    assert moe._out(None, (2, 3), moe.BF16, "out", like).dtype == torch.bfloat16
    assert moe._out(None, (2, 3), torch.float32, "out", like).dtype == torch.float32
