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


def test_whole_numbers_past_32_bits_are_refused():
    # ctypes would pass their low 32 bits on: 2^32 + 8 columns as 8
    called = []
    for bad in ((1 << 32) + 8, 1 << 31, -(1 << 31) - 1, 1 << 40):
        with pytest.raises(moe.MoeGmmError):
            moe._launch(lambda *a: called.append(a), (torch.zeros(1),), 4, bad, None, 1.0)
    assert not called
    for fmt, E, N, K in ((moe.MXFP4, (1 << 32) + 1, 64, 128), (moe.MXFP4, 1, (1 << 32) + 64, 128),
                         (moe.MXFP4, 1, 64, (1 << 32) + 128), (1 << 32, 1, 64, 128)):
        with pytest.raises(moe.MoeGmmError):
            moe.packed_weight_bytes(fmt, E, N, K)
    assert moe.packed_weight_bytes(moe.MXFP4, 1, 64, 128) > 0
