"""What a bf16 gradient of the dense block rounds: d once, as the product's
operand, and the result once; an f32 gradient rounds neither.

Gates of 0 and 64, where the sigmoid is 1/2 and 1, make d exact in f32 (16 bits:
products of two bf16 values and of powers of two), so its rounding to bf16 is
known to the bit.  Against that product in float64 a bf16 result is off by half a
step (2^-8 of the value) and by the f32 sum's own error, for which the suite
allows 1e-5 of the largest result.
"""

import numpy as np
import pytest
import torch

import moe_grouped_gemm_route_amd as moe
from tests.gpu_util import DEV, REL_TOL

pytestmark = pytest.mark.gpu

F, B = moe.F32, moe.BF16


def near(got, want, half):
    assert np.all(np.abs(got.double().cpu().numpy() - want) <= half * np.abs(want) + REL_TOL * np.max(np.abs(want)))


# bf16 plans of one share and of several, in tiles of 64 to 256 rows
@pytest.mark.parametrize("shape", [(1, 480, 4112), (64, 512, 320), (300, 272, 1416), (969, 144, 264), (1237, 2832, 2560)])
def test_bf16_gradients_round_d_once_and_f32_ones_do_not(shape):
    M, N, K = shape
    g = torch.Generator().manual_seed(1)
    n = lambda *s: torch.randn(s, generator=g).bfloat16()  # noqa: E731
    dh, x, w, u = n(M, N // 2), n(M, K), n(N, K), n(M, N // 2)
    on = torch.rand((M, N // 2), generator=g) > 0.5
    pre = torch.cat((torch.where(on, 64.0, 0.0).bfloat16(), u), 1)
    e = dh.double()
    d = torch.cat((torch.where(on, e * u, e * u / 2), torch.where(on, e * 64, 0.0)), 1)
    assert torch.equal(d.float().double(), d)
    rounded = d.float().bfloat16().double()
    assert not torch.equal(rounded, d)
    args = [t.to(DEV) for t in (dh, x, w, pre)]
    bx, bw = moe.gate_up_bwd(*args, dx_dtype=B, dw_dtype=B)
    near(bx, (rounded @ w.double()).numpy(), 2.0 ** -8)
    near(bw, (rounded.t() @ x.double()).numpy(), 2.0 ** -8)
    fx, fw = moe.gate_up_bwd(*args)
    wx, ww = (d @ w.double()).numpy(), (d.t() @ x.double()).numpy()
    near(fx, wx, 0.0)
    near(fw, ww, 0.0)
    # a bf16 gradient of the whole d: the f32 one, rounded
    near(fx.bfloat16(), wx, 2.0 ** -8)
    near(fw.bfloat16(), ww, 2.0 ** -8)
    # beside the other gradient in f32 a bf16 one has the same bits
    assert torch.equal(moe.gate_up_bwd(*args, dx_dtype=B, dw_dtype=F)[0], bx)
    assert torch.equal(moe.gate_up_bwd(*args, dx_dtype=F, dw_dtype=B)[1], bw)
