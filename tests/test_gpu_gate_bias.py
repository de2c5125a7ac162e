"""An expert that the bias alone takes out of the choice: never chosen, yet
part of every softmax (forward, keys and gradient), as include/moe_gmm.h says.
Tolerances as in test_gpu_grads."""

import numpy as np
import pytest
import torch

import moe_grouped_gemm_route_amd as moe
from tests.gpu_util import DEV
from tests.test_gpu_grads import EPS, close, f64, gate_bound

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_bias_takes_experts_out_of_the_choice_and_not_out_of_the_softmax(score, renorm):
    T, E, k, scale = 33, 70, 8, 2.5
    gen = torch.Generator(DEV).manual_seed(70)
    x = torch.randn((T, E), device=DEV, generator=gen)
    out = [2, 5, 69]
    x[:, out] += 3.0                                   # the largest scores, had they no bias
    x[1, 7] = -float("inf")                            # a masked logit adds nothing
    b = torch.randn(E, device=DEV, generator=gen) * 0.1
    b[2], b[5], b[69] = float("nan"), -float("inf"), float("nan")
    code = moe.GATE_SOFTMAX if score == "softmax" else moe.GATE_SIGMOID
    ids, w = moe.topk_gate(x, k, score=code, bias=b, renormalize=renorm, scale=scale)
    # the definition in float64, over all 70 experts
    x64, b64 = f64(x), f64(b)
    p = np.exp(x64) / np.exp(x64).sum(axis=1, keepdims=True) if score == "softmax" else 1 / (1 + np.exp(-x64))
    p[1, 7] = 0.0
    key = np.where(np.isfinite(x64) & np.isfinite(b64), p + b64, -np.inf)
    rid = np.argsort(-key, axis=1, kind="stable")[:, :k]
    assert np.array_equal(ids.cpu().numpy(), rid) and not np.isin(rid, out).any()
    s = np.take_along_axis(p, rid, axis=1)
    rw = scale * (s / s.sum(axis=1, keepdims=True) if renorm else s)
    close(f64(w), rw, gate_bound(x64, rid, rw), torch.float32)
    # the gradient takes no bias: of softmax without renormalisation these
    # experts have one, -p_e sum_i g_i p_i
    g = torch.randn((T, k), device=DEV, generator=gen)
    d = f64(moe.topk_gate_bwd(x, ids, g, score=code, renormalize=renorm, scale=scale))
    if score == "softmax" and not renorm:
        mean = (scale * f64(g) * s).sum(axis=1, keepdims=True)
        size = scale * np.abs(f64(g)).max(axis=1, keepdims=True) * 3
        spread = 2 * np.abs(np.where(np.isfinite(x64), x64, 0)).max(axis=1, keepdims=True)
        close(d[:, out], (-p * mean)[:, out], EPS * (4 * (2 * spread + 4) + 32 + 2 * k) * size, torch.float32)
    else:
        assert not d[:, out].any()
