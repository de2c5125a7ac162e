"""topk_gate_bwd against differences of the weights that topk_gate itself
returns.  Tolerances as in test_gpu_grads."""

import itertools

import numpy as np
import pytest
import torch

import moe_grouped_gemm_route_amd as moe
from tests.gpu_util import DEV
from tests.test_gpu_grads import EPS, close, f64, gate_bound

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_gate_gradient_is_the_difference_of_the_gates_own_weights(dtype):
    # topk_gate's f32 weights at x_e +- h.  Logits lie 1/4 apart (exact in
    # bf16, as h is), so the choice and its order stay as they are.  Three
    # errors: the weights' rounding (gate_bound, twice, over 2h); the third
    # order of the difference, h^2 / 6 times the third derivative of sum g w:
    # each weight is, in one logit, an affine function of a logistic one with a
    # factor of at most 1, whose third derivative is at most 1/8; and the
    # gradient's own rounding, in f32 and once to the type.
    T, E, k, h, scale = 6, 12, 3, 2.0 ** -4, 2.5
    rng = np.random.default_rng(3)
    x = torch.from_numpy(np.stack([rng.permutation(E) for _ in range(T)]) * 0.25 - 1.5).to(DEV).to(dtype)
    g = torch.from_numpy(rng.uniform(-0.5, 0.5, size=(T, k))).float().to(DEV)
    total = scale * np.abs(f64(g)).sum(axis=1)
    for code, renorm in itertools.product([moe.GATE_SOFTMAX, moe.GATE_SIGMOID], [True, False]):
        kw = dict(score=code, renormalize=renorm, scale=scale)
        ids, w = moe.topk_gate(x, k, **kw)
        d = f64(moe.topk_gate_bwd(x, ids, g, **kw))
        wtol = gate_bound(f64(x) + np.sign(f64(x)) * h, None, np.full((T, k), scale)).max(axis=1)
        gtol = EPS * (4 * (2 * 4.0 + 4) + 32 + 2 * k) * total * 3
        for e in range(E):
            vals = []
            for s in (h, -h):
                xe = x.clone()
                xe[:, e] += s
                ie, we = moe.topk_gate(xe, k, **kw)
                assert torch.equal(ie, ids)
                vals.append((f64(we) * f64(g)).sum(axis=1))
            tol = 2 * wtol * np.abs(f64(g)).sum(axis=1) / (2 * h) + h * h / 6 / 8 * total + gtol
            close(d[:, e], (vals[0] - vals[1]) / (2 * h), tol, dtype)
