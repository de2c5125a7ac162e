"""The dense operators as a layer uses them: a training step through routed and
shared experts together, and a decode step of a layer held in 4-bit integers,
each against float64."""

import numpy as np
import pytest
import torch

import moe_grouped_gemm_route_amd as moe
import oracle
from tests.gpu_util import DEV, REL_TOL, to_dev

pytestmark = pytest.mark.gpu


def f64(t):
    return t.double().cpu().numpy()


def norm_err(got, want):
    return float(np.linalg.norm(f64(got) - want) / np.linalg.norm(want))


def test_training_step_of_routed_and_shared_experts():
    """out = sum of the token's routed experts (4-bit, frozen) + the shared
    expert (bf16, trained); the gradients of x and of the shared weights.  Each
    side is computed in f32 from bf16 operands; what the layer rounds to bf16 on
    the way (h, its gradient and the kept sums' gradients) is rounded at most
    2^-8 a value, three times at most on a path: 2-norms within 3 * 2^-8."""
    T, H, I, E, k = 50, 256, 192, 8, 2
    g = torch.Generator().manual_seed(1)
    x = torch.randn((T, H), generator=g).bfloat16().to(DEV)
    logits = torch.randn((T, E), generator=g).to(DEV)
    w13 = (torch.randn((2 * I, H), generator=g) * H ** -0.5).bfloat16().to(DEV)
    w2 = (torch.randn((H, I), generator=g) * I ** -0.5).bfloat16().to(DEV)
    dout = torch.randn((T, H), generator=g).to(DEV)
    rng = np.random.default_rng(2)
    routed = {"fmt": "mxfp4", "codes": rng.integers(0, 256, (E, 2 * H, H // 2), dtype=np.uint8),
              "scales": rng.integers(119, 122, (E, 2 * H, H // 32), dtype=np.uint8)}
    down = {"fmt": "mxfp4", "codes": rng.integers(0, 256, (E, H, H // 2), dtype=np.uint8),
            "scales": rng.integers(119, 122, (E, H, H // 32), dtype=np.uint8)}
    p13, p2 = (moe.mxfp4_encode(to_dev(w["codes"]), to_dev(w["scales"])) for w in (routed, down))

    ids, weights = moe.topk_gate(logits, k)
    r = moe.route_sort(ids, E)
    M = T * k
    sums = moe.moe_gmm(p13, moe.MXFP4, E, 2 * H, H, x, r["group_offsets"], M, row_index=r["sorted_token"])
    hr = moe.silu_mul(sums, out_dtype=moe.BF16)
    y2 = moe.moe_gmm(p2, moe.MXFP4, E, H, H, hr, r["group_offsets"], M)
    h, pre = moe.gate_up(x, w13, out_dtype=moe.BF16, preact_dtype=moe.F32)
    out = moe.moe_combine(y2, weights, r["pair_row"]) + (h.float() @ w2.float().t())

    dy2, _ = moe.moe_combine_bwd(dout, y2, weights, r["pair_row"], out_dtype=moe.BF16)
    ds = moe.moe_gmm_dgrad(p2, moe.MXFP4, E, H, H, dy2, r["group_offsets"], M, out_dtype=moe.BF16,
                           act=moe.ACT_SILU_MUL, preact=sums)
    dxr = moe.moe_dispatch_bwd(moe.moe_gmm_dgrad(p13, moe.MXFP4, E, 2 * H, H, ds, r["group_offsets"], M),
                               r["pair_row"], k)
    dh = dout @ w2.float()
    dxs, dw13 = moe.gate_up_bwd(dh, x, w13, pre)
    dx = dxr + dxs

    # the oracle, in float64 all the way
    ro = oracle.route_sort(ids.cpu().numpy(), E)
    xb = x.view(torch.int16).cpu().numpy().view(np.uint16)
    osums = oracle.gmm(xb, ro["sorted_token"], ro["group_offsets"], routed)
    ohr = oracle.silu_mul(osums)
    W = [oracle.dense_weights(down, e) for e in range(E)]
    off = ro["group_offsets"]
    oy2 = np.concatenate([ohr[off[e]:off[e + 1]] @ W[e].T for e in range(E)])
    oh, opre = oracle.gate_up(f64(x), f64(w13))
    want = oracle.combine(oy2, f64(weights), ro["pair_row"]) + oh @ f64(w2).T
    assert norm_err(out, want) <= 3 * 2.0 ** -8
    ody2, _ = oracle.combine_bwd(f64(dout), oy2, f64(weights), ro["pair_row"])
    ods = oracle.silu_mul_bwd(osums, oracle.gmm_dgrad(ody2, off, down))
    odxr = oracle.dispatch_bwd(oracle.gmm_dgrad(ods, off, routed), ro["pair_row"], k)
    odxs, odw, _ = oracle.gate_up_bwd(f64(dout) @ f64(w2), f64(x), f64(w13), opre)
    assert norm_err(dx, odxr + odxs) <= 3 * 2.0 ** -8
    # the shared expert's own gradients are f32 all the way
    assert np.max(np.abs(f64(dw13) - odw)) <= REL_TOL * np.max(np.abs(odw))
    assert np.max(np.abs(f64(dxs) - odxs)) <= REL_TOL * np.max(np.abs(odxs))


@pytest.mark.parametrize("T", [1, 5])
def test_decode_step_in_4_bit_integers(T):
    """Router, routed experts (two launches, no sort) and the shared expert of a
    few tokens, one of them padding; h is bf16 between the two products (2^-8 a
    value), the rest f32."""
    H, I, E, k, G = 512, 320, 16, 4, 32
    g = torch.Generator().manual_seed(5)

    def weights(lead, K):
        codes = torch.randint(0, 256, lead + (K // 2,), generator=g, dtype=torch.uint8)
        scales = ((0.5 + torch.rand(lead + (K // G,), generator=g)) / (4 * K ** 0.5)).bfloat16()
        zeros = torch.randint(6, 11, lead + (K // G,), generator=g, dtype=torch.uint8)
        return codes.to(DEV), scales.to(DEV), zeros.to(DEV)

    w13, w2, s13, s2 = weights((E, 2 * I), H), weights((E, H), I), weights((2 * I,), H), weights((H,), I)
    x = torch.randn((T, H), generator=g).bfloat16().to(DEV)
    logits = torch.randn((T, E), generator=g).to(DEV)
    if T > 1:
        logits[T - 1] = float("-inf")
    ids, gate = moe.topk_gate(logits, k)
    h = moe.w4_gemv(w13[0], w13[1], x, zeros=w13[2], topk_ids=ids, act=moe.ACT_SILU_MUL, out_dtype=moe.BF16)
    y = moe.w4_gemv(w2[0], w2[1], h, zeros=w2[2], topk_ids=ids, topk_weights=gate)
    hs = moe.w4_gemv(s13[0], s13[1], x, zeros=s13[2], act=moe.ACT_SILU_MUL, out_dtype=moe.BF16)
    y = y + moe.w4_gemv(s2[0], s2[1], hs, zeros=s2[2])

    def host(w):
        return w[0].cpu().numpy(), f64(w[1])

    i, z = ids.cpu().numpy(), lambda w: w[2].cpu().numpy()
    oh = oracle.w4_gemv(*host(w13), f64(x), z(w13), i, act=True)
    want = oracle.w4_gemv(*host(w2), oh, z(w2), i, f64(gate))
    ohs = oracle.w4_gemv(*host(s13), f64(x), z(s13), act=True)
    want = want + oracle.w4_gemv(*host(s2), ohs, z(s2))
    assert norm_err(y, want) <= 2.0 ** -8
    if T > 1:                              # the padding token: the shared expert alone
        assert bool((ids[T - 1] == -1).all())
        assert norm_err(y[T - 1], want[T - 1]) <= 2.0 ** -8
