"""Every kernel that moe_gmm_dgrad chooses from, with and without the
activation's gradient, both output types and both types of the kept sums.
The choice depends on E, K and M; plan() states it, and each test says which
choice it expects.  Tolerances as in test_gpu_grads."""

import numpy as np
import pytest
import torch

import moe_grouped_gemm_route_amd as moe
import oracle
from tests.gpu_util import DEV, bf16_bits_to_f64, to_dev
from tests.test_gpu_grads import BOTH, ENUM, act_bound, bands, close, dgrad_bound, f64, make_weights, random_dy

pytestmark = pytest.mark.gpu


def plan(E, K, M):
    """(16-row subtiles of a tile, k blocks of a wave, groups of waves that
    share n): by the mean band, then by an upper bound of the workgroups."""
    subtiles = 2 if M <= 24 * E else 4 if M < 72 * E else 8
    if subtiles > 2:
        return subtiles, 2, 1
    groups = (M // 32 + min(E, M)) * -(-K // 256)
    if groups * 2 <= 256:
        return 2, 1, 4
    return 2, 2, 4 if groups <= 256 else 2 if groups <= 512 else 1


def check(counts, N, K, fmt, want, seed):
    """All output types, without and with the activation's gradient."""
    E = len(counts)
    off, M = bands(counts, extra=1)
    live = int(off[-1])
    assert plan(E, K, M) == want
    w, packed = make_weights(E, N, K, fmt, seed=seed)
    bits = random_dy(M, N, seed=seed + 1)
    dy64 = bf16_bits_to_f64(bits)
    ref, tol = oracle.gmm_dgrad(dy64, off, w)[:live], dgrad_bound(dy64, off, w, N)[:live]
    enum = moe.MXFP4 if fmt == "mxfp4" else moe.NVFP4
    dy, o = to_dev(bits), to_dev(off)
    for odt in BOTH:
        out = torch.full((M, K), 9.0, device=DEV, dtype=odt)
        moe.moe_gmm_dgrad(packed, enum, E, N, K, dy, o, M, out_dtype=ENUM[odt], out=out)
        close(f64(out)[:live], ref, tol, odt)
        assert bool((out[live:] == 9.0).all())
    gen = torch.Generator(DEV).manual_seed(seed)
    for pdt in BOTH:
        pre = (torch.randn((M, 2 * K), device=DEV, generator=gen) * 2).to(pdt)
        p64 = f64(pre)[:live]
        aref, atol = oracle.silu_mul_bwd(p64, ref), act_bound(tol, ref, p64)
        for odt in BOTH:
            out = torch.full((M, 2 * K), 9.0, device=DEV, dtype=odt)
            moe.moe_gmm_dgrad(packed, enum, E, N, K, dy, o, M, out_dtype=ENUM[odt], act=moe.ACT_SILU_MUL, preact=pre,
                              out=out)
            close(f64(out)[:live], aref, atol, odt)
            assert bool((out[live:] == 9.0).all())


GRIDS = [(6, 896, 2, (2, 1, 4)), (40, 1024, 1, (2, 2, 4)), (30, 896, 7, (2, 2, 4)), (100, 1024, 1, (2, 2, 2)),
         (210, 1024, 1, (2, 2, 1)), (12, 640, 40, (4, 2, 1)), (5, 640, 100, (8, 2, 1))]


# n of one stage (fewer than the groups of waves) and of five (which no group
# count divides)
@pytest.mark.parametrize("E,K,rows,want", GRIDS)
@pytest.mark.parametrize("N", [64, 320])
@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4", "nvfp4_pow2"])
def test_dgrad_every_plan_with_and_without_the_activation(E, K, rows, want, N, fmt):
    # empty bands, bands of one tile and one band of more
    counts = [(rows, 0, 2 * rows, rows)[i % 4] for i in range(E)]
    counts[0] = 3 * rows + 30
    check(counts, N, K, fmt, want, seed=E + K + N)


# bands of `rows` rows under each height of the row tile: every number of
# 16-row subtiles, whole and cut ones, and bands of several tiles
@pytest.mark.parametrize("rows", [1, 16, 17, 32, 33, 48, 49, 64, 65, 80, 81, 96, 97, 112, 113, 128, 129, 255, 257])
@pytest.mark.parametrize("height", [32, 64, 128])
def test_dgrad_every_band_size_under_every_tile(rows, height):
    # empty bands bring the mean band under the height's limit, a long one over it
    if height == 32:
        counts = [rows, 3] + [0] * (rows // 20)
        want = (2, 1, 4)
    elif height == 64:
        counts = [rows, 100] + [0] * (-(-(rows + 100) // 60) - 2)
        want = (4, 2, 1)
    else:
        counts = [rows, 400]
        want = (8, 2, 1)
    for fmt in ("mxfp4", "nvfp4", "nvfp4_pow2"):
        check(counts, 128, 384, fmt, want, seed=rows + height)
