"""The GPU tests of the dense block run every plan (instance and shares of a sum)
that its products take over the sizes below; a change of an estimate that brings
another plan up fails here until a test has it."""

import math
import random

import moe_grouped_gemm_route_amd as moe
from tests.dense_plans import Plans
from tests.test_gpu_gate_up_plans import SHAPES
from tests.test_gpu_gate_up_shares import SHAPES as MORE


def sizes(seed, count):
    rng = random.Random(seed)
    log = lambda lo, hi: int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))  # noqa: E731
    while count:
        M, N, K = log(1, 65536), 16 * log(1, 4096), 8 * log(1, 8192)
        if M * N * K <= 1 << 40:
            count -= 1
            yield M, N, K


def test_the_tables_are_read_as_the_library_has_them():
    """The shares that a plan has show in the workspace that a call needs."""
    p = Plans()
    assert sorted((n, len(t)) for n, t in p.tables.items()) == [
        ("kDw", 3), ("kDw3", 1), ("kDx", 4), ("kDx3", 3), ("kForward", 6)]
    for M, N, K in sizes(1, 300):
        for x, w in ((moe.F32, moe.F32), (moe.BF16, moe.BF16), (moe.F32, None), (None, moe.BF16), (moe.BF16, moe.F32)):
            need = moe.gate_up_bwd_workspace_bytes(M, N, K, x, w)
            assert need > 0
            sums = 0
            if x is not None:
                shares = p.plan("kDx" if x == moe.BF16 else "kDx3", M, K, N)[1]
                sums = shares * M * K * 4 if shares > 1 else 0
            if w is not None:
                shares = p.plan("kDw" if w == moe.BF16 else "kDw3", N, K, M)[1]
                sums = max(sums, shares * N * K * 4 if shares > 1 else 0)
            parts = 3 if moe.F32 in (x, w) else 1
            assert need == -(-parts * M * N * 2 // 256) * 256 + sums, (M, N, K, x, w)


def test_every_plan_is_tested():
    p = Plans()
    tested = set().union(*(p.of(*s) for s in SHAPES + MORE))
    taken = {}
    for s in sizes(2, 12000):
        for plan in p.of(*s):
            taken.setdefault(plan, s)
    assert len(taken) >= 55
    assert {k: v for k, v in taken.items() if k not in tested} == {}
