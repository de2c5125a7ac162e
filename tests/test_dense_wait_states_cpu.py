"""The wait states of tests/test_wait_states_cpu.py in the dense block's kernels."""

import os
import subprocess

import pytest

from moe_grouped_gemm_route_amd import build
from tests.test_wait_states_cpu import functions, loads_at_barriers, short_waits


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("asm") / "k.s")
    cmd = [build.hipcc()] + build.FLAGS + ["-x", "hip", "-S", "--cuda-device-only",
                                           os.path.join(build.CSRC, "gateup.hip"), "-o", out]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    assert r.stderr.count("reserved registers") == 0
    with open(out) as f:
        bodies = functions(f.read())
    loads = sum(name is not None and name.startswith("buffer_load") and "lds" in " ".join(ops)
                for b in bodies for _, name, ops in b)
    assert len(bodies) >= 12 and loads > 0
    return bodies


def test_loads_wait_for_their_scalar_operands(kernels):
    early = [(k, " ".join([b[i][1]] + b[i][2])) for k, b in enumerate(kernels) for i in sorted(short_waits(b))]
    assert not early, "%d too early: %s" % (len(early), early[:3])


def test_no_load_is_on_its_way_at_a_barrier(kernels):
    assert sum(name == "s_barrier" for b in kernels for _, name, _ in b) > 0
    assert [(k, i) for k, b in enumerate(kernels) for i in sorted(loads_at_barriers(b))] == []
