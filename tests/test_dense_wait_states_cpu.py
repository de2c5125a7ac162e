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


def second_barriers(body):
    """Indices of the barriers that some path reaches with a direct-to-LDS load
    on its way that has passed one already."""
    at = {label: i for i, (label, _, _) in enumerate(body) if label}
    seen, work, bad = set(), [(0, -1)], set()
    while work:
        i, passed = work.pop()                     # -1: no load on its way
        if i >= len(body) or (i, passed) in seen:
            continue
        seen.add((i, passed))
        _, name, ops = body[i]
        goes = [i + 1]
        if name:
            text = " ".join(ops)
            if name.startswith("buffer_load") and " lds" in " " + text:
                passed = max(passed, 0)
            elif name == "s_waitcnt" and "vmcnt(0)" in text:
                passed = -1
            elif name == "s_barrier" and passed >= 0:
                if passed:
                    bad.add(i)
                passed = 1
            if name in ("s_endpgm", "s_setpc_b64"):
                goes = []
            elif name == "s_branch":
                goes = [at[ops[0]]]
            elif name.startswith("s_cbranch"):
                goes.append(at[ops[0]])
        work.extend((j, passed) for j in goes)
    return bad


def test_the_check_itself():
    load = "buffer_load_dwordx4 v1, s[20:23], s3 offen lds"
    f = lambda *lines: second_barriers(functions("f:\n" + "\n".join(lines) + "\n.Lfunc_end0:")[0])  # noqa: E731
    assert f(load, "s_barrier", "s_waitcnt vmcnt(0)", "s_barrier", load, "s_barrier") == set()
    assert f(load, "s_barrier", "s_waitcnt vmcnt(1)", "s_barrier") == {4}
    assert f(load, "s_barrier", load, "s_barrier") == {4}
    assert f(".LBB0_1:", "s_barrier", load, "s_cbranch_scc1 .LBB0_1", "s_barrier", "s_barrier", "s_endpgm") == {2, 5, 6}


def test_no_load_is_on_its_way_at_a_barrier_but_where_two_halves_load_in_turns(kernels):
    """A load is waited for in full before the next barrier; in the kernels of
    which half of the waves load a stage, before the one after it."""
    assert sum(name == "s_barrier" for b in kernels for _, name, _ in b) > 0
    assert [(k, i) for k, b in enumerate(kernels) for i in sorted(second_barriers(b))] == []
    uses = [b for b in kernels if any(n and n.startswith("buffer_load") and "lds" in " ".join(o) for _, n, o in b)]
    turns = [b for b in uses if loads_at_barriers(b)]
    assert (len(uses) - len(turns), len(turns)) == (6, 11)
