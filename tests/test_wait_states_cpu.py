"""Wait states that the hardware leaves to software, checked in the assembly of
the sources that issue loads as inline assembly (the compiler inserts them for
its own instructions and does not look inside an asm statement; no GPU needed).

gfx950: a vector memory instruction may read a scalar register 5 wait states
after a vector instruction wrote it, and a direct-to-LDS load may follow a
write of M0 after 1.  An instruction is one wait state, s_nop N is N + 1.
"""

import os
import re
import subprocess

import pytest

from moe_grouped_gemm_route_amd import build

VALU_TO_VMEM, M0_TO_LDS_LOAD = 5, 1
TWO_RESULTS = ("v_add_co", "v_sub_co", "v_subrev_co", "v_addc_co", "v_subb_co", "v_subbrev_co", "v_div_scale",
               "v_mad_u64", "v_mad_i64")


def scalars(operand):
    """Scalar registers an operand names."""
    operand = operand.strip().split()[0] if operand.strip() else ""
    if operand in ("vcc", "vcc_lo", "vcc_hi"):
        return {"vcc"}
    if operand == "m0":
        return {"m0"}
    m = re.fullmatch(r"s(\d+)", operand)
    if m:
        return {"s" + m.group(1)}
    m = re.fullmatch(r"s\[(\d+):(\d+)\]", operand)
    return {"s%d" % i for i in range(int(m.group(1)), int(m.group(2)) + 1)} if m else set()


def functions(text):
    """Each function of an assembly listing as [(label, mnemonic, operands)]."""
    out, body = [], []
    for line in text.splitlines():
        line = line.split(";")[0].strip()
        if line.startswith(".Lfunc_end"):
            out.append(body)
            body = []
        elif re.fullmatch(r"[\w.$]+:", line):
            body.append((line[:-1], None, []))
        elif line and not line.startswith("."):
            name, _, rest = line.partition(" ") if " " in line else line.partition("\t")
            body.append((None, name, re.split(r",\s*(?![^\[]*\])", rest.strip()) if rest.strip() else []))
    return out


def short_waits(body):
    """Indices of the vector memory instructions that come too early, over
    every path: per instruction the fewest wait states since each scalar
    register was written, merged where paths meet."""
    at = {label: i for i, (label, _, _) in enumerate(body) if label}
    state, work, bad = {0: {}}, [0], set()
    while work:
        i = work.pop()
        if i >= len(body):
            continue
        label, name, ops = body[i]
        age = dict(state[i])
        goes = [i + 1]
        if name:
            vmem = name.startswith(("buffer_", "global_", "flat_", "scratch_"))
            if vmem:
                read = set().union(*(scalars(o) for o in ops)) if ops else set()
                lds_load = " lds" in " " + " ".join(ops)
                if any(age.get(("valu", s), VALU_TO_VMEM) < VALU_TO_VMEM for s in read):
                    bad.add(i)
                if lds_load and age.get(("m0",), M0_TO_LDS_LOAD) < M0_TO_LDS_LOAD:
                    bad.add(i)
            wait = int(ops[0], 0) + 1 if name == "s_nop" else 1
            age = {k: v + wait for k, v in age.items() if v + wait < VALU_TO_VMEM}
            if name.startswith("v_") and ops:
                written = scalars(ops[0])
                if name.startswith(TWO_RESULTS) and len(ops) > 1:
                    written |= scalars(ops[1])
                age.update({("valu", s): 0 for s in written})
            elif name.startswith("s_") and ops and not name.startswith(("s_nop", "s_cmp", "s_bitcmp", "s_waitcnt")):
                for s in scalars(ops[0]):
                    age.pop(("valu", s), None)          # a scalar write is waited for by the hardware
                    if s == "m0":
                        age[("m0",)] = 0
            if name in ("s_endpgm", "s_setpc_b64"):
                goes = []
            elif name == "s_branch":
                goes = [at[ops[0]]]
            elif name.startswith("s_cbranch"):
                goes.append(at[ops[0]])
        for j in goes:
            old = state.get(j)
            new = dict(age) if old is None else {k: min(old.get(k, 99), age.get(k, 99)) for k in old.keys() | age.keys()}
            if new != old:
                state[j] = new
                work.append(j)
    return bad


def test_the_check_itself():
    def run(*lines):
        return short_waits(functions("f:\n" + "\n".join(lines) + "\n.Lfunc_end0:")[0])

    load = "buffer_load_dwordx4 v1, s[20:23], s3 offen lds"
    first = ["v_readfirstlane_b32 s21, v0", "s_mov_b32 m0, s4"]
    assert run(*first, "s_nop 0", load) == {4}
    assert run(*first, "s_nop 2", load) == {4} and run(*first, "s_nop 3", load) == set()
    assert run("s_mov_b32 m0, s4", load) == {2} and run("s_mov_b32 m0, s4", "s_nop 0", load) == set()
    fly = functions("f:\n" + load + "\ns_waitcnt vmcnt(1)\ns_barrier\ns_waitcnt vmcnt(0)\ns_barrier\n.Lfunc_end0:")[0]
    assert loads_at_barriers(fly) == {3}
    assert run("v_cmp_eq_u32_e64 s[2:3], v0, v1", "s_nop 3", load) == {3}
    # around a loop: the write stands behind the load
    assert run(".LBB0_1:", load, "v_readfirstlane_b32 s20, v0", "s_cbranch_scc1 .LBB0_1", "s_endpgm") == {2}
    # a scalar write of the register is another value, which the hardware waits for
    assert run("v_readfirstlane_b32 s21, v0", "s_mov_b32 s21, s9", "s_mov_b32 m0, s4", "s_nop 0", load) == set()


def loads_at_barriers(body):
    """Indices of the barriers that some path reaches with a direct-to-LDS load
    on its way: one after which no s_waitcnt vmcnt(0) has come."""
    at = {label: i for i, (label, _, _) in enumerate(body) if label}
    seen, work, bad = set(), [(0, False)], set()
    while work:
        i, flying = work.pop()
        if i >= len(body) or (i, flying) in seen:
            continue
        seen.add((i, flying))
        label, name, ops = body[i]
        goes = [i + 1]
        if name:
            text = " ".join(ops)
            if name.startswith("buffer_load") and " lds" in " " + text:
                flying = True
            elif name == "s_waitcnt" and "vmcnt(0)" in text:
                flying = False
            elif name == "s_barrier" and flying:
                bad.add(i)
            if name in ("s_endpgm", "s_setpc_b64"):
                goes = []
            elif name == "s_branch":
                goes = [at[ops[0]]]
            elif name.startswith("s_cbranch"):
                goes.append(at[ops[0]])
        work.extend((j, flying) for j in goes)
    return bad


@pytest.fixture(scope="module", params=["dgrad.hip"])
def kernels(request, tmp_path_factory):
    """The functions of a source as the build compiles it."""
    out = str(tmp_path_factory.mktemp("asm") / "k.s")
    cmd = [build.hipcc()] + build.FLAGS + ["-x", "hip", "-S", "--cuda-device-only",
                                           os.path.join(build.CSRC, request.param), "-o", out]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    # M0 in a clobber list is a register that the compiler does not promise to keep
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
