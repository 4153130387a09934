"""The wait states before direct loads to LDS, checked on the compiled gfx950 assembly (host-only).

A direct load takes its place in LDS from M0, and the hardware asks for one wait state between a scalar write
of M0 and a load that uses it; an SGPR written by a vector instruction (v_readfirstlane, a comparison) needs
five before a vector-memory instruction reads it.  The compiler keeps both for the instructions that it emits itself,
but does not look inside inline asm, so a load issued from there has to bring its wait along.  Without it
the load may take the M0 of the load before: its piece then lands in that one's place, and its own place
keeps what an earlier stage left there.

Checked here: in every kernel, on every way that leads to a direct load, that both distances are kept.
"""

from __future__ import annotations

import glob
import os
import re
import subprocess
from concurrent.futures import ThreadPoolExecutor

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "post_weight_quantization_03_amd", "csrc")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
FILES = sorted(glob.glob(os.path.join(CSRC, "k_*.hip")))

DIRECT = re.compile(r"^\s*(global_load_lds_\w+|(?:buffer|global|scratch)_load_\w+ .*\blds\b)")
LABEL = re.compile(r"^(\.LBB\w+):")
BRANCH = re.compile(r"^\s*s_(cbranch_\w+|branch)\s+(\.LBB\w+)")
NOWHERE = re.compile(r"^\s*s_(endpgm|branch|setpc_b64)\b")  # nothing falls through
INSTR = re.compile(r"^\s*([a-z]\w*)\s*(.*)")
M0_STATES, SGPR_STATES = 1, 5


def kernels(text):
    """kernel symbol -> its labels and instructions."""
    out, name = {}, None
    for ln in text.splitlines():
        m = re.match(r"^(_Z\w+):", ln)
        if m:
            name = m.group(1)
            out[name] = []
        elif ln.startswith(".Lfunc_end"):
            name = None
        elif name is not None:
            ln = ln.split(";")[0].rstrip()
            if LABEL.match(ln) or (INSTR.match(ln) and not ln.strip().startswith(".")):
                out[name].append(ln)
    return out


def sgprs(text):
    """Numbers of the scalar registers that a list of operands names (vcc as -2 and -1)."""
    found = set()
    for m in re.finditer(r"\bs\[(\d+):(\d+)\]|\bs(\d+)\b|\b(vcc)\b", text):
        if m.group(4):
            found |= {-2, -1}
        elif m.group(3):
            found.add(int(m.group(3)))
        else:
            found |= set(range(int(m.group(1)), int(m.group(2)) + 1))
    return found


def written(name, operands):
    """(whether M0 is written by a scalar instruction, SGPRs that a vector instruction writes)."""
    outs = operands.split(",")
    if name.startswith("s_"):
        return outs[0].strip() == "m0" and not name.startswith(("s_cmp", "s_bitcmp")), set()
    if name.startswith("v_"):
        # a scalar result comes first, or second as a carry
        regs = sgprs(outs[0]) if not re.match(r"\s*[va]\d|\s*[va]\[", outs[0]) else set()
        if re.match(r"v_(add|sub|subrev|addc|subb|subbrev)_co|v_mad_[ui]64|v_div_scale", name) and len(outs) > 1:
            regs |= sgprs(outs[1])
        return False, regs
    return False, set()


def states(name, operands):
    return int(operands.split()[0], 0) + 1 if name == "s_nop" else 1


def unmet(body):
    """[(line, load, what it is too close to)] of the direct loads that come too early on some way."""
    at = {m.group(1): i for i, ln in enumerate(body) for m in [LABEL.match(ln)] if m}
    sources = {}
    for i, ln in enumerate(body):
        m = BRANCH.match(ln)
        if m:
            sources.setdefault(at[m.group(2)], []).append(i)
    found = set()
    for i, ln in enumerate(body):
        if not DIRECT.match(ln):
            continue
        reads = sgprs(INSTR.match(ln).group(2))
        todo, seen = [(i, 0)], set()  # places that the load is reached from, with the wait states in between
        while todo:
            j, n = todo.pop()
            if (j, n) in seen or n >= SGPR_STATES:
                continue
            seen.add((j, n))
            before = list(sources.get(j, ()))  # what has been executed last: branches to here, the line above
            if j > 0 and LABEL.match(body[j - 1]):
                todo.append((j - 1, n))
            elif j > 0 and not NOWHERE.match(body[j - 1]):
                before.append(j - 1)
            for k in before:
                name, operands = INSTR.match(body[k]).groups()
                m0, regs = written(name, operands)
                if m0 and n < M0_STATES or regs & reads:
                    found.add((i, ln.strip(), body[k].strip()))
                todo.append((k, n + states(name, operands)))
    return sorted(found)


def _asm(src, tmp):
    out = tmp / (os.path.basename(src) + ".s")
    cmd = [HIPCC, "--offload-arch=gfx950", "-O3", "-std=c++20", "-fPIC", "-Xclang", "-target-feature", "-Xclang",
           "-packed-fp32-ops", "-I", os.path.join(ROOT, "include"), "--cuda-device-only", "-S", src, "-o", str(out)]
    r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-3000:]
    return out.read_text()


@pytest.fixture(scope="module")
def assembly(tmp_path_factory):
    tmp = tmp_path_factory.mktemp("asm")
    with ThreadPoolExecutor(max_workers=8) as ex:
        return dict(zip(FILES, ex.map(lambda f: _asm(f, tmp), FILES)))


@pytest.mark.parametrize("src", FILES, ids=os.path.basename)
def test_direct_loads_keep_their_distance(assembly, src):
    bad = {name: f"{len(b)} times, first {b[0]}" for name, body in kernels(assembly[src]).items()
           for b in [unmet(body)] if b}
    assert not bad, bad


def test_the_files_with_direct_loads_are_looked_at(assembly):
    loads = {os.path.basename(f): sum(DIRECT.match(ln) is not None for b in kernels(t).values() for ln in b)
             for f, t in assembly.items()}
    assert {f for f, n in loads.items() if n} == {"k_factor.hip", "k_gemm.hip", "k_hessian.hip", "k_int8_tile.hip",
                                                  "k_quant.hip"}, loads


HEAD = ["	s_mov_b32 s4, 0"] * 6
LOAD = ["	buffer_load_dwordx4 v1, s[4:7], 0 offen lds"]


def test_the_check_tells_faults():
    m0, nop = ["	s_add_i32 m0, s8, 0x400"], ["	s_nop 0"]
    assert unmet(HEAD + LOAD) == []
    assert unmet(HEAD + m0 + nop + LOAD) == []
    assert len(unmet(HEAD + m0 + LOAD)) == 1
    assert len(unmet(HEAD + m0 + ["	global_load_lds_dwordx4 v1, s[2:3]"])) == 1
    # the scalar address, from a vector instruction
    lane = ["	v_readfirstlane_b32 s5, v3"]
    assert len(unmet(HEAD + lane + ["	s_nop 3"] + LOAD)) == 1
    assert unmet(HEAD + lane + ["	s_nop 4"] + LOAD) == []
    assert unmet(HEAD + ["	v_readfirstlane_b32 s9, v3"] + LOAD) == []
    # round a loop, and past a branch
    branch = ["	s_cbranch_scc1 .LBB0_1"]
    assert unmet(HEAD + [".LBB0_1:"] + LOAD + m0 + branch) == []  # the branch is a wait state
    assert len(unmet(HEAD + [".LBB0_1:"] + LOAD + lane + branch)) == 1
    assert len(unmet(HEAD + m0 + [".LBB0_1:"] + LOAD + branch)) == 1
    assert unmet(HEAD + lane + ["	s_branch .LBB0_2", ".LBB0_1:"] + LOAD + [".LBB0_2:"]) == []
