"""The counted waits of the 8-bit product's pipelines, checked on the compiled gfx950 assembly (host-only).

Each tile kernel brings a stage of codes into LDS with LPW loads a wave and ends it with `s_waitcnt
vmcnt(N)` and a barrier.  Loads complete in issue order, so when the only vector-memory instructions of the
loop are those loads, LPW of them between one barrier and the next, the wait retires every stage but the newest
N / LPW.  Checked: that, with N a whole number of stages as the kernel's template says, and that no kernel uses
scratch memory (whose accesses would be counted, too).
"""

from __future__ import annotations

import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "post_weight_quantization_03_amd", "csrc")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
# template arguments: RB, TB, WA, WB, KS, BUFS, SETS, EARLY
FORM = re.compile(r"k_int8_tileILi(\d+)ELi(\d+)ELi(\d+)ELi(\d+)ELi(\d+)ELi(\d+)ELi(\d+)ELb(\d)E")
VMEM = re.compile(r"^\s*(global_|buffer_|scratch_|flat_)\w+")
LABEL = re.compile(r"^(\.LBB\d+_\d+):")
BRANCH = re.compile(r"^\s*s_cbranch_\w+\s+(\.LBB\d+_\d+)")
WAIT = re.compile(r"^\s*s_waitcnt vmcnt\((\d+)\)")


def asm(src, tmp_path):
    out = tmp_path / (src + ".s")
    cmd = [HIPCC, "--offload-arch=gfx950", "-O3", "-std=c++20", "-fPIC", "-Xclang", "-target-feature", "-Xclang",
           "-packed-fp32-ops", "-I", os.path.join(ROOT, "include"), "--cuda-device-only", "-S",
           os.path.join(CSRC, src), "-o", str(out)]
    r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-3000:]
    return out.read_text()


def kernels(text):
    """kernel symbol -> its lines without comments."""
    out, name = {}, None
    for ln in text.splitlines():
        m = re.match(r"^(_Z\w+):", ln)
        if m:
            name = m.group(1)
            out[name] = []
        elif ln.startswith(".Lfunc_end"):
            name = None
        elif name is not None:
            out[name].append(ln.split(";")[0].rstrip())
    return out


def pipeline_loops(body):
    """The lines of every innermost loop that holds direct loads to LDS and a barrier."""
    at = {m.group(1): i for i, ln in enumerate(body) for m in [LABEL.match(ln)] if m}
    found = []
    for i, ln in enumerate(body):
        m = BRANCH.match(ln)
        if m and at.get(m.group(1), i) < i:
            loop = body[at[m.group(1)]:i]
            if any(" lds" in x for x in loop) and any("s_barrier" in x for x in loop):
                found.append(loop)
    return found


def faults(loop, lpw, outstanding):
    """What the loop does otherwise than LPW loads a stage and a wait for all but `outstanding` stages' loads."""
    found = [ln.strip() for ln in loop if VMEM.match(ln) and not re.match(r"^\s*buffer_load_dwordx4 .* lds$", ln)]
    loads, stages = 0, 0
    for i, ln in enumerate(loop):
        loads += VMEM.match(ln) is not None
        if re.match(r"^\s*s_barrier", ln):
            waits = [WAIT.match(x) for x in loop[max(0, i - 3):i]]
            waits = [int(w.group(1)) for w in waits if w]
            if loads != lpw or waits[-1:] != [outstanding * lpw]:
                found.append(f"{loads} loads, wait {waits}")
            loads, stages = 0, stages + 1
    return found if stages else found + ["no barrier"]


def test_every_stage_is_retired_by_its_count(tmp_path):
    found = {n: b for n, b in kernels(asm("k_int8_tile.hip", tmp_path)).items() if FORM.search(n)}
    assert len(found) == 7
    for name, body in found.items():
        rb, tb, wa, wb, ks, bufs, _, early = (int(x) for x in FORM.search(name).groups())
        lpw = 16 * (rb * wa + tb * wb) * ks // 1024 // (wa * wb)
        loops = pipeline_loops(body)
        assert len(loops) == 1, name
        assert faults(loops[0], lpw, bufs - 2 if early else bufs - 3) == [], name


@pytest.mark.parametrize("src", ["k_int8_tile.hip", "k_int8_rows.hip", "k_int8_tokens.hip", "k_kv_tree.hip"])
def test_no_scratch_memory(src, tmp_path):
    sizes = re.findall(r"; ScratchSize: (\d+)", asm(src, tmp_path))
    assert sizes and set(sizes) == {"0"}


LOOP = """
	buffer_load_dwordx4 v1, s[4:7], 0 offen lds
	buffer_load_dwordx4 v2, s[4:7], 0 offen lds
	s_waitcnt vmcnt(2)
	s_barrier
"""


def test_the_check_tells_faults():
    sound = LOOP.splitlines()
    assert faults(sound, 2, 1) == []
    assert faults(sound, 2, 2) and faults(sound, 3, 1)
    assert faults(sound[:2] + sound[3:], 2, 1)
    assert faults(["	scratch_load_dword v3, off, off"] + sound, 2, 1)
