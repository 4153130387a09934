"""Scratch memory of the attention kernels, on the compiled gfx950 assembly (host-only): no form holds more than it did
when it was measured, and those that held none hold none."""

from __future__ import annotations

import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "post_weight_quantization_03_amd", "csrc")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
# kernel, (dim, bf16, waves or row tiles, masked) -> bytes a lane
HELD = {("k_kv_rows", 128, 1, 2, 1): 56, ("k_kv_prompt", 128, 0, 8, 0): 68, ("k_kv_prompt", 128, 0, 8, 1): 68,
        ("k_kv_prompt", 128, 1, 4, 0): 20, ("k_kv_prompt", 128, 1, 4, 1): 40, ("k_kv_prompt", 256, 1, 4, 0): 116,
        ("k_kv_prompt", 256, 1, 4, 1): 116, ("k_kv_prompt", 256, 0, 4, 0): 452, ("k_kv_prompt", 256, 0, 4, 1): 388}


@pytest.mark.parametrize("kernel,forms", [("k_kv_rows", 18), ("k_kv_prompt", 14)])
def test_scratch_is_bounded(kernel, forms, tmp_path):
    out = tmp_path / "k.s"
    cmd = [HIPCC, "--offload-arch=gfx950", "-O3", "-std=c++20", "-fPIC", "-Xclang", "-target-feature", "-Xclang",
           "-packed-fp32-ops", "-I", os.path.join(ROOT, "include"), "--cuda-device-only", "-S",
           os.path.join(CSRC, kernel + ".hip"), "-o", str(out)]
    r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-3000:]
    seen = 0
    for name, size in re.findall(r"\.amdhsa_kernel (\S+).*?\.amdhsa_private_segment_fixed_size (\d+)", out.read_text(),
                                 re.S):
        m = re.search(kernel + r"ILi(\d+)ELb(\d)ELi(\d)ELb(\d)E", name)
        form = (kernel, *map(int, m.groups())) if m else None
        seen += m is not None
        assert int(size) <= HELD.get(form, 0), (name, size)
    assert seen == forms
