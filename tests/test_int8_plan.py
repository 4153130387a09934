"""Which kernel a call of the 8-bit product takes (int8_plan.h, compiled with g++), and that the sizes of the GPU
tests reach every kernel with more stages than its buffers hold."""

from __future__ import annotations

import os
import shutil
import subprocess

import pytest

from int8forms import LONG, PIPELINES, random_size
from test_gpu_int8_forms import SEEDS

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "post_weight_quantization_03_amd", "csrc")


@pytest.fixture(scope="module")
def chosen(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ not found")
    exe = tmp_path_factory.mktemp("plan") / "int8_plan"
    subprocess.run([gxx, "-std=c++20", "-O2", "-Wall", "-Werror", "-I", CSRC,
                    os.path.join(ROOT, "tests", "int8_plan_driver.cpp"), "-o", str(exe)], check=True)

    def run(sizes):
        text = "".join(f"{t} {r} {c}\n" for t, r, c in sizes)
        out = subprocess.run([str(exe)], input=text, capture_output=True, text=True, timeout=60, check=True).stdout
        return out.split()
    return run


def test_sizes_take_the_kernel_that_they_are_for(chosen):
    assert dict(zip(LONG, chosen(LONG))) == LONG


def test_every_kernel_is_reached_with_its_ring_going_round():
    for name, (cols, buffers) in PIPELINES.items():
        stages = [-(-c // cols) for (_, _, c), n in LONG.items() if n == name]
        ragged = [c % cols for (_, _, c), n in LONG.items() if n == name]
        assert max(stages) > 3 * buffers and min(stages) > buffers, name
        assert any(ragged), name


def test_the_other_sizes_are_spread_over_the_kernels(chosen):
    names = chosen([random_size(s) for s in SEEDS])
    assert set(names) == set(PIPELINES), names


def test_the_pipelines_are_those_of_the_sources():
    with open(os.path.join(CSRC, "k_int8_tile.hip")) as f:
        source = f.read()
    for name, (cols, buffers) in PIPELINES.items():
        if name != "rows":
            line = next(ln for ln in source.splitlines() if "launch<" in ln and f"T{name}:" in ln or
                        name == "32x16" and "default: return launch<" in ln)
            args = [a.strip() for a in line[line.index("launch<") + 7:line.index(">(")].split(",")]
            rows, tokens = 16 * int(args[0]) * int(args[2]), 16 * int(args[1]) * int(args[3])
            assert f"{rows}x{tokens}" == name and [int(args[4]), int(args[5])] == [cols, buffers]
