"""GPU test of examples/decode_attention.py: a step allocates nothing, as its note says."""

import os
import sys

import pytest

from gpuhelp import torch_dev

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.parametrize("new", [1, 20])
def test_a_step_allocates_nothing(new):
    import decode_attention as E
    torch, dev = torch_dev()
    block = E.AttentionBlock(hidden=256, q_heads=4, kv_heads=2, dim=64, bits=4, block=32, max_tokens=400, batch=2)
    b = block.buffers(2 * new, new)
    x = torch.randn((2 * new, 256), device=dev)
    first = block.step(x, b).clone()  # loads what is loaded once
    block.kv_len.zero_()
    before = torch.cuda.memory_stats(dev)["allocation.all.allocated"]
    y = block.step(x, b)
    assert torch.cuda.memory_stats(dev)["allocation.all.allocated"] == before
    assert b["positions"].tolist() == list(range(new)) * 2
    assert torch.equal(y, first)
