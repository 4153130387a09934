"""GPU test of examples/decode_attention.py: a packed attention block over a prompt and a few decode
steps, against the same block in fp64 on the dequantized weights with keys and values kept exactly.

The two differ by the cache's rounding alone: a stored element is off by at most one step, 2^-6 of
its block's largest, so an output by a few percent; a wrong position, page, head or mask is off by 1.
"""

import os
import sys

import numpy as np
import pytest

from gpuhelp import say, torch_dev
from oracle import attn_ref as R

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def _reference(block, prompt, steps):
    f = lambda t: t.double().cpu().numpy()  # noqa: E731
    qkv, o = f(block.qkv.w_hat), f(block.o.w_hat)
    qw, kw, cos, sin = (f(t) for t in (block.q_weight, block.k_weight, block.rope.cos, block.rope.sin))
    qh, kh, d = block.q_heads, block.kv_heads, block.dim
    outs = []
    for b in range(prompt.shape[0]):
        x, keys, vals, got = f(prompt[b]), np.zeros((0, kh, d)), np.zeros((0, kh, d)), []
        for _ in range(steps + 1):
            pos = np.arange(len(keys), len(keys) + len(x))
            h = (x @ qkv.T).reshape(len(x), -1, d)
            q = R.norm_rope(h[:, :qh], qw, cos, sin, pos)
            keys = np.concatenate([keys, R.norm_rope(h[:, qh:qh + kh], kw, cos, sin, pos)])
            vals = np.concatenate([vals, h[:, qh + kh:]])
            y = R.attention(q, keys, vals, d ** -0.5)[0].reshape(len(x), -1) @ o.T
            got.append(y)
            x = y[-1:]
        outs.append(got)
    return outs


@pytest.mark.parametrize("heads", [(4, 4, 64), (8, 2, 128)])
def test_decode_against_the_block_in_64_bits(heads):
    import decode_attention as E
    torch, dev = torch_dev()
    qh, kh, d = heads
    say(f"decode example, heads {heads}")
    block = E.AttentionBlock(hidden=256, q_heads=qh, kv_heads=kh, dim=d, bits=8, block=16, max_tokens=64, batch=3)
    prompt = torch.randn((3, 37, 256), device=dev, generator=torch.Generator(device=dev).manual_seed(5))
    want = _reference(block, prompt, 4)
    first, outs = E.decode(block, prompt, 4)
    assert block.kv_len.tolist() == [41] * 3
    for b in range(3):
        e = first[b].double().cpu().numpy() - want[b][0]
        rel = np.linalg.norm(e) / np.linalg.norm(want[b][0])
        say(f"   prompt {b}: {rel:.4f}")
        assert rel < 0.03
        for s in range(4):
            e = outs[s, b].double().cpu().numpy() - want[b][s + 1][0]
            rel = np.linalg.norm(e) / np.linalg.norm(want[b][s + 1])
            say(f"   step {s}: {rel:.4f}")
            assert rel < 0.1  # the steps feed their own error back


def test_replayed_steps_equal_eager_steps():
    import decode_attention as E
    torch, dev = torch_dev()
    block = E.AttentionBlock(hidden=256, q_heads=4, kv_heads=2, dim=64, bits=4, block=32, max_tokens=400, batch=2)
    prompt = torch.randn((2, 300, 256), device=dev)
    a = E.decode(block, prompt, 6, graph=False)
    block.kv_len.zero_()
    b = E.decode(block, prompt, 6, graph=True)
    assert torch.equal(a[0], b[0])
    # the recorded step runs once before it is recorded: it may grow a block's scale before its time
    assert float((a[1] - b[1]).norm() / a[1].norm()) < 0.02
