"""GPU tests of the decode example's block of 8-bit layers: a prompt, trees of drafted tokens and the paths
kept of them, against the same block in fp64 on the dequantized weights with tokens, keys and values kept
exactly.

The two differ by the rounding of tokens (half a step of 1/127 of a token's largest element) and of the cache
(a step of 2^-6 of a block's largest): an output by a few percent; a wrong position, page, head, mask or path
is off by 1.
"""

import os
import sys

import numpy as np
import pytest

from gpuhelp import say, torch_dev
from oracle import attn_ref as R
from oracle import mask_ref as M

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


class Exact:
    """One sequence of the block in fp64."""

    def __init__(self, block):
        f = lambda t: t.double().cpu().numpy()  # noqa: E731
        self.b, self.qkv, self.o = block, f(block.qkv.w_hat), f(block.o.w_hat)
        self.w = [f(t) for t in (block.q_weight, block.k_weight)]
        self.rope = f(block.rope.cos), f(block.rope.sin)
        self.k = self.v = np.zeros((0, block.kv_heads, block.dim))

    def run(self, x, positions, sees, keep=True):
        b, n = self.b, len(x)
        h = (x @ self.qkv.T).reshape(n, -1, b.dim)
        q = R.norm_rope(h[:, :b.q_heads], self.w[0], *self.rope, positions)
        k = R.norm_rope(h[:, b.q_heads:b.q_heads + b.kv_heads], self.w[1], *self.rope, positions)
        k = np.concatenate([self.k, k])
        v = np.concatenate([self.v, h[:, b.q_heads + b.kv_heads:]])
        out = M.attention(q, k, v, b.dim ** -0.5, sees)[0].reshape(n, -1) @ self.o.T
        self.new = k[len(self.k):], v[len(self.v):]
        if keep:
            self.k, self.v = k, v
        return out

    def extend(self, x):
        n, t = len(x), len(self.k) + len(x)
        return self.run(x, np.arange(t - n, t), M.window_sees(n, t, self.b.window, self.b.sinks))

    def draft(self, x, parents, path):
        before = len(self.k)
        at, among = M.tree(parents, before, self.b.window, self.b.sinks)
        out = self.run(x, at, M.tree_sees(at, among, before, self.b.window, self.b.sinks), keep=False)
        self.k, self.v = (np.concatenate([a, b[path]]) for a, b in zip((self.k, self.v), self.new))
        return out


def compare(what, got, want):
    rel = np.linalg.norm(got.double().cpu().numpy() - want) / np.linalg.norm(want)
    say(f"   {what}: {rel:.4f}")
    assert rel < 0.06


@pytest.mark.parametrize("heads", [(4, 4, 64), (8, 2, 128)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (40, 4)])
@pytest.mark.parametrize("prompt", [1, 150])
def test_prompts_trees_and_kept_paths(heads, window, sinks, prompt):
    import decode_attention as E
    torch, dev = torch_dev()
    qh, kh, d = heads
    say(f"draft block, heads {heads} window {window} sinks {sinks} prompt {prompt}")
    block = E.DraftBlock(window, sinks, hidden=256, q_heads=qh, kv_heads=kh, dim=d, block=16, max_tokens=256, batch=2)
    gen = torch.Generator(device=dev).manual_seed(5)
    exact = [Exact(block) for _ in range(2)]
    x = torch.randn((2, prompt, 256), device=dev, generator=gen)
    y = block.extend(x)
    for b in range(2):
        compare(f"prompt {b}", y[b], exact[b].extend(x[b].double().cpu().numpy()))
    rng = np.random.default_rng(6)
    for turn in range(3):
        n = (7, 1, 20)[turn]
        parents = np.array([[rng.integers(-1, i) if i else -1 for i in range(n)] for _ in range(2)])
        paths = []
        for p in parents:  # a deepest token's path, as long in both sequences
            depth = M.tree(p, 0)[0]
            a, path = int(depth.argmax()), []
            while a >= 0:
                path.insert(0, a)
                a = p[a]
            paths.append(path)
        kept = min(len(p) for p in paths)
        paths = np.array([p[:kept] for p in paths])
        x = torch.randn((2, n, 256), device=dev, generator=gen)
        y = block.draft(x, torch.from_numpy(parents.astype(np.int32)).to(dev))
        block.keep(torch.from_numpy(paths).to(dev))
        for b in range(2):
            want = exact[b].draft(x[b].double().cpu().numpy(), parents[b], paths[b])
            compare(f"tree {turn} of {n}, {kept} kept", y[b], want)
    x = torch.randn((2, 3, 256), device=dev, generator=gen)
    y = block.extend(x)
    for b in range(2):
        compare("after the trees", y[b], exact[b].extend(x[b].double().cpu().numpy()))
    assert block.kv_len.tolist() == [len(exact[0].k)] * 2


def test_the_example_runs():
    import decode_attention as E
    E.check_drafts(2, 70, 9, rounds=2)
