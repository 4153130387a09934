"""Greedy decoding steps of one attention block whose projections are packed by GPTQ and whose
keys and values live in a paged 8-bit cache.

    python examples/decode_attention.py [--batch 4] [--prompt 600] [--steps 8] [--bits 4] [--drafts 0]

A block of Llama-2-7B's attention shape unless told otherwise (hidden 4096, 32 heads of 128), with
random weights: q, k, v and o are quantized, packed and served by gptq_dequant_gemm; every query and
key head goes through an RMS norm and the position rotation; a prompt fills the cache, then each step
feeds the block's output back as the next token's input.  Each step is seven calls on one stream, with
nothing allocated inside, recorded once as a HIP graph and replayed.

``DraftBlock`` is the same block of 8-bit layers with one scale a row, for many tokens at a time: prompts and
trees of drafted tokens go through the 8-bit integer product and see a window of the cache and its first
tokens; of a tree, the tokens that are kept are stored again in their places.
"""

from __future__ import annotations

import argparse
import math
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import post_weight_quantization_03_amd as g  # noqa: E402


class PackedLinear:
    """A linear layer quantized against H = I and packed; serves fp32 outputs."""

    def __init__(self, W, bits, groupsize=128):
        rows, cols = W.shape
        H = torch.eye(cols, device=W.device)
        out = g.quantize(W, H, g.Params(bits=bits, groupsize=groupsize))
        self.packed = torch.empty((rows, cols * bits // 32), dtype=torch.int32, device=W.device)
        g.gptq_pack(out["codes"], bits, self.packed)
        self.scales, self.zeros, self.w_hat = out["scales"], out["zeros"], out["w_hat"]
        self.bits, self.groupsize = bits, groupsize

    def __call__(self, X, Y, workspace):
        return g.gptq_dequant_gemm(self.packed, self.scales, self.zeros, self.bits, self.groupsize, X, Y,
                                   workspace=workspace)

    def workspace_bytes(self, batch):
        return g.gptq_dequant_gemm_workspace_bytes(self.w_hat.shape[0], self.w_hat.shape[1], self.bits,
                                                   self.groupsize, batch)


class AttentionBlock:
    """q, k, v in one packed projection, norm and rotation, the cache, attention, the output projection."""

    def __init__(self, hidden=4096, q_heads=32, kv_heads=32, dim=128, bits=4, block=64, max_tokens=4096, batch=4,
                 device="cuda:0", seed=0, groupsize=128):
        gen = torch.Generator(device=device).manual_seed(seed)

        def weight(rows, cols):
            return torch.randn((rows, cols), generator=gen, device=device) / math.sqrt(cols)

        self.hidden, self.q_heads, self.kv_heads, self.dim, self.batch = hidden, q_heads, kv_heads, dim, batch
        self.qkv = PackedLinear(weight((q_heads + 2 * kv_heads) * dim, hidden), bits, groupsize)
        self.o = PackedLinear(weight(hidden, q_heads * dim), bits, groupsize)
        self.q_weight = 1.0 + 0.1 * torch.randn(dim, generator=gen, device=device)
        self.k_weight = 1.0 + 0.1 * torch.randn(dim, generator=gen, device=device)
        inv = 10000.0 ** (-torch.arange(0, dim, 2, device=device, dtype=torch.float64) / dim)
        angle = torch.arange(max_tokens, device=device, dtype=torch.float64)[:, None] * inv
        self.rope = g.Rope(angle.cos().float().contiguous(), angle.sin().float().contiguous())
        blocks = -(-max_tokens // block)
        self.cache = g.KVCache.empty(batch * blocks, kv_heads, block, dim, device)
        # pages as an allocator would hand them out: in no order
        self.table = torch.randperm(batch * blocks, generator=gen, device=device).to(torch.int32).view(batch, blocks)
        self.kv_len = torch.zeros(batch, dtype=torch.int32, device=device)
        self.max_tokens, self.device = max_tokens, device

    def buffers(self, rows, new):
        """What calls of `new` tokens a sequence write to and work in."""
        h, t = self.q_heads + 2 * self.kv_heads, torch.float32
        start = torch.arange(0, rows + 1, new, dtype=torch.int32, device=self.device)
        plan = g.KVBatch(start, self.kv_len, self.table, rows, new, self.max_tokens)
        need = max(self.qkv.workspace_bytes(rows), self.o.workspace_bytes(rows),
                   g.gptq_kv_attention_workspace_bytes(self.cache, plan, self.q_heads, g.GPTQ_F32))
        return {"plan": plan, "new": new, "qkv": torch.empty((rows, h, self.dim), dtype=t, device=self.device),
                "attended": torch.empty((rows, self.q_heads, self.dim), dtype=t, device=self.device),
                "y": torch.empty((rows, self.hidden), dtype=t, device=self.device),
                "positions": torch.empty(rows, dtype=torch.int32, device=self.device),
                "offsets": torch.arange(-new, 0, dtype=torch.int32, device=self.device),  # from a sequence's end
                "workspace": torch.empty(max(need, 1), dtype=torch.uint8, device=self.device)}

    def step(self, x, b):
        """Output [rows, hidden] of the block for the next tokens x [rows, hidden] of every sequence."""
        rows, new = x.shape[0], b["new"]
        self.kv_len += new
        torch.add(self.kv_len[:, None], b["offsets"], out=b["positions"].view(-1, new))
        q, k, v = b["qkv"].split([self.q_heads, self.kv_heads, self.kv_heads], 1)
        self.qkv(x, b["qkv"].view(rows, -1), b["workspace"])
        g.gptq_qk_norm_rope(q, None, b["positions"], self.rope, self.q_weight, q_out=q)
        g.gptq_kv_append(self.cache, b["plan"], k, v, self.rope, self.k_weight)
        g.gptq_kv_attention(q, self.cache, b["plan"], out=b["attended"], workspace=b["workspace"])
        return self.o(b["attended"].view(rows, -1), b["y"], b["workspace"])


class DraftBlock(AttentionBlock):
    """The block with 8-bit layers of one scale a row, tokens rounded to 8 bits, and attention limited to the
    last `window` tokens and the first `sinks`."""

    def __init__(self, window=0, sinks=0, **sizes):
        super().__init__(bits=8, groupsize=-1, **sizes)
        self.window, self.sinks = window, sinks

    def _project(self, layer, x, dtype=torch.float32):
        return g.gptq_int8_gemm(layer.packed, layer.scales, layer.zeros, g.gptq_quantize_tokens(x), dtype=dtype)

    def _plan(self, rows, new):
        start = torch.arange(0, rows + 1, new, dtype=torch.int32, device=self.device)
        return g.KVBatch(start, self.kv_len, self.table, rows, new, self.max_tokens)

    def _attend(self, x, plan, positions, tree=None):
        """Outputs of x at its positions, with its keys and values in the cache, and these."""
        q, k, v = self._project(self.qkv, x).view(len(x), -1, self.dim).split(
            [self.q_heads, self.kv_heads, self.kv_heads], 1)
        q, k = g.gptq_qk_norm_rope(q, k, positions, self.rope, self.q_weight, self.k_weight)
        g.gptq_kv_append(self.cache, plan, k, v)
        a = g.gptq_kv_attention(q, self.cache, plan, window=self.window, sinks=self.sinks, tree=tree)
        return self._project(self.o, a.reshape(len(x), -1)), k, v

    def extend(self, x):
        """Outputs [batch, new, hidden] for the next tokens x [batch, new, hidden] of every sequence."""
        batch, new, hidden = x.shape
        positions = (self.kv_len[:, None] + torch.arange(new, dtype=torch.int32, device=self.device)).flatten()
        self.kv_len += new
        return self._attend(x.reshape(-1, hidden), self._plan(batch * new, new), positions)[0].view(x.shape)

    def draft(self, x, parents):
        """Outputs [batch, new, hidden] of drafted tokens x, a tree a sequence (parents [batch, new], -1: after
        the last token).  They stay in the cache until `keep` says which of them remain."""
        batch, new, hidden = x.shape
        self.kv_len += new
        plan = self._plan(batch * new, new)
        tree = g.gptq_kv_tree(plan, parents.flatten().contiguous(), self.window, self.sinks)
        y, k, v = self._attend(x.reshape(-1, hidden), plan, tree.positions, tree)
        self.drafted = new, k, v
        return y.view(x.shape)

    def keep(self, path):
        """Of the drafted tokens of every sequence those of path [batch, kept] remain, in this order: a token, one
        that followed it, and so on."""
        new, k, v = self.drafted
        batch, kept = path.shape
        rows = (path + new * torch.arange(batch, device=self.device)[:, None]).flatten()
        self.kv_len += kept - new
        if kept:
            g.gptq_kv_append(self.cache, self._plan(batch * kept, kept), k[rows], v[rows])


def decode(block, prompt, steps, graph=True):
    """Feeds prompt [batch, tokens, hidden], then `steps` times the last output of each sequence.
    Returns the outputs of the prompt [batch, tokens, hidden] and of the steps [steps, batch, hidden]."""
    batch, tokens, hidden = prompt.shape
    whole = block.buffers(batch * tokens, tokens)
    first = block.step(prompt.reshape(-1, hidden), whole).view(batch, tokens, hidden).clone()
    one = block.buffers(batch, 1)
    x = first[:, -1].clone()
    outs = []

    def once():
        x.copy_(block.step(x, one))

    if graph:
        kept = x.clone(), block.kv_len.clone()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):  # the step once outside the graph, then undone
            once()
        torch.cuda.current_stream().wait_stream(side)
        x.copy_(kept[0])
        block.kv_len.copy_(kept[1])
        recorded = torch.cuda.CUDAGraph()
        with torch.cuda.graph(recorded):
            once()
    for _ in range(steps):
        recorded.replay() if graph else once()
        outs.append(x.clone())
    return first, torch.stack(outs)


def half_tree(drafts):
    """Parents of a tree of `drafts` tokens, each token after its half, and the path to its last, a deepest one."""
    parents = [(i + 1) // 2 - 1 for i in range(drafts)]
    path, at = [], drafts - 1
    while at >= 0:
        path.insert(0, at)
        at = parents[at]
    return parents, path


def check_drafts(batch, prompt, drafts, rounds=8):
    """Times rounds of a tree of `drafts` tokens a sequence of which the longest path is kept."""
    block = DraftBlock(batch=batch, max_tokens=prompt + (rounds + 1) * drafts, window=1024, sinks=4)
    parents, path = (torch.tensor(t, dtype=torch.int32, device=block.device).expand(batch, -1)
                     for t in half_tree(drafts))
    block.extend(torch.randn((batch, prompt, block.hidden), device=block.device))
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    for i in range(rounds + 1):
        if i == 1:
            begin.record()
        y = block.draft(torch.randn((batch, parents.shape[1], block.hidden), device=block.device), parents)
        block.keep(path)
    end.record()
    torch.cuda.synchronize()
    print(f"{rounds} trees of {parents.shape[1]} tokens, {path.shape[1]} kept, for each of {batch} sequences after "
          f"{prompt} tokens: {begin.elapsed_time(end):.2f} ms, last output norm {float(y.norm()):.4f}")


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--batch", type=int, default=4)
    ap.add_argument("--prompt", type=int, default=600)
    ap.add_argument("--steps", type=int, default=64)
    ap.add_argument("--bits", type=int, default=4)
    ap.add_argument("--drafts", type=int, default=0, help="drafted tokens of a tree checked after the prompt")
    a = ap.parse_args()
    if a.drafts:
        return check_drafts(a.batch, a.prompt, a.drafts)
    block = AttentionBlock(bits=a.bits, batch=a.batch, max_tokens=a.prompt + a.steps + 1)
    prompt = torch.randn((a.batch, a.prompt, block.hidden), device=block.device)
    decode(block, prompt, 4)
    block.kv_len.zero_()
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    begin.record()
    _, outs = decode(block, prompt, a.steps)
    end.record()
    torch.cuda.synchronize()
    print(f"prompt of {a.prompt} tokens and {a.steps} steps of {a.batch} sequences: {begin.elapsed_time(end):.2f} ms, "
          f"last output norm {float(outs[-1].norm()):.4f}")


if __name__ == "__main__":
    main()
