"""Greedy decoding steps of one attention block whose projections are packed by GPTQ and whose
keys and values live in a paged 8-bit cache.

    python examples/decode_attention.py [--batch 4] [--prompt 600] [--steps 8] [--bits 4]

A block of Llama-2-7B's attention shape unless told otherwise (hidden 4096, 32 heads of 128), with
random weights: q, k, v and o are quantized, packed and served by gptq_dequant_gemm; every query and
key head goes through an RMS norm and the position rotation; a prompt fills the cache, then each step
feeds the block's output back as the next token's input.  Each step is seven calls on one stream, with
nothing allocated inside, recorded once as a HIP graph and replayed.
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
                 device="cuda:0", seed=0):
        gen = torch.Generator(device=device).manual_seed(seed)

        def weight(rows, cols):
            return torch.randn((rows, cols), generator=gen, device=device) / math.sqrt(cols)

        self.hidden, self.q_heads, self.kv_heads, self.dim, self.batch = hidden, q_heads, kv_heads, dim, batch
        self.qkv = PackedLinear(weight((q_heads + 2 * kv_heads) * dim, hidden), bits)
        self.o = PackedLinear(weight(hidden, q_heads * dim), bits)
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


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--batch", type=int, default=4)
    ap.add_argument("--prompt", type=int, default=600)
    ap.add_argument("--steps", type=int, default=64)
    ap.add_argument("--bits", type=int, default=4)
    a = ap.parse_args()
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
