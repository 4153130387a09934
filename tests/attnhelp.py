"""Shared pieces of the attention operators' GPU tests: seeded inputs, the device side of a paged
cache and its oracle, and the error bounds, derived from the kernels' arithmetic.

u = 2^-24 is fp32's unit roundoff, H = 2^-8 that of a bf16 result, F = 2^-11 of an fp16 weight.
"""

from __future__ import annotations

import numpy as np

from gpuhelp import to_dev, torch_dev
from oracle import attn_ref as R

U, H, F = 2.0 ** -24, 2.0 ** -8, 2.0 ** -11


def rotation(rng, positions, rot):
    a = rng.uniform(0, 2 * np.pi, (positions, rot // 2))
    return np.cos(a).astype(np.float32), np.sin(a).astype(np.float32)


def bf16_round(x):
    torch, _ = torch_dev()
    return torch.from_numpy(np.asarray(x, dtype=np.float32)).to(torch.bfloat16)


def on_device(x, bf16, layout="plain"):
    """x [tokens, heads, dim] (already exact in the type) on the device, as a plain tensor, as a
    slice of a wider buffer, one that no 16-byte vector reaches, or with heads outermost."""
    torch, dev = torch_dev()
    t = bf16_round(x) if bf16 else torch.from_numpy(np.asarray(x, dtype=np.float32))
    n, h, d = t.shape
    if layout == "plain":
        return t.to(dev)
    if layout == "slice":
        w = torch.zeros((n, h + 3, d), dtype=t.dtype)
        w[:, 2:h + 2] = t
        return w.to(dev)[:, 2:h + 2]
    if layout == "odd":
        w = torch.zeros((n, h, d + 5), dtype=t.dtype)
        w[..., 1:d + 1] = t
        return w.to(dev)[..., 1:d + 1]
    assert layout == "heads first"
    return t.transpose(0, 1).contiguous().to(dev).transpose(0, 1)


def values(rng, shape, bf16, scale=1.0):
    """Normal values with a few large channels, exact in the type, as fp64."""
    x = rng.standard_normal(shape) * scale
    x[..., rng.integers(0, shape[-1], max(1, shape[-1] // 40))] *= 8.0
    return (bf16_round(x).float().numpy() if bf16 else x.astype(np.float32)).astype(np.float64)


def close(what, got, want, bound):
    err = np.abs(got.astype(np.float64) - want)
    worst = float(np.max(err / np.maximum(bound, 1e-300), initial=0.0))
    print(f"   {what}: max error {err.max(initial=0):.2e}, {worst:.3f} of its bound", flush=True)
    assert np.all(np.isfinite(got))
    assert np.all(err <= bound), f"{what}: {worst} times its bound"


class Paged:
    """A paged cache on the device and its oracle, with a shuffled block table for sequences of
    the given lengths; unused table entries are out of range."""

    def __init__(self, rng, lengths, kv_heads, block, dim, spare=2, contents=True, spread=1.0):
        import post_weight_quantization_03_amd as g
        torch, dev = torch_dev()
        need = [-(-n // block) for n in lengths]
        pages = sum(need) + spare
        order = rng.permutation(pages)
        self.table = np.full((len(lengths), max(max(need), 1) + 1), -7, dtype=np.int32)
        at = 0
        for b, k in enumerate(need):
            self.table[b, :k] = order[at:at + k]
            at += k
        self.lengths, self.block, self.kv_heads, self.dim = list(lengths), block, kv_heads, dim
        kc = rng.integers(-127, 128, (pages, kv_heads, block, dim)).astype(np.int8)
        vc = rng.integers(-127, 128, (pages, kv_heads, block // 16, dim, 16)).astype(np.int8)
        # scales as different as a long sequence's blocks have them; garbage where nothing was stored
        ks = 2.0 ** rng.integers(-7, -7 + max(1, int(2 * spread)), (pages, kv_heads))
        vs = 2.0 ** rng.integers(-9, -9 + max(1, int(6 * spread)), (pages, kv_heads))
        unused = order[at:]
        ks[unused], vs[unused] = np.nan, np.inf
        if not contents:
            ks[:], vs[:] = np.nan, -1.0
        self.ref = R.Cache(kc, vc, ks, vs)
        self.dev = g.KVCache(to_dev(kc), to_dev(vc), to_dev(ks.astype(np.float32)), to_dev(vs.astype(np.float32)))

    def plan(self, new, lengths=None, total=None, slack=0):
        """KVBatch of `new` tokens a sequence."""
        import post_weight_quantization_03_amd as g
        lengths = self.lengths if lengths is None else lengths
        start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        rows = int(start[-1]) if total is None else total
        return g.KVBatch(to_dev(start), to_dev(np.asarray(lengths, dtype=np.int32)), to_dev(self.table), rows,
                         max(new) + slack, max(lengths) if not slack else max(lengths) + 1), start

    def kv(self, b, length=None):
        n = self.lengths[b] if length is None else length
        return self.ref.read(self.table[b], n, False), self.ref.read(self.table[b], n, True)


def attention_bound(out, more, length, dim, bf16, vmax):
    """|error| of the operator's out and lse.  A score is a sum of dim exact products accumulated in
    fp32 and three more roundings (its two factors; in the exponent's fma), so it is off by at most
    ds = (dim + 8) 2u smag, relative error of the weight (with 2^-20 for the exponential of an argument
    up to 64 in size).  Weights are rounded to F (two parts: 2^-21) and have an absolute error of 2^-31
    of the largest where they are subnormal (the value scale included, vmax the largest value); the
    sums over tokens are accumulated in fp32 (length 2u); the result is rounded once."""
    ds = ((dim + 8) * 2 * U * more["smag"] + 2.0 ** -20)[..., None]
    w = 2 * ds + (F if bf16 else 2.0 ** -21) + length * 2 * U
    bound = w * 1.1 * more["absv"] + length * 2.0 ** -31 * vmax + (H if bf16 else 4 * U) * np.abs(out)
    lse = ds[..., 0] * 1.1 + length * 2 * U + 8 * U * (1 + np.abs(np.where(np.isfinite(more["lse"]), more["lse"], 0)))
    return bound, lse
