"""fp64 references of masked attention over the cache (gptq_mask.h), from its definitions.

window_sees(n, length, window, sinks, causal)   which tokens each new one sees, without a tree
tree(parents, before, window, sinks)            positions, and which new tokens each new one sees
tree_sees(positions, among, before, ...)        which tokens each new one sees, with a tree
words(among, count)                             the rows' masks in words of 64 bits
attention(q, k, v, sm_scale, sees)              as attn_ref.attention, for any pattern
"""

from __future__ import annotations

import numpy as np


def window_sees(n, length, window=0, sinks=0, causal=True):
    p = np.arange(length - n, length)[:, None]
    j = np.arange(length)
    sees = (j <= p) if causal else np.ones((n, length), dtype=bool)
    return sees & ((j > p - window) | (j < sinks)) if window else sees


def tree(parents, before, window=0, sinks=0):
    n = len(parents)
    depth, among = np.zeros(n, dtype=np.int64), np.zeros((n, n), dtype=bool)
    for i, p in enumerate(parents):
        if p >= 0:
            depth[i] = depth[p] + 1
            among[i] = among[p]
        among[i, i] = True
    at = before + depth
    if window:
        among &= (at[None] > at[:, None] - window) | (at[None] < sinks)
    return at, among


def tree_sees(positions, among, before, window=0, sinks=0):
    n = len(positions)
    p, j = np.asarray(positions)[:, None], np.arange(before)
    first = np.ones((n, before), dtype=bool)
    if window:
        first &= (j > p - window) | (j < sinks)
    return np.concatenate([first, among], 1)


def words(among, count):
    n = among.shape[1]
    w = np.zeros((among.shape[0], count), dtype=np.uint64)
    for a in range(n):
        w[:, a // 64] |= among[:, a].astype(np.uint64) << np.uint64(a % 64)
    return w


def attention(q, k, v, sm_scale, sees):
    """out [n, q_heads, dim], lse [n, q_heads] and dict(absv, smag) of q over k, v [len, kv_heads, dim]
    where sees [n, len]."""
    n, qh, dim = q.shape
    group = qh // k.shape[1]
    out, lse = np.zeros((n, qh, dim)), np.full((n, qh), -np.inf)
    absv, smag = np.zeros((n, qh, dim)), np.zeros((n, qh))
    for h in range(qh):
        kk, vv = k[:, h // group], v[:, h // group]
        for i in range(n):
            if not sees[i].any():
                continue
            ki, vi = kk[sees[i]], vv[sees[i]]
            s = ki @ q[i, h] * sm_scale
            m = s.max()
            w = np.exp(s - m)
            total = w.sum()
            out[i, h], lse[i, h] = w @ vi / total, m + np.log(total)
            absv[i, h] = w @ np.abs(vi) / total
            smag[i, h] = (np.abs(ki) @ np.abs(q[i, h])).max() * abs(sm_scale)
    return out, lse, {"absv": absv, "smag": smag}
