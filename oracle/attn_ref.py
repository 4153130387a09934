"""fp64 references of the attention operators (gptq_attn.h), from their definitions.

rope(x, cos, sin, interleaved)         rotation of the last axis' first 2 * cos.shape[-1] elements
norm_rope(x, w, ...)                   RMS norm (w None: none), then the rotation
norm_rope_backward(dy, x, w, ...)      gradients of x and w by the formula
Cache                                  the paged 8-bit cache: append, read, attention
"""

from __future__ import annotations

import numpy as np

MIN_EXP = -100


def rope(x, cos, sin, interleaved=False, back=False):
    """cos, sin broadcast against x[..., :rot / 2]."""
    half = cos.shape[-1]
    s = -sin if back else sin
    y = np.array(x, dtype=np.float64)
    a = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else (slice(0, half), slice(half, 2 * half))
    p, q = y[..., a[0]].copy(), y[..., a[1]].copy()
    y[..., a[0]] = p * cos - q * s
    y[..., a[1]] = p * s + q * cos
    return y


def norm(x, w, eps):
    x = np.asarray(x, dtype=np.float64)
    if w is None:
        return x
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(w, dtype=np.float64)


def norm_rope(x, w, cos, sin, positions, interleaved=False, eps=1e-6):
    """x [tokens, heads, dim]; cos, sin [max_pos, rot / 2]."""
    c, s = (np.asarray(t, dtype=np.float64)[positions][:, None] for t in (cos, sin))
    return rope(norm(x, w, eps), c, s, interleaved)


def norm_rope_backward(dy, x, w, cos, sin, positions, interleaved=False, eps=1e-6):
    """(dx, dw); dw None without w."""
    c, s = (np.asarray(t, dtype=np.float64)[positions][:, None] for t in (cos, sin))
    dn = rope(np.asarray(dy, dtype=np.float64), c, s, interleaved, back=True)
    if w is None:
        return dn, None
    x, w = np.asarray(x, dtype=np.float64), np.asarray(w, dtype=np.float64)
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    g = dn * w
    dx = r * g - x * r ** 3 * (g * x).mean(-1, keepdims=True)
    return dx, (dn * x * r).sum((0, 1))


def needed_scale(amax):
    """The least 2^e, e >= MIN_EXP, with amax <= 127 * 2^e; NaN where amax is not finite."""
    amax = np.asarray(amax, dtype=np.float64)
    with np.errstate(all="ignore"):
        m, e = np.frexp(np.where(np.isfinite(amax), amax, 1.0))
    e = np.where(m <= 127 / 128, e - 7, e - 6)
    e = np.where((m == 0) | (e < MIN_EXP), MIN_EXP, e)
    return np.where(np.isfinite(amax), np.ldexp(1.0, e), np.nan)


class Cache:
    """Pages in the layout of gptq_kv_cache, as numpy arrays that the operators' results are
    compared with: k_codes [pages, heads, block, dim], v_codes [pages, heads, block / 16, dim, 16],
    scales [pages, heads]."""

    def __init__(self, k_codes, v_codes, k_scales, v_scales):
        self.k_codes, self.v_codes = k_codes, v_codes
        self.k_scales, self.v_scales = k_scales.astype(np.float64), v_scales.astype(np.float64)
        self.block = k_codes.shape[2]

    def _tokens_of(self, page, is_v):
        """Codes of a page as [block, heads, dim]."""
        if not is_v:
            return self.k_codes[page].transpose(1, 0, 2)
        c = self.v_codes[page]  # heads, block / 16, dim, 16
        return c.transpose(1, 3, 0, 2).reshape(self.block, c.shape[0], c.shape[2])

    def _store(self, page, codes, is_v):
        if not is_v:
            self.k_codes[page] = codes.transpose(1, 0, 2)
        else:
            b, h, d = codes.shape
            self.v_codes[page] = codes.reshape(b // 16, 16, h, d).transpose(2, 0, 3, 1)

    def append(self, k, v, table, before):
        """Stores one sequence's new tokens k, v [n, heads, dim] (already normed and rotated) at
        places before, before + 1, ..."""
        n = k.shape[0]
        for blk in range(before // self.block, (before + n - 1) // self.block + 1):
            lo, hi = max(before - blk * self.block, 0), min(before + n - blk * self.block, self.block)
            at = blk * self.block + lo - before
            page = table[blk]
            for is_v, x, scales in ((False, k, self.k_scales), (True, v, self.v_scales)):
                x = x[at:at + hi - lo]
                with np.errstate(invalid="ignore"):
                    amax = np.where(np.isfinite(x).all((0, 2)), np.abs(x).max((0, 2)), np.inf)
                scale = needed_scale(amax)
                codes = self._tokens_of(page, is_v).astype(np.float64)
                if lo > 0:
                    was = scales[page].copy()
                    scale = np.where(np.isnan(was) | np.isnan(scale), np.nan, np.maximum(scale, was))
                    grown = scale > was
                    codes[:lo] = np.where(grown[:, None], np.rint(codes[:lo] * (was / scale)[:, None]), codes[:lo])
                with np.errstate(invalid="ignore"):
                    q = np.rint(x / scale[:, None])
                codes[lo:hi] = np.where(np.isfinite(q), np.clip(q, -127, 127), 0)
                scales[page] = scale
                self._store(page, codes.astype(np.int8), is_v)

    def read(self, table, tokens, is_v):
        """Values [tokens, heads, dim] of a sequence's first tokens."""
        scales = self.v_scales if is_v else self.k_scales
        blocks = -(-tokens // self.block)
        parts = [self._tokens_of(p, is_v).astype(np.float64) * scales[p][:, None] for p in table[:blocks]]
        if not parts:
            return np.zeros((0, self.k_codes.shape[1], self.k_codes.shape[3]))
        return np.concatenate(parts)[:tokens]


def attention(q, k, v, sm_scale, causal=True, window=0):
    """out [n, q_heads, dim], lse [n, q_heads] of a sequence's last n tokens q over its k, v [len,
    kv_heads, dim], and, for error bounds, dict(absv: sum of weight * |v| over the weights' sum,
    smag: the largest sum of |q_d k_d| sm_scale a row sees)."""
    n, qh, dim = q.shape
    length, kh = k.shape[:2]
    out, lse = np.zeros((n, qh, dim)), np.full((n, qh), -np.inf)
    absv, smag = np.zeros((n, qh, dim)), np.zeros((n, qh))
    j = np.arange(length)
    for i in range(n):
        p = length - n + i
        see = (j <= p) if causal else np.ones(length, dtype=bool)
        if window:
            see &= j > p - window
        if not see.any():
            continue
        for h in range(qh):
            kk, vv = k[see, h // (qh // kh)], v[see, h // (qh // kh)]
            s = kk @ q[i, h] * sm_scale
            with np.errstate(invalid="ignore"):
                m = s.max()
                w = np.exp(s - m)
                total = w.sum()
                out[i, h], lse[i, h] = w @ vv / total, m + np.log(total)
                absv[i, h] = w @ np.abs(vv) / total
                smag[i, h] = (np.abs(kk) @ np.abs(q[i, h])).max() * abs(sm_scale)
    return out, lse, {"absv": absv, "smag": smag}
