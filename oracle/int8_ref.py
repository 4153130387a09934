"""References of the 8-bit integer product (gptq_int8.h), from its definition.

quantize_tokens(x)                        codes, scales and sums, every quotient exact
product(codes, scales, sums, w, ws, wz)   the integer sums, and their values rounded as the definition says
"""

from __future__ import annotations

import numpy as np

LEAST_SCALE = np.float32(2.0 ** -120)


def quantize_tokens(x):
    """x [tokens, cols] (values exact in fp32) -> (codes int8, scales fp32, sums int32).  The quotient of
    two fp32 numbers that is not a half lies at least 2^-49 of itself away from one, so fp64 rounds it
    to the right side."""
    x = np.asarray(x, dtype=np.float64)
    with np.errstate(invalid="ignore"):
        finite = np.isfinite(x).all(1)
    most = np.abs(np.where(finite[:, None], x, 0.0)).max(1)
    scales = np.maximum((most / 127.0).astype(np.float32), LEAST_SCALE)
    codes = np.rint(np.where(finite[:, None], x, 0.0) / scales.astype(np.float64)[:, None]).astype(np.int8)
    return codes, np.where(finite, scales, np.float32(np.nan)), codes.sum(1, dtype=np.int64).astype(np.int32)


def product_sums(codes, w, zeros):
    """sum_k (w[r, k] - zeros[r]) codes[t, k] as int64 [tokens, rows], exact: fp64 products of integers
    below 2^15 whose sums stay below 2^53."""
    w = np.asarray(w, dtype=np.float64) - np.asarray(zeros, dtype=np.float64).reshape(-1, 1)
    return (np.asarray(codes, dtype=np.float64) @ w.T).astype(np.int64)


def product(codes, scales, w, w_scales, zeros):
    """fp32 [tokens, rows]: the sums rounded to fp32, times the token's scale, times the row's."""
    sums = product_sums(codes, w, zeros).astype(np.float32)
    with np.errstate(all="ignore"):
        return (sums * np.asarray(scales, np.float32)[:, None]) * np.asarray(w_scales, np.float32).reshape(1, -1)
