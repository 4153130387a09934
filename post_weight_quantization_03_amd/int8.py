"""The 8-bit integer product of libgptq.so (``include/gptq_int8.h``): tokens to int8 codes with one
scale each, and their product with a layer of 8-bit codes with one scale and zero point a row.

``Tokens`` holds quantized tokens together with the C struct built from them once; several layers may
share them.  The functions carry the C names, marshal arguments, and raise ``GptqError`` on a non-zero
status.  A call is made on the device of its tensors, and a call on another ``stream`` allocates what
it needs from that stream.  They are for serving: inputs that require gradients, or carry them in
forward mode, are refused.
"""

from __future__ import annotations

import ctypes

import post_weight_quantization_03_amd as _g
from .attn import _apart, _elsewhere, _empty, _one_device, _raw_stream, _refuse_gradients

_vp, _i64 = ctypes.c_void_p, ctypes.c_int64


class gptq_tokens(ctypes.Structure):
    _fields_ = [("codes", _vp), ("scales", _vp), ("sums", _vp), ("tokens", _i64), ("cols", _i64), ("stride", _i64)]


def bind(L):
    """Argument and result types of the entry points of gptq_int8.h."""
    P, ci = ctypes.POINTER, ctypes.c_int
    L.gptq_token_stride.argtypes = [_i64]
    L.gptq_token_stride.restype = _i64
    L.gptq_quantize_tokens.argtypes = [_vp, ci, _i64, P(gptq_tokens), _vp]
    L.gptq_quantize_tokens.restype = ci
    L.gptq_int8_gemm.argtypes = [_vp, _vp, _vp, _i64, P(gptq_tokens), _vp, ci, _i64, _vp]
    L.gptq_int8_gemm.restype = ci


def gptq_token_stride(cols: int) -> int:
    """Bytes that a token's codes take: cols rounded up to a multiple of 128."""
    n = -(-cols // 128) * 128
    if not 1 <= cols <= 65536:
        raise ValueError("cols must be in [1, 65536]")
    return n


class Tokens:
    """Quantized tokens: codes int8 [tokens, stride] (stride >= gptq_token_stride(cols), unit column
    stride, zeros from cols to there), scales fp32 [tokens], sums int32 [tokens] of the codes."""

    def __init__(self, codes, scales, sums, cols: int):
        torch = _g._torch()
        self.device = _one_device(codes, scales, sums)
        n = codes.shape[0]
        if (codes.dim() != 2 or codes.dtype != torch.int8 or scales.dtype != torch.float32 or sums.dtype != torch.int32
                or tuple(scales.shape) != (n,) or tuple(sums.shape) != (n,) or not scales.is_contiguous()
                or not sums.is_contiguous() or codes.stride(1) != 1 or codes.shape[1] < gptq_token_stride(cols)):
            raise ValueError("codes must be int8 [tokens, stride], scales fp32 [tokens], sums int32 [tokens]")
        stride = codes.stride(0) if n > 1 else codes.shape[1]
        if stride < codes.shape[1] or stride % 16:
            raise ValueError("codes must have a row stride of whole 16 bytes")
        self._hold(codes, scales, sums, n, cols, stride)

    def _hold(self, codes, scales, sums, n, cols, stride):
        self.codes, self.scales, self.sums, self.tokens, self.cols = codes, scales, sums, n, cols
        self.c = gptq_tokens(codes.data_ptr(), scales.data_ptr(), sums.data_ptr(), n, cols, stride)

    @classmethod
    def _new(cls, like, stream, device, tokens, cols):
        """Room made for a call on `stream`, on like's device."""
        torch = _g._torch()
        stride = gptq_token_stride(cols)
        t = cls.__new__(cls)
        t.device = device
        if stream is None:
            make = like.new_empty
            t._hold(make((tokens, stride), dtype=torch.int8), make(tokens, dtype=torch.float32),
                    make(tokens, dtype=torch.int32), tokens, cols, stride)
        else:
            t._hold(_empty((tokens, stride), like, stream, torch.int8), _empty((tokens,), like, stream, torch.float32),
                    _empty((tokens,), like, stream, torch.int32), tokens, cols, stride)
        return t

    @classmethod
    def empty(cls, tokens: int, cols: int, device):
        """Room for the codes of `tokens` tokens."""
        torch = _g._torch()
        return cls(torch.empty((tokens, gptq_token_stride(cols)), dtype=torch.int8, device=device),
                   torch.empty(tokens, dtype=torch.float32, device=device),
                   torch.empty(tokens, dtype=torch.int32, device=device), cols)


def _matrix(name, t, device):
    """Checks a 2-D tensor with unit column stride and returns its row stride."""
    if t.get_device() != device:
        raise _elsewhere(name, t, device)
    if t.dim() != 2 or t.stride(1) != 1 and t.shape[1] > 1:
        raise ValueError(f"{name} must be a 2-D device tensor with unit column stride")
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]  # a single row may carry any stride


def gptq_quantize_tokens(X, out: Tokens = None, stream=None) -> Tokens:
    """Codes, scales and sums of X [tokens, cols] (bf16 or fp32, unit column stride), new ones or `out`."""
    torch = _g._torch()
    _refuse_gradients("rounding tokens to 8 bits", torch, X)
    device = X.get_device()
    raw = _raw_stream(torch, device, stream)
    if raw is None:
        with torch.cuda.device(device):
            return gptq_quantize_tokens(X, out, stream)
    ldx = _matrix("X", X, device)
    tokens, cols = X.shape
    if out is None:
        out = Tokens._new(X, stream, device, tokens, cols)
    elif out.device != device:
        raise _apart(device, out)
    elif out.tokens != tokens or out.cols != cols:
        raise ValueError("out must have X's tokens and cols")
    st = _g.lib().gptq_quantize_tokens(X.data_ptr(), _g._dtype_code(X), ldx, out.c, raw)
    if st:
        raise _g.GptqError(st, "gptq_quantize_tokens")
    return out


def gptq_int8_gemm(packed, scales, zeros, x: Tokens, Y=None, dtype=None, stream=None):
    """Y [tokens, rows] (bf16 unless `dtype` or Y says fp32) = the tokens through the layer of packed
    [rows, cols / 4] 8-bit codes (int32 words), scales fp32 and zeros uint8 [rows] or [rows, 1]."""
    torch = _g._torch()
    _refuse_gradients("the 8-bit product", torch, scales)
    device = packed.get_device()
    raw = _raw_stream(torch, device, stream)
    if raw is None:
        with torch.cuda.device(device):
            return gptq_int8_gemm(packed, scales, zeros, x, Y, dtype, stream)
    for name, t in (("scales", scales), ("zeros", zeros)):
        if t.get_device() != device:
            raise _elsewhere(name, t, device)
    if x.device != device:
        raise _apart(device, x)
    rows = packed.shape[0]
    if (packed.dim() != 2 or packed.element_size() != 4 or packed.shape[1] * 4 != x.cols
            or scales.dtype != torch.float32 or zeros.dtype != torch.uint8 or scales.numel() != rows
            or zeros.numel() != rows or scales.shape[0] != rows or zeros.shape[0] != rows):
        raise ValueError("shape or dtype mismatch")
    if not packed.is_contiguous() or not scales.is_contiguous() or not zeros.is_contiguous():
        raise ValueError("packed, scales and zeros must be contiguous")
    if Y is None:
        Y = _empty((x.tokens, rows), scales, stream, torch.bfloat16 if dtype is None else dtype)
        ldy = rows
    else:
        ldy = _matrix("Y", Y, device)
        if tuple(Y.shape) != (x.tokens, rows) or dtype is not None and Y.dtype != dtype:
            raise ValueError("shape or dtype mismatch")
    st = _g.lib().gptq_int8_gemm(packed.data_ptr(), scales.data_ptr(), zeros.data_ptr(), rows, x.c, Y.data_ptr(),
                                 _g._dtype_code(Y), ldy, raw)
    if st:
        raise _g.GptqError(st, "gptq_int8_gemm")
    return Y
