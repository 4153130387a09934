"""The attention operators of libgptq.so (``include/gptq_attn.h``): per-head norm with
position rotation, the paged 8-bit cache, and attention over it.

``KVCache``, ``KVBatch`` and ``Rope`` hold the tensors a call refers to together with
the C struct built from them once; keep them between calls.  The functions carry the C
names, marshal arguments, and raise ``GptqError`` on a non-zero status.  Index data on
the device (positions, lengths, tables) is checked by the kernels: pass ``d_status``, a
zeroed device int32 tensor, to see whether any was out of range.

A call is made on the device of its tensors, and a call on another ``stream`` allocates what it
needs from that stream.  gptq_qk_norm_rope is recorded by autograd; the cache's operators are for
serving and are not.
"""

from __future__ import annotations

import ctypes
import math

import post_weight_quantization_03_amd as _g

_vp, _i64, _i32, _sz, _f = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t, ctypes.c_float


class gptq_rope(ctypes.Structure):
    _fields_ = [("cos", _vp), ("sin", _vp), ("max_pos", _i64), ("rot", _i32), ("interleaved", _i32), ("eps", _f)]


class gptq_heads(ctypes.Structure):
    _fields_ = [("x", _vp), ("x_token", _i64), ("x_head", _i64), ("y", _vp), ("y_token", _i64), ("y_head", _i64),
                ("weight", _vp), ("heads", _i32)]


class gptq_heads_grad(ctypes.Structure):
    _fields_ = [("dy", _vp), ("dy_token", _i64), ("dy_head", _i64), ("x", _vp), ("x_token", _i64), ("x_head", _i64),
                ("dx", _vp), ("dx_token", _i64), ("dx_head", _i64), ("weight", _vp), ("dweight", _vp),
                ("heads", _i32)]


class gptq_kv_cache(ctypes.Structure):
    _fields_ = [("k_codes", _vp), ("v_codes", _vp), ("k_scales", _vp), ("v_scales", _vp), ("pages", _i64),
                ("kv_heads", _i32), ("block", _i32), ("dim", _i32)]


class gptq_kv_batch(ctypes.Structure):
    _fields_ = [("q_start", _vp), ("kv_len", _vp), ("block_table", _vp), ("table_stride", _i64), ("batch", _i64),
                ("total", _i64), ("max_new", _i64), ("max_kv", _i64)]


class gptq_attention(ctypes.Structure):
    _fields_ = [("q_heads", _i32), ("sm_scale", _f), ("causal", _i32), ("window", _i64)]


def bind(L):
    """Argument and result types of the entry points of gptq_attn.h."""
    P, ci = ctypes.POINTER, ctypes.c_int
    L.gptq_qk_norm_rope.argtypes = [P(gptq_heads), P(gptq_heads), ci, _i64, _i32, _vp, P(gptq_rope), _vp, _vp]
    L.gptq_qk_norm_rope.restype = ci
    L.gptq_qk_norm_rope_backward_workspace_bytes.argtypes = [_i64, _i32, _i32, _i32]
    L.gptq_qk_norm_rope_backward_workspace_bytes.restype = _sz
    L.gptq_qk_norm_rope_backward.argtypes = [P(gptq_heads_grad), P(gptq_heads_grad), ci, _i64, _i32, _vp,
                                             P(gptq_rope), _vp, _sz, _vp, _vp]
    L.gptq_qk_norm_rope_backward.restype = ci
    L.gptq_kv_append.argtypes = [P(gptq_kv_cache), P(gptq_kv_batch), _vp, _i64, _i64, _vp, _i64, _i64, ci, _vp,
                                 P(gptq_rope), _vp, _vp]
    L.gptq_kv_append.restype = ci
    L.gptq_kv_read.argtypes = [P(gptq_kv_cache), P(gptq_kv_batch), _vp, _i64, _i64, _vp, _i64, _i64, ci, _vp, _vp]
    L.gptq_kv_read.restype = ci
    L.gptq_kv_attention_workspace_bytes.argtypes = [P(gptq_kv_cache), P(gptq_kv_batch), ci, P(gptq_attention)]
    L.gptq_kv_attention_workspace_bytes.restype = _sz
    L.gptq_kv_attention.argtypes = [P(gptq_kv_cache), P(gptq_kv_batch), P(gptq_attention), _vp, _i64, _i64, _vp,
                                    _i64, _i64, _vp, ci, _vp, _sz, _vp, _vp]
    L.gptq_kv_attention.restype = ci


# --------------------------------------------------------------------------- helpers

def _elsewhere(name, t, device):
    """The error of a tensor that is not on the call's device."""
    if not t.is_cuda:
        return ValueError(f"{name} must be a device tensor")
    return ValueError(f"{name} is on device {t.get_device()}, the call on {device}: a call's tensors are on one device")


def _raw_stream(torch, d, stream):
    """The HIP stream of `stream`, or of device d's current one, for a call on device d (None: d is not the current
    device)."""
    if d < 0:
        raise ValueError("the tensors must be device tensors")
    if stream is not None and stream.device_index != d:
        raise ValueError(f"the stream is on device {stream.device_index}, the call on {d}: they are on one device")
    if d != torch._C._cuda_getDevice():
        return None
    return torch._C._cuda_getCurrentRawStream(d) if stream is None else stream.cuda_stream


def _int32(name, t, device, shape=None):
    torch = _g._torch()
    if t.get_device() != device:
        raise _elsewhere(name, t, device)
    if t.dtype != torch.int32 or t.stride(-1) != 1 and t.shape[-1] > 1:
        raise ValueError(f"{name} must be an int32 device tensor with unit stride")
    if shape is not None and tuple(t.shape) != shape:
        raise ValueError(f"{name} must have shape {shape}")


def _status(t, device):
    _int32("d_status", t, device)
    if t.numel() < 1:
        raise ValueError("d_status must hold one int32")
    return t.data_ptr()


def _heads(name, t, device, dtype=None, shape=None):
    """Checks a [tokens, heads, dim] tensor with unit stride in dim, any strides before it, and returns its strides."""
    s = t.stride()
    if t.get_device() != device:
        raise _elsewhere(name, t, device)
    if len(s) != 3 or s[2] != 1 and t.shape[2] > 1:
        raise ValueError(f"{name} must be a [tokens, heads, dim] device tensor with unit stride in dim")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must have dtype {dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}")
    return s


def _weight(name, w, like, device):
    if w is None:
        return None
    if w.get_device() != device:
        raise _elsewhere(name, w, device)
    if w.dtype != like.dtype or w.dim() != 1 or w.numel() != like.shape[2] or not w.is_contiguous():
        raise ValueError(f"{name} must be a contiguous [dim] device tensor of dtype {like.dtype}")
    return w.data_ptr()


def _given(name, t, device):
    """(pointer, bytes) of a workspace."""
    if t.get_device() != device:
        raise _elsewhere(name, t, device)
    return t.data_ptr(), t.numel() * t.element_size()


def _apart(device, *handles):
    """The error of a handle whose tensors are not on the call's device."""
    h = next(h for h in handles if h.device != device)
    return ValueError(f"the {type(h).__name__} is on device {h.device}, the call on {device}: a call's tensors are on "
                      "one device")


def _on(like, stream, make):
    """An output of the binding's own, made by `make`: from the stream that writes it (as a
    workspace), and kept until the caller's stream, which reads it, has done so."""
    if stream is None:
        return make()
    torch = _g._torch()
    callers = torch.cuda.current_stream(like.device)
    with torch.cuda.stream(stream):
        t = make()
    t.record_stream(callers)
    return t


def _empty(shape, like, stream, dtype):
    return _on(like, stream, lambda: like.new_empty(shape, dtype=dtype))


def _empty_as(like, stream, dtype=None):
    """A contiguous tensor of like's shape."""
    torch = _g._torch()
    if stream is None:
        return torch.empty_like(like, dtype=dtype, memory_format=torch.contiguous_format)
    return _on(like, stream, lambda: torch.empty_like(like, dtype=dtype, memory_format=torch.contiguous_format))


# --------------------------------------------------------------------------- handles

def _one_device(*tensors):
    """The index of the device that holds all of a handle's tensors."""
    d = tensors[0].get_device()
    for t in tensors:
        if d < 0 or t.get_device() != d:
            raise _elsewhere("a tensor", t, d)
    return d


class Rope:
    """cos and sin [max_pos, rot / 2] (fp32, contiguous) of a position rotation, its pairing, and
    the eps of the norm before it.  Rope(None, None) rotates nothing."""

    def __init__(self, cos, sin, interleaved: bool = False, eps: float = 1e-6):
        torch = _g._torch()
        self.cos, self.sin, self.device = cos, sin, None
        if cos is None:
            self.c = gptq_rope(None, None, 0, 0, int(interleaved), eps)
            return
        if (cos.dtype != torch.float32 or sin.dtype != torch.float32 or cos.dim() != 2 or cos.shape != sin.shape):
            raise ValueError("cos and sin must be fp32 [max_pos, rot / 2]")
        _g._check_dev(cos, sin)
        self.device = _one_device(cos, sin)
        self.c = gptq_rope(cos.data_ptr(), sin.data_ptr(), cos.shape[0], 2 * cos.shape[1], int(interleaved), eps)


class KVCache:
    """The paged cache: k_codes int8 [pages, kv_heads, block, dim], v_codes int8 [pages, kv_heads,
    block / 16, dim, 16], k_scales and v_scales fp32 [pages, kv_heads], all contiguous."""

    def __init__(self, k_codes, v_codes, k_scales, v_scales):
        torch = _g._torch()
        _g._check_dev(k_codes, v_codes, k_scales, v_scales)
        pages, heads, block, dim = k_codes.shape
        if (k_codes.dtype != torch.int8 or v_codes.dtype != torch.int8 or k_scales.dtype != torch.float32
                or v_scales.dtype != torch.float32 or block % 16
                or tuple(v_codes.shape) != (pages, heads, block // 16, dim, 16)
                or tuple(k_scales.shape) != (pages, heads) or k_scales.shape != v_scales.shape):
            raise ValueError("shape or dtype mismatch")
        self.k_codes, self.v_codes, self.k_scales, self.v_scales = k_codes, v_codes, k_scales, v_scales
        self.pages, self.kv_heads, self.block, self.dim = pages, heads, block, dim
        self.device = _one_device(k_codes, v_codes, k_scales, v_scales)
        self.c = gptq_kv_cache(k_codes.data_ptr(), v_codes.data_ptr(), k_scales.data_ptr(), v_scales.data_ptr(),
                               pages, heads, block, dim)

    @classmethod
    def empty(cls, pages: int, kv_heads: int, block: int, dim: int, device):
        """A cache of `pages` pages; nothing has to be cleared."""
        torch = _g._torch()
        return cls(torch.empty((pages, kv_heads, block, dim), dtype=torch.int8, device=device),
                   torch.empty((pages, kv_heads, block // 16, dim, 16), dtype=torch.int8, device=device),
                   torch.empty((pages, kv_heads), dtype=torch.float32, device=device),
                   torch.empty((pages, kv_heads), dtype=torch.float32, device=device))


class KVBatch:
    """Sequences and their new tokens: q_start [batch + 1], kv_len [batch] and block_table [batch,
    blocks], int32 device tensors whose contents may change between calls; total: the rows of the
    token tensors; max_new, max_kv: upper bounds of a sequence's new tokens and of kv_len."""

    def __init__(self, q_start, kv_len, block_table, total: int, max_new: int, max_kv: int):
        batch = kv_len.shape[0]
        self.device = _one_device(kv_len, q_start, block_table)
        _int32("kv_len", kv_len, self.device, (batch,))
        _int32("q_start", q_start, self.device, (batch + 1,))
        _int32("block_table", block_table, self.device)
        if block_table.dim() != 2 or block_table.shape[0] != batch:
            raise ValueError("block_table must be [batch, blocks]")
        self.q_start, self.kv_len, self.block_table = q_start, kv_len, block_table
        self.total, self.max_new, self.max_kv = total, max_new, max_kv
        self.blocks = block_table.shape[1]
        stride = block_table.stride(0) if batch > 1 else self.blocks
        self.c = gptq_kv_batch(q_start.data_ptr(), kv_len.data_ptr(), block_table.data_ptr(), stride, batch, total,
                               max_new, max_kv)


def _check_plan(cache, batch):
    if batch.max_kv > batch.blocks * cache.block:
        raise ValueError("block_table has too few blocks for max_kv")


# --------------------------------------------------------------------------- entry points

def _side(name, x, weight, out, device, stream):
    if x is None:
        return None, None
    sx = _heads(name, x, device)
    if out is None:
        out = _empty_as(x, stream)
        sy = out.stride()
    else:
        sy = _heads(name + "_out", out, device, x.dtype, x.shape)
    return out, gptq_heads(x.data_ptr(), sx[0], sx[1], out.data_ptr(), sy[0], sy[1],
                           _weight(name + "_weight", weight, x, device), x.shape[1])


_recorded = None


def _autograd():
    """gptq_qk_norm_rope as a function of q, k and the weights that autograd records."""
    global _recorded
    if _recorded is None:
        torch = _g._torch()

        class NormRope(torch.autograd.Function):
            @staticmethod
            def forward(ctx, q, k, q_weight, k_weight, positions, rope, d_status):
                ctx.save_for_backward(q, k, q_weight, k_weight, positions)
                ctx.rope = rope
                return gptq_qk_norm_rope(q, k, positions, rope, q_weight, k_weight, d_status=d_status)

            @staticmethod
            @torch.autograd.function.once_differentiable
            def backward(ctx, dq_out, dk_out):
                q, k, q_weight, k_weight, positions = ctx.saved_tensors
                # a gradient may come broadcast, with any strides
                dy = [d if d is None or d.stride(2) == 1 else d.contiguous() for d in (dq_out, dk_out)]
                dq, dk, dqw, dkw = gptq_qk_norm_rope_backward(*dy, q, k, positions, ctx.rope, q_weight, k_weight)
                return (dq, dk, None if dqw is None else dqw.to(q_weight.dtype),
                        None if dkw is None else dkw.to(k_weight.dtype), None, None, None)

        _recorded = NormRope
    return _recorded


def gptq_qk_norm_rope(q, k, positions, rope: Rope, q_weight=None, k_weight=None, q_out=None, k_out=None,
                      d_status=None, stream=None):
    """(q_out, k_out): RMS norm (where a weight [dim] is given) and rotation of every head of
    q and k [tokens, heads, dim] (bf16 or fp32) at positions [tokens] (int32).  q or k may be None;
    q_out may be q.  Where autograd records and q, k or a weight requires gradients, the outputs carry
    them (weights' gradients rounded to the weight's type); q_out, k_out and stream are then refused."""
    like = q if q is not None else k
    if like is None:
        raise ValueError("q or k must be given")
    torch = _g._torch()
    if torch.is_grad_enabled() and (like.requires_grad or k is not None and k.requires_grad or
                                    q_weight is not None and q_weight.requires_grad or
                                    k_weight is not None and k_weight.requires_grad):
        if q_out is not None or k_out is not None or stream is not None:
            raise ValueError("gradients are recorded for new outputs on the current stream only (torch.no_grad() "
                             "calls without them)")
        return _autograd().apply(q, k, q_weight, k_weight, positions, rope, d_status)
    device = like.get_device()
    raw = _raw_stream(torch, device, stream)
    if raw is None:
        with torch.cuda.device(device):
            return gptq_qk_norm_rope(q, k, positions, rope, q_weight, k_weight, q_out, k_out, d_status, stream)
    q_out, cq = _side("q", q, q_weight, q_out, device, stream)
    k_out, ck = _side("k", k, k_weight, k_out, device, stream)
    tokens, _, dim = like.shape
    if k is not None and (k.shape[0] != tokens or k.shape[2] != dim or k.dtype != like.dtype):
        raise ValueError("q and k must have the same tokens, dim and dtype")
    if positions is not None:
        _int32("positions", positions, device, (tokens,))
    if rope.device != device and rope.device is not None:
        raise _apart(device, rope)
    st = _g.lib().gptq_qk_norm_rope(cq, ck, _g._dtype_code(like), tokens, dim,
                                    None if positions is None else positions.data_ptr(),
                                    rope.c, None if d_status is None else _status(d_status, device), raw)
    if st:
        raise _g.GptqError(st, "gptq_qk_norm_rope")
    return q_out, k_out


def gptq_qk_norm_rope_backward_workspace_bytes(tokens: int, dim: int, q_heads: int, k_heads: int) -> int:
    return int(_g.lib().gptq_qk_norm_rope_backward_workspace_bytes(tokens, dim, q_heads, k_heads))


def _grad_side(name, dy, x, weight, device, stream):
    if dy is None:
        return None, None, None
    sg = _heads("d" + name, dy, device)
    sx = (0, 0)
    if weight is not None:
        if x is None:
            raise ValueError(f"{name} is needed with its weight")
        sx = _heads(name, x, device, dy.dtype, dy.shape)
    dx = _empty_as(dy, stream)
    dw = None if weight is None else _empty_as(weight, stream, _g._torch().float32)
    sd = dx.stride()
    return dx, dw, gptq_heads_grad(dy.data_ptr(), sg[0], sg[1], None if weight is None else x.data_ptr(), sx[0], sx[1],
                                   dx.data_ptr(), sd[0], sd[1], _weight(name + "_weight", weight, dy, device),
                                   None if dw is None else dw.data_ptr(), dy.shape[1])


def gptq_qk_norm_rope_backward(dq_out, dk_out, q, k, positions, rope: Rope, q_weight=None, k_weight=None,
                               workspace=None, d_status=None, stream=None):
    """(dq, dk, dq_weight, dk_weight) of gptq_qk_norm_rope from the gradients of its outputs and its
    inputs; the weights' gradients are fp32 (None without a weight)."""
    like = dq_out if dq_out is not None else dk_out
    if like is None:
        raise ValueError("dq_out or dk_out must be given")
    torch = _g._torch()
    device = like.get_device()
    raw = _raw_stream(torch, device, stream)
    if raw is None:
        with torch.cuda.device(device):
            return gptq_qk_norm_rope_backward(dq_out, dk_out, q, k, positions, rope, q_weight, k_weight, workspace,
                                              d_status, stream)
    dq, dqw, cq = _grad_side("q", dq_out, q, q_weight, device, stream)
    dk, dkw, ck = _grad_side("k", dk_out, k, k_weight, device, stream)
    tokens, _, dim = like.shape
    if dk_out is not None and (dk_out.shape[0] != tokens or dk_out.shape[2] != dim or dk_out.dtype != like.dtype):
        raise ValueError("dq_out and dk_out must have the same tokens, dim and dtype")
    if positions is not None:
        _int32("positions", positions, device, (tokens,))
    if workspace is None and (dqw is not None or dkw is not None):
        need = gptq_qk_norm_rope_backward_workspace_bytes(tokens, dim, 0 if dq is None else dq.shape[1],
                                                          0 if dk is None else dk.shape[1])
        workspace = _g._workspace(need, like, stream)
    if rope.device != device and rope.device is not None:
        raise _apart(device, rope)
    wp, wn = (None, 0) if workspace is None else _given("workspace", workspace, device)
    st = _g.lib().gptq_qk_norm_rope_backward(cq, ck, _g._dtype_code(like), tokens, dim,
                                             None if positions is None else positions.data_ptr(),
                                             rope.c, wp, wn,
                                             None if d_status is None else _status(d_status, device), raw)
    if st:
        raise _g.GptqError(st, "gptq_qk_norm_rope_backward")
    return dq, dk, dqw, dkw


def gptq_kv_append(cache: KVCache, batch: KVBatch, k, v, rope: Rope = None, k_weight=None, d_status=None,
                   stream=None):
    """Stores the batch's new tokens: k, v [total, kv_heads, dim] (bf16 or fp32), k through the norm
    (k_weight) and rotation (rope) at its place in the sequence."""
    torch = _g._torch()
    device = k.get_device()
    raw = _raw_stream(torch, device, stream)
    if raw is None:
        with torch.cuda.device(device):
            return gptq_kv_append(cache, batch, k, v, rope, k_weight, d_status, stream)
    _check_plan(cache, batch)
    sk = _heads("k", k, device, None, (batch.total, cache.kv_heads, cache.dim))
    sv = _heads("v", v, device, k.dtype, k.shape)
    if cache.device != device or batch.device != device:
        raise _apart(device, cache, batch)
    if rope is not None and rope.device != device and rope.device is not None:
        raise _apart(device, rope)
    st = _g.lib().gptq_kv_append(cache.c, batch.c, k.data_ptr(), sk[0], sk[1], v.data_ptr(), sv[0], sv[1],
                                 _g._dtype_code(k), _weight("k_weight", k_weight, k, device),
                                 None if rope is None else rope.c,
                                 None if d_status is None else _status(d_status, device), raw)
    if st:
        raise _g.GptqError(st, "gptq_kv_append")


def gptq_kv_read(cache: KVCache, batch: KVBatch, dtype=None, k_out=None, v_out=None, d_status=None, stream=None):
    """(k, v) [total, kv_heads, dim] of the batch's new tokens out of the cache, bf16 unless `dtype`
    or the given outputs say fp32."""
    torch = _g._torch()
    device = cache.device
    raw = _raw_stream(torch, device, stream)
    if raw is None:
        with torch.cuda.device(device):
            return gptq_kv_read(cache, batch, dtype, k_out, v_out, d_status, stream)
    _check_plan(cache, batch)
    shape = (batch.total, cache.kv_heads, cache.dim)
    given = k_out if k_out is not None else v_out
    if dtype is None:
        dtype = torch.bfloat16 if given is None else given.dtype
    if k_out is None and v_out is None:
        k_out = _empty(shape, cache.k_codes, stream, dtype)
        v_out = _empty(shape, cache.k_codes, stream, dtype)
    sk = sv = (0, 0)
    if k_out is not None:
        sk = _heads("k_out", k_out, device, dtype, shape)
    if v_out is not None:
        sv = _heads("v_out", v_out, device, dtype, shape)
    like = k_out if k_out is not None else v_out
    if batch.device != device:
        raise _apart(device, batch)
    st = _g.lib().gptq_kv_read(cache.c, batch.c, None if k_out is None else k_out.data_ptr(), sk[0], sk[1],
                               None if v_out is None else v_out.data_ptr(), sv[0], sv[1], _g._dtype_code(like),
                               None if d_status is None else _status(d_status, device), raw)
    if st:
        raise _g.GptqError(st, "gptq_kv_read")
    return k_out, v_out


def gptq_kv_attention_workspace_bytes(cache: KVCache, batch: KVBatch, q_heads: int, dtype: int, causal: bool = True,
                                      window: int = 0) -> int:
    """Workspace bytes of gptq_kv_attention; dtype: GPTQ_BF16 or GPTQ_F32."""
    return int(_g.lib().gptq_kv_attention_workspace_bytes(cache.c, batch.c, dtype,
                                                          gptq_attention(q_heads, 1.0, int(causal), window)))


def gptq_kv_attention(q, cache: KVCache, batch: KVBatch, sm_scale=None, causal: bool = True, window: int = 0,
                      out=None, lse=None, want_lse: bool = False, workspace=None, d_status=None, stream=None):
    """Attention of the batch's new tokens q [total, q_heads, dim] (bf16 or fp32) over the cache.
    sm_scale: dim^-1/2 unless given.  Returns out, or (out, lse) when lse [total, q_heads] (fp32)
    is given or wanted.  Rows that no sequence owns are left as they are."""
    torch = _g._torch()
    device = q.get_device()
    raw = _raw_stream(torch, device, stream)
    if raw is None:
        with torch.cuda.device(device):
            return gptq_kv_attention(q, cache, batch, sm_scale, causal, window, out, lse, want_lse, workspace, d_status,
                                     stream)
    _check_plan(cache, batch)
    sq = _heads("q", q, device)
    total, heads, dim = q.shape
    if total != batch.total or dim != cache.dim:
        raise ValueError("shape mismatch")
    if out is None:
        out = _empty_as(q, stream)
        so = out.stride()
    else:
        so = _heads("out", out, device, q.dtype, q.shape)
    if lse is None:
        if want_lse:
            lse = _empty((total, heads), q, stream, torch.float32)
    elif lse.get_device() != device:
        raise _elsewhere("lse", lse, device)
    elif lse.dtype != torch.float32 or tuple(lse.shape) != (total, heads) or not lse.is_contiguous():
        raise ValueError("lse must be a contiguous fp32 [total, q_heads] device tensor")
    a = gptq_attention(heads, 1.0 / math.sqrt(dim) if sm_scale is None else sm_scale, int(causal), window)
    dt = _g._dtype_code(q)
    if cache.device != device or batch.device != device:
        raise _apart(device, cache, batch)
    L = _g.lib()
    if workspace is None:
        need = L.gptq_kv_attention_workspace_bytes(cache.c, batch.c, dt, a)
        if need:
            workspace = _g._workspace(need, q, stream)
    wp, wn = (None, 0) if workspace is None else _given("workspace", workspace, device)
    st = L.gptq_kv_attention(cache.c, batch.c, a, q.data_ptr(), sq[0], sq[1], out.data_ptr(), so[0], so[1],
                             None if lse is None else lse.data_ptr(), dt, wp, wn,
                             None if d_status is None else _status(d_status, device), raw)
    if st:
        raise _g.GptqError(st, "gptq_kv_attention")
    return out if lse is None else (out, lse)
