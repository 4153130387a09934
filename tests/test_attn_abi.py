"""The attention operators' C ABI on the host (no GPU): every declared symbol is exported, and
argument errors are reported before any device work.  Pointers passed here are never dereferenced:
every call below returns from its host-side checks."""

import ctypes
import os
import re
import subprocess

import pytest

import post_weight_quantization_03_amd as g
from post_weight_quantization_03_amd import attn

HEADER = os.path.join(os.path.dirname(os.path.dirname(__file__)), "include", "gptq_attn.h")
A = 0x1000  # an aligned address that is not used


def test_every_declared_symbol_is_exported():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(gptq_[a-z_]+)\s*\(", text))
    assert names == {"gptq_qk_norm_rope", "gptq_qk_norm_rope_backward", "gptq_qk_norm_rope_backward_workspace_bytes",
                     "gptq_kv_append", "gptq_kv_read", "gptq_kv_attention", "gptq_kv_attention_workspace_bytes"}
    for lib in (g.lib(), ctypes.CDLL(os.path.join(os.path.dirname(g.LIB_PATH), "libgptq_trace.so"))):
        for n in names:
            assert hasattr(lib, n), n
    for n in names:
        assert callable(getattr(g, n))


def rope(cos=A, sin=A, max_pos=100, rot=64, interleaved=0, eps=1e-6):
    return attn.gptq_rope(cos, sin, max_pos, rot, interleaved, eps)


def heads(x=A, y=2 * A, strides=(4096, 128, 4096, 128), weight=None, n=4):
    return attn.gptq_heads(x, strides[0], strides[1], y, strides[2], strides[3], weight, n)


def norm_rope(q=None, k=None, dtype=0, tokens=3, dim=128, positions=A, r=None, status=None):
    return g.lib().gptq_qk_norm_rope(q if q is not None else heads(), k, dtype, tokens, dim, positions,
                                     rope() if r is None else r, status, None)


def test_norm_rope_refusals():
    E, U, OK = g.GPTQ_EINVAL, g.GPTQ_EUNSUPPORTED, g.GPTQ_OK
    assert norm_rope(tokens=0) == OK
    assert norm_rope(q=heads(n=0)) == OK
    assert norm_rope(tokens=-1) == E
    assert norm_rope(dtype=7) == E
    assert norm_rope(dim=0) == E
    assert norm_rope(dim=120) == U and norm_rope(dim=528) == U
    assert norm_rope(q=heads(x=None)) == E and norm_rope(q=heads(y=None)) == E
    assert norm_rope(q=heads(x=A + 1)) == E                                # element alignment
    assert norm_rope(q=heads(x=A, y=A, strides=(4096, 128, 8192, 128))) == E   # in place, other strides
    assert norm_rope(q=heads(weight=A + 1)) == E
    assert norm_rope(q=heads(n=-1)) == E
    assert norm_rope(positions=None) == E and norm_rope(positions=A + 2) == E
    assert norm_rope(status=A + 2) == E
    assert norm_rope(r=rope(rot=130)) == E and norm_rope(r=rope(rot=-2)) == E
    assert norm_rope(r=rope(rot=40)) == U
    assert norm_rope(r=rope(cos=None)) == E and norm_rope(r=rope(sin=A + 4)) == E
    assert norm_rope(r=rope(interleaved=2)) == E
    assert norm_rope(r=rope(eps=-1.0)) == E and norm_rope(r=rope(eps=float("nan"))) == E
    assert norm_rope(r=rope(max_pos=-1)) == E
    assert norm_rope(tokens=1 << 29) == U                                   # work items past 32 bits
    assert g.lib().gptq_qk_norm_rope(None, None, 0, 3, 128, A, None, None, None) == E


def grads(dy=A, x=2 * A, dx=3 * A, weight=4 * A, dweight=5 * A, n=4, strides=(512, 128)):
    return attn.gptq_heads_grad(dy, *strides, x, *strides, dx, *strides, weight, dweight, n)


def backward(q=None, tokens=3, dim=128, ws=A, ws_bytes=1 << 30):
    return g.lib().gptq_qk_norm_rope_backward(q if q is not None else grads(), None, 0, tokens, dim, A, rope(), ws,
                                              ws_bytes, None, None)


def test_norm_rope_backward_refusals():
    E = g.GPTQ_EINVAL
    need = g.gptq_qk_norm_rope_backward_workspace_bytes(3, 128, 4, 0)
    assert need > 0 and need % (128 * 4) == 0
    assert g.gptq_qk_norm_rope_backward_workspace_bytes(0, 128, 4, 2) == 0
    assert g.gptq_qk_norm_rope_backward_workspace_bytes(3, 120, 4, 2) == 0
    assert backward(ws_bytes=need - 1) == g.GPTQ_EWORKSPACE and backward(ws=None) == g.GPTQ_EWORKSPACE
    assert backward(ws=A + 2) == E
    assert backward(q=grads(dy=None)) == E and backward(q=grads(dx=None)) == E and backward(q=grads(x=None)) == E
    assert backward(q=grads(dx=2 * A)) == E                                  # dx must not be x
    assert backward(q=grads(dweight=5 * A + 2)) == E
    assert backward(tokens=-1) == E
    assert backward(q=grads(weight=None, x=None, dweight=None), tokens=0) == g.GPTQ_OK


def cache(k=A, v=A, ks=A, vs=A, pages=8, kv_heads=2, block=64, dim=128):
    return attn.gptq_kv_cache(k, v, ks, vs, pages, kv_heads, block, dim)


def batch(start=A, length=A, table=A, stride=4, n=2, total=6, max_new=4, max_kv=256):
    return attn.gptq_kv_batch(start, length, table, stride, n, total, max_new, max_kv)


def append(c=None, b=None, k=A, v=A, strides=(256, 128, 256, 128), dtype=0, weight=None, r=None, status=None):
    return g.lib().gptq_kv_append(c if c is not None else cache(), b if b is not None else batch(), k, strides[0],
                                  strides[1], v, strides[2], strides[3], dtype, weight, r, status, None)


BAD_CACHES = [(dict(block=48), "U"), (dict(block=8), "U"), (dict(block=0), "E"), (dict(dim=96), "U"),
              (dict(dim=-1), "E"), (dict(kv_heads=0), "E"), (dict(pages=-1), "E"), (dict(pages=0), "E"),
              (dict(k=A + 8), "E"), (dict(v=None), "E"), (dict(ks=None), "E"), (dict(vs=A + 2), "E")]
BAD_BATCHES = [dict(start=None), dict(length=None), dict(table=None), dict(start=A + 1), dict(length=A + 2),
               dict(table=A + 2), dict(stride=3), dict(n=-1), dict(total=-1), dict(max_new=-1), dict(max_kv=-1)]
EMPTY_BATCHES = [dict(n=0), dict(total=0), dict(max_new=0)]


@pytest.mark.parametrize("bad,how", BAD_CACHES)
def test_cache_refusals(bad, how):
    want = g.GPTQ_EUNSUPPORTED if how == "U" else g.GPTQ_EINVAL
    assert append(c=cache(**bad)) == want
    assert read(c=cache(**bad)) == want
    assert attention(c=cache(**bad)) == want


@pytest.mark.parametrize("bad", BAD_BATCHES)
def test_batch_refusals(bad):
    assert append(b=batch(**bad)) == g.GPTQ_EINVAL
    assert read(b=batch(**bad)) == g.GPTQ_EINVAL
    assert attention(b=batch(**bad)) == g.GPTQ_EINVAL


@pytest.mark.parametrize("empty", EMPTY_BATCHES)
def test_empty_batches_do_nothing(empty):
    assert append(b=batch(**empty)) == g.GPTQ_OK
    assert read(b=batch(**empty)) == g.GPTQ_OK
    assert attention(b=batch(**empty)) == g.GPTQ_OK


def test_append_refusals():
    E = g.GPTQ_EINVAL
    assert append(k=None) == E and append(v=None) == E and append(k=A + 1) == E
    assert append(dtype=3) == E
    assert append(weight=A) == E                       # a norm without its eps
    assert append(weight=A + 1, r=rope()) == E
    assert append(r=rope(rot=24)) == g.GPTQ_EUNSUPPORTED
    assert append(r=rope(rot=144)) == E
    assert append(strides=(1 << 41, 128, 256, 128)) == E
    assert append(status=A + 1) == E
    big = batch(n=1 << 24, total=1 << 24, max_new=1024, max_kv=256)
    assert append(b=big) == g.GPTQ_EUNSUPPORTED


def read(c=None, b=None, k=A, v=A, dtype=0):
    return g.lib().gptq_kv_read(c if c is not None else cache(), b if b is not None else batch(), k, 256, 128, v, 256,
                                128, dtype, None, None)


def test_read_refusals():
    assert read(k=None, v=None) == g.GPTQ_OK
    assert read(k=A + 1) == g.GPTQ_EINVAL and read(v=A + 1) == g.GPTQ_EINVAL and read(dtype=2) == g.GPTQ_EINVAL


def attention(c=None, b=None, q=A, out=2 * A, lse=None, dtype=0, q_heads=4, scale=0.1, causal=1, window=0, ws=A,
              ws_bytes=1 << 40, status=None):
    return g.lib().gptq_kv_attention(c if c is not None else cache(), b if b is not None else batch(),
                                     attn.gptq_attention(q_heads, scale, causal, window), q, 512, 128, out, 512, 128,
                                     lse, dtype, ws, ws_bytes, status, None)


def test_attention_refusals():
    E = g.GPTQ_EINVAL
    assert attention(q=None) == E and attention(out=None) == E and attention(out=A) == E
    assert attention(q=A + 1) == E and attention(lse=A + 2) == E and attention(status=A + 2) == E
    assert attention(dtype=5) == E
    assert attention(q_heads=3) == E and attention(q_heads=0) == E
    assert attention(scale=float("inf")) == E and attention(scale=float("nan")) == E
    assert attention(causal=2) == E and attention(window=-1) == E
    long = batch(n=1, total=1, max_new=1, max_kv=100000, stride=2000)
    need = int(g.lib().gptq_kv_attention_workspace_bytes(cache(), long, 0, attn.gptq_attention(4, 0.1, 1, 0)))
    assert need > 0
    assert attention(b=long, ws_bytes=need - 1) == g.GPTQ_EWORKSPACE
    assert attention(b=long, ws=None) == g.GPTQ_EWORKSPACE
    assert attention(b=long, ws=A + 8, ws_bytes=need) == E
    assert attention(b=batch(n=1 << 20, total=1 << 20, max_new=1 << 20, max_kv=256)) == g.GPTQ_EUNSUPPORTED


def test_binding_refusals():
    """The binding's own checks (shapes, types, devices) need no device."""
    import torch
    x = torch.zeros((3, 4, 128), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        g.gptq_qk_norm_rope(x, None, None, attn.Rope(None, None))  # not on a device
    with pytest.raises(ValueError):
        g.gptq_qk_norm_rope(None, None, None, attn.Rope(None, None))
    with pytest.raises(ValueError):
        attn.Rope(torch.zeros((4, 8)), torch.zeros((4, 7)))
    with pytest.raises(ValueError):
        attn.KVCache.empty(2, 2, 64, 128, "cpu")
    with pytest.raises(ValueError):
        attn.KVBatch(torch.zeros(3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32),
                     torch.zeros((2, 4), dtype=torch.int32), 2, 1, 4)


def test_header_is_plain_c(tmp_path):
    src = tmp_path / "user.c"
    src.write_text('#include "gptq_attn.h"\nint main(void) { gptq_kv_cache c = {0}; gptq_kv_batch b = {0};\n'
                   '  gptq_attention a = {32, 0.1f, 1, 0};\n'
                   '  return (int)gptq_kv_attention_workspace_bytes(&c, &b, GPTQ_BF16, &a); }\n')
    r = subprocess.run(["gcc", "-std=c99", "-Wall", "-Wextra", "-Werror", "-fsyntax-only", "-I",
                        os.path.dirname(HEADER), str(src)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
