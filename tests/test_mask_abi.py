"""The masked attention's C ABI and binding on the host (no GPU): exported symbols, argument errors before
any device work, tensors of two devices, plans.  Pointers passed here are never dereferenced."""

import ctypes
import os
import re
import subprocess

import pytest

import post_weight_quantization_03_amd as g
from post_weight_quantization_03_amd import attn
from test_binding_devices import Tensor, arguments, cached, calls  # noqa: F401

HEADER = os.path.join(os.path.dirname(os.path.dirname(__file__)), "include", "gptq_mask.h")
A = 0x1000  # an aligned address that is not used
E, U, OK = g.GPTQ_EINVAL, g.GPTQ_EUNSUPPORTED, g.GPTQ_OK


def test_every_declared_symbol_is_exported():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(gptq_[a-z0-9_]+)\s*\(", text))
    assert names == {"gptq_kv_masked_attention", "gptq_kv_masked_attention_workspace_bytes", "gptq_kv_tree"}
    for lib in (g.lib(), ctypes.CDLL(os.path.join(os.path.dirname(g.LIB_PATH), "libgptq_trace.so"))):
        for n in names:
            assert hasattr(lib, n), n
    assert callable(g.gptq_kv_tree)


def test_header_is_plain_c(tmp_path):
    src = tmp_path / "user.c"
    src.write_text('#include "gptq_mask.h"\nint main(void) { gptq_kv_cache c = {0}; gptq_kv_batch b = {0};\n'
                   '  gptq_attention a = {32, 0.1f, 1, 64}; gptq_kv_mask m = {4, 0, 0, 0};\n'
                   '  return (int)gptq_kv_masked_attention_workspace_bytes(&c, &b, GPTQ_BF16, &a, &m); }\n')
    r = subprocess.run(["gcc", "-std=c99", "-Wall", "-Wextra", "-Werror", "-fsyntax-only", "-I",
                        os.path.dirname(HEADER), str(src)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


def cache(dim=128, block=64, heads=4, pages=10):
    return attn.gptq_kv_cache(A, A, A, A, pages, heads, block, dim)


def batch(n=2, total=8, max_new=4, max_kv=300, stride=5):
    return attn.gptq_kv_batch(A, A, A, stride, n, total, max_new, max_kv)


def masked(m, a=None, b=None, ws=A, ws_bytes=1 << 40, status=None):
    return g.lib().gptq_kv_masked_attention(cache(), b or batch(), a or attn.gptq_attention(8, 0.1, 1, 64), m, A, 1024,
                                            128, 2 * A, 1024, 128, None, 0, ws, ws_bytes, status, None)


def test_masked_attention_refusals():
    M = attn.gptq_kv_mask
    empty = batch(total=0)
    assert masked(M(4, None, 0, None), b=empty) == OK
    assert masked(None) == E
    assert masked(M(-1, None, 0, None)) == E
    assert masked(M(0, A, 0, A), b=empty) == E                   # too few words
    assert masked(M(0, A, 1 << 41, A), b=empty) == E
    assert masked(M(0, A, 1, A), b=empty) == OK
    assert masked(M(0, A, 1, A), b=batch(total=0, max_new=65)) == E
    assert masked(M(0, A, 2, A), b=batch(total=0, max_new=65)) == OK
    assert masked(M(0, A, 1, A), a=attn.gptq_attention(8, 0.1, 0, 64)) == E  # a tree is causal
    assert masked(M(0, A + 4, 1, A)) == E
    assert masked(M(0, A, 1, None)) == E                         # a window counts from positions
    assert masked(M(0, A, 1, A + 2)) == E
    assert masked(M(4, None, 0, None), a=attn.gptq_attention(7, 0.1, 1, 64)) == E
    assert masked(M(4, None, 0, None), a=attn.gptq_attention(8, float("nan"), 1, 64)) == E
    assert masked(M(4, None, 0, None), status=A + 2) == E
    long = batch(n=1, total=1, max_new=1, max_kv=100000, stride=2000)
    a, m = attn.gptq_attention(8, 0.1, 1, 50000), M(4, None, 0, None)
    need = int(g.lib().gptq_kv_masked_attention_workspace_bytes(cache(), long, 0, a, m))
    assert need > 0
    assert masked(m, a, long, ws_bytes=need - 1) == g.GPTQ_EWORKSPACE
    assert masked(m, a, long, ws=None) == g.GPTQ_EWORKSPACE
    assert masked(m, a, long, ws=A + 8, ws_bytes=need) == E
    many = batch(n=1 << 20, total=1 << 20, max_new=1 << 20, max_kv=256)
    assert masked(M(0, A, 1 << 20, A), attn.gptq_attention(8, 0.1, 1, 0), many) == U


def workspace(max_kv, window, sinks, tree=None, max_new=1, n=1):
    b = batch(n=n, total=n * max_new, max_new=max_new, max_kv=max_kv, stride=max_kv // 64 + 1)
    return int(g.lib().gptq_kv_masked_attention_workspace_bytes(
        cache(), b, 0, attn.gptq_attention(8, 0.1, 1, window), attn.gptq_kv_mask(sinks, tree, 1 << 20, A)))


def test_plans_follow_what_is_seen():
    """A window with sinks is planned for its own length, not the sequence's; without a window sinks are
    nothing; numbers near the ends of their ranges do not wrap."""
    long = 1 << 22
    whole = workspace(long, 0, 0)
    assert whole > 0 and workspace(long, 0, 1 << 62) == whole and workspace(long, 0, 7, A) == whole
    assert workspace(long, 1 << 62, 5) == whole and workspace(long, (1 << 63) - 1, (1 << 63) - 1) == whole
    assert workspace(long, 1000, 4) < whole
    assert workspace(long, 1000, long) == workspace(long, 1000, 1 << 62) == whole
    assert workspace(long, 1000, long - 1) == whole
    assert workspace(4096, 100, 70) == workspace(1 << 30, 100, 70)  # the same tokens


def tree(b=None, parents=A, window=0, sinks=0, positions=2 * A, words=3 * A, stride=1, status=None):
    return g.lib().gptq_kv_tree(b or batch(), parents, window, sinks, positions, words, stride, status, None)


def test_tree_refusals():
    assert tree(batch(total=0)) == OK
    assert tree(batch(n=0)) == OK
    assert tree(batch(max_new=0), stride=0) == OK
    assert g.lib().gptq_kv_tree(None, A, 0, 0, 2 * A, 3 * A, 1, None, None) == E
    assert tree(batch(n=-1)) == E
    assert tree(batch(total=-1)) == E
    assert tree(batch(max_kv=-1)) == E
    assert tree(window=-1) == E
    assert tree(sinks=-1) == E
    assert tree(stride=0) == E
    assert tree(batch(max_new=65)) == E
    assert tree(status=A + 1) == E
    for bad in (dict(parents=None), dict(parents=A + 2), dict(positions=None), dict(positions=A), dict(positions=A + 1),
                dict(words=None), dict(words=A + 4), dict(b=attn.gptq_kv_batch(None, A, A, 5, 2, 8, 4, 300)),
                dict(b=attn.gptq_kv_batch(A, None, A, 5, 2, 8, 4, 300))):
        assert tree(**bad) == E
    assert tree(batch(n=1 << 24, total=1 << 24)) == U
    assert tree(batch(n=1 << 16, total=1 << 20, max_new=256 * 256 + 1), stride=1025) == U
    assert tree(batch(total=1 << 25, max_new=65535 * 256 + 1), stride=1 << 18) == U


def binding_arguments(odd=None):
    import torch
    a = arguments(odd)

    def t(name, shape, dtype):
        return Tensor(shape, dtype, 0 if name == odd else 1)
    a["parents"] = t("parents", (3,), torch.int32)
    a["places"], a["mask"] = t("places", (3,), torch.int32), t("mask", (3, 1), torch.int64)
    return a


def made(a, window=None, sinks=None):
    return g.KVTree(a["places"], a["mask"], window, sinks)


CALLS = {
    "gptq_kv_masked_attention": (("q", "out", "lse", "workspace", "codes", "table", "status", "mask", "places"),
                                 lambda a: g.gptq_kv_attention(a["q"], *cached(a), out=a["out"], lse=a["lse"],
                                                               workspace=a["workspace"], d_status=a["status"], window=9,
                                                               sinks=2, tree=made(a))),
    "gptq_kv_tree": (("parents", "mask", "places", "start", "len", "status"),
                     lambda a: g.gptq_kv_tree(cached(a)[1], a["parents"], out=made(a), d_status=a["status"])),
}


@pytest.mark.parametrize("name", CALLS)
def test_the_call_is_made_on_its_tensors_device(calls, name):  # noqa: F811
    CALLS[name][1](binding_arguments())
    assert calls == [(name, 1)]


@pytest.mark.parametrize("name,odd", [(n, o) for n in CALLS for o in CALLS[n][0]])
def test_tensors_of_two_devices_are_refused(calls, name, odd):  # noqa: F811
    with pytest.raises(ValueError, match="one device"):
        CALLS[name][1](binding_arguments(odd))
    assert calls == []


def test_calls_without_a_mask_are_the_plain_ones(calls):  # noqa: F811
    a = binding_arguments()
    g.gptq_kv_attention(a["q"], *cached(a), out=a["out"], workspace=a["workspace"], window=9)
    g.gptq_kv_attention(a["q"], *cached(a), out=a["out"], workspace=a["workspace"], window=9, sinks=1)
    assert [c[0] for c in calls] == ["gptq_kv_attention", "gptq_kv_masked_attention"]


def test_trees_are_checked(calls):  # noqa: F811
    import torch
    a = binding_arguments()
    for tree_, window, sinks in ((made(a, 9, 2), 8, 2), (made(a, 9, 2), 9, 0), (made(a, 0, 0), 9, 0)):
        with pytest.raises(ValueError, match="made for"):
            g.gptq_kv_attention(a["q"], *cached(a), out=a["out"], window=window, sinks=sinks, tree=tree_)
    g.gptq_kv_attention(a["q"], *cached(a), out=a["out"], workspace=a["workspace"], window=9, sinks=2,
                        tree=made(a, 9, 2))
    b = g.KVBatch(a["start"], a["len"], a["table"], 3, 65, 40)  # needs two words
    with pytest.raises(ValueError):
        g.gptq_kv_attention(a["q"], cached(a)[0], b, out=a["out"], tree=made(a))
    with pytest.raises(ValueError):
        g.KVTree(a["places"], Tensor((3, 1), torch.int32))
    with pytest.raises(ValueError):
        g.KVTree(Tensor((2,), torch.int32), a["mask"])
    assert [c[0] for c in calls] == ["gptq_kv_masked_attention"]


SAME = [((0, 4), (0, 0)), ((0, 0), (0, 7)), ((40, 0), (0, 0)), ((1 << 40, 3), (50, 5)), ((9, 40), (0, 0)),
        ((9, 50), (8, 1 << 40)), ((9, None), (9, 0)), ((None, None), (9, 2))]
OTHER = [((39, 0), (0, 0)), ((9, 39), (9, 38)), ((9, 39), (0, 0)), ((9, None), (9, 1)), ((9, 1), (10, 1))]


@pytest.mark.parametrize("made_for,called_with", SAME)
def test_limits_that_mean_the_same_are_the_same(calls, made_for, called_with):  # noqa: F811
    """First tokens without a window, a window as long as any sequence (40) and first tokens that are all of them limit
    nothing."""
    a = binding_arguments()
    for one, two in ((made_for, called_with), (called_with, made_for)):
        if None not in two:
            g.gptq_kv_attention(a["q"], *cached(a), out=a["out"], workspace=a["workspace"], window=two[0],
                                sinks=two[1], tree=made(a, *one))
            assert calls.pop()[0] == "gptq_kv_masked_attention"


@pytest.mark.parametrize("made_for,called_with", OTHER)
def test_limits_that_differ_are_refused(calls, made_for, called_with):  # noqa: F811
    a = binding_arguments()
    with pytest.raises(ValueError, match="made for"):
        g.gptq_kv_attention(a["q"], *cached(a), out=a["out"], window=called_with[0], sinks=called_with[1],
                            tree=made(a, *made_for))
    assert calls == []
