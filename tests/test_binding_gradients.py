"""Derivatives and the operators' binding (no GPU): an operator without them refuses inputs that carry them, in reverse
and in forward mode, instead of returning outputs cut off from their inputs."""

import pytest

torch = pytest.importorskip("torch")

from torch.autograd import forward_ad  # noqa: E402

import post_weight_quantization_03_amd as g  # noqa: E402
from test_binding_devices import Tensor, arguments, cached, calls  # noqa: E402,F401


def tree(a):
    return g.KVTree(a["positions"], Tensor((3, 1), torch.int64))


def tokens():
    return g.Tokens(Tensor((3, 128), torch.int8), Tensor((3,), torch.float32), Tensor((3,), torch.int32), 64)


def product(x):
    """The product with x in the place of the layer's scales."""
    return g.gptq_int8_gemm(Tensor((4, 16), torch.int32), x, Tensor((4,), torch.uint8), tokens())


CALLS = {
    "quantize_tokens": lambda x, a: g.gptq_quantize_tokens(x),
    "int8_gemm": lambda x, a: product(x),
    "first tokens": lambda x, a: g.gptq_kv_attention(x, *cached(a), window=8, sinks=2),
    "tree": lambda x, a: g.gptq_kv_attention(x, *cached(a), tree=tree(a)),
}
FORWARD = CALLS | {
    "attention": lambda x, a: g.gptq_kv_attention(x, *cached(a)),
    "norm and rotation of q": lambda x, a: g.gptq_qk_norm_rope(x, None, a["positions"], g.Rope(a["cos"], a["sin"])),
    "norm and rotation of k": lambda x, a: g.gptq_qk_norm_rope(leaf(), x, a["positions"], g.Rope(a["cos"], a["sin"])),
    "norm and rotation, a weight": lambda x, a: g.gptq_qk_norm_rope(leaf(), None, a["positions"],
                                                                    g.Rope(a["cos"], a["sin"]), x),
}


def leaf(**more):
    return torch.ones((3, 4, 64), dtype=torch.bfloat16, **more)


@pytest.mark.parametrize("name", CALLS)
def test_inputs_that_require_gradients_are_refused(calls, name):  # noqa: F811
    x = leaf(requires_grad=True)
    with pytest.raises(ValueError, match="no gradients"):
        CALLS[name](x, arguments())
    assert calls == []
    for harmless in (x.detach(), x):  # refused for something else
        with torch.no_grad(), pytest.raises(ValueError, match="device"):
            CALLS[name](harmless, arguments())


@pytest.mark.parametrize("name", FORWARD)
def test_dual_tensors_are_refused(calls, name):  # noqa: F811
    with forward_ad.dual_level():
        x = forward_ad.make_dual(leaf(), leaf())
        for mode in (torch.enable_grad, torch.no_grad):
            with mode(), pytest.raises(ValueError, match="no gradients|forward"):
                FORWARD[name](x, arguments())
        assert calls == []
        for harmless in (leaf(), forward_ad.unpack_dual(x).primal):
            with pytest.raises(ValueError, match="device"):
                FORWARD[name](harmless, arguments())
        with torch.inference_mode(), pytest.raises(ValueError, match="device"):  # carries nothing on
            FORWARD[name](x, arguments())


def test_other_calls_are_made(calls):  # noqa: F811
    a = arguments()
    g.gptq_kv_attention(a["q"], *cached(a), window=8, sinks=2)
    g.gptq_kv_attention(a["q"], *cached(a), tree=tree(a))
    assert [c[0] for c in calls] == ["gptq_kv_masked_attention"] * 2


def test_attention_without_a_mask_takes_inputs_that_require_gradients(calls):  # noqa: F811
    a = arguments()
    a["q"].requires_grad = True
    g.gptq_kv_attention(a["q"], *cached(a))
    assert [c[0] for c in calls] == ["gptq_kv_attention"]
