"""The attention operators' plans on the host (no GPU): workspace sizes and refusals at the ends of
the arguments' ranges.  Pointers passed here are never dereferenced."""

import pytest

import post_weight_quantization_03_amd as g
from post_weight_quantization_03_amd import attn

A = 0x1000  # an aligned address that is not used


def cache(kv_heads=8, block=64, dim=128, pages=1 << 20):
    return attn.gptq_kv_cache(A, A, A, A, pages, kv_heads, block, dim)


def batch(n=1, total=1, max_new=1, max_kv=131035, block=64):
    return attn.gptq_kv_batch(A, A, A, -(-max_kv // block), n, total, max_new, max_kv)


def workspace(c, b, q_heads=32, dtype=0, causal=1, window=0):
    return int(g.lib().gptq_kv_attention_workspace_bytes(c, b, dtype, attn.gptq_attention(q_heads, 0.1, causal, window)))


SIZES = [dict(), dict(n=4, total=2000, max_new=500, max_kv=12001), dict(total=4096, max_new=4096, max_kv=4096),
         dict(n=2, total=80, max_new=40, max_kv=3000)]


@pytest.mark.parametrize("sizes", SIZES)
@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("causal", [0, 1])
def test_a_window_as_long_as_the_sequences_is_no_window(sizes, dtype, causal):
    """The workspace holds the splits of what is seen: every window from max_kv on sees all."""
    want = workspace(cache(), batch(**sizes), dtype=dtype, causal=causal)
    for window in (batch(**sizes).max_kv, 1 << 31, 1 << 62, (1 << 63) - 1 - batch(**sizes).max_new, (1 << 63) - 1):
        assert workspace(cache(), batch(**sizes), dtype=dtype, causal=causal, window=window) == want


def attend(c, b, q_heads, ws_bytes=(1 << 64) - 1):
    return g.lib().gptq_kv_attention(c, b, attn.gptq_attention(q_heads, 0.1, 1, 0), A, 128, 128, 2 * A, 128, 128, None,
                                     0, A, ws_bytes, None, None)


BIG = 1 << 30


@pytest.mark.parametrize("n,max_new,q_heads,kv_heads,max_kv", [
    (BIG, BIG, 65536, 1, 64),            # 2^68 workgroups: 0 in 64 bits
    (BIG, BIG, 65536, 65536, 64),
    ((1 << 29) + 1, BIG, 65536, 1, 64),
    (BIG, BIG, 65536, 1, 1 << 20),       # the same with splits
    (BIG, BIG - 256, 49152, 1, 64),
])
def test_calls_past_what_a_launch_holds_are_refused(n, max_new, q_heads, kv_heads, max_kv):
    assert attend(cache(kv_heads), batch(n, BIG, max_new, max_kv), q_heads) == g.GPTQ_EUNSUPPORTED


def norm_rope(tokens, max_pos, backward=False, rot=64):
    r = attn.gptq_rope(A, A, max_pos, rot, 0, 1e-6)
    if backward:
        side = attn.gptq_heads_grad(A, 512, 128, 2 * A, 512, 128, 3 * A, 512, 128, None, None, 4)
        return g.lib().gptq_qk_norm_rope_backward(side, None, 0, tokens, 128, A, r, None, 0, None, None)
    return g.lib().gptq_qk_norm_rope(attn.gptq_heads(A, 512, 128, 2 * A, 512, 128, None, 4), None, 0, tokens, 128, A, r,
                                     None, None)


@pytest.mark.parametrize("backward", [False, True])
def test_tables_without_positions_are_refused(backward):
    """No position is in range of cos and sin without rows, nor is there a row to read in its place."""
    assert norm_rope(3, 0, backward) == g.GPTQ_EINVAL
    assert norm_rope(0, 0, backward) == g.GPTQ_OK


def test_a_side_without_heads_needs_no_workspace():
    """Its weight's gradient is zero; the other side's gradients without a weight need no sums.  (No tokens, so
    that the call ends on the host unless the zero is asked for.)"""
    none = attn.gptq_heads_grad(None, 0, 0, None, 0, 0, None, 0, 0, A, None, 0)
    other = attn.gptq_heads_grad(A, 512, 128, None, 0, 0, 2 * A, 512, 128, None, None, 4)
    r = attn.gptq_rope(None, None, 0, 0, 0, 1e-6)
    assert g.lib().gptq_qk_norm_rope_backward(none, other, 0, 0, 128, None, r, None, 0, None, None) == g.GPTQ_OK
    none.dweight = A + 2
    assert g.lib().gptq_qk_norm_rope_backward(none, other, 0, 0, 128, None, r, None, 0, None, None) == g.GPTQ_EINVAL
