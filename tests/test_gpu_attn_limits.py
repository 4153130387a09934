"""GPU tests of the attention operators at the ends of their arguments' ranges."""

import numpy as np
import pytest

from attnhelp import Paged, on_device, values
from gpuhelp import say, torch_dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("new", [1, 5, 100])
@pytest.mark.parametrize("causal", [True, False])
def test_windows_longer_than_any_sequence(new, causal):
    """A window from max_kv on, up to the type's largest, gives the bits of no window, over a sequence that is
    split and one that holds fewer tokens than are new."""
    import post_weight_quantization_03_amd as g
    torch, _ = torch_dev()
    say(f"long windows, {new} new tokens, causal={causal}")
    rng = np.random.default_rng(61)
    c = Paged(rng, [5000, 300], 2, 32, 64)
    q = on_device(values(rng, (2 * new, 4, 64), True), True)
    plan, _ = c.plan([new, new], [5000, max(1, new // 2)])
    want, want_lse = g.gptq_kv_attention(q, c.dev, plan, causal=causal, want_lse=True)
    for window in (5000, (1 << 63) - 1 - new, (1 << 63) - 1):
        got, lse = g.gptq_kv_attention(q, c.dev, plan, causal=causal, window=window, want_lse=True)
        assert torch.equal(got, want) and torch.equal(lse, want_lse)
