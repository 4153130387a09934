"""GPU tests of the 8-bit product's kernels over many stages, each with its buffers used over and over: all bits
against the integer reference, outputs beside them left as they were, and the same bits from calls in a row.  Which kernel
a size takes is checked in test_int8_plan.py."""

import numpy as np
import pytest

from gpuhelp import say, to_dev, torch_dev
from int8forms import LONG, random_size
from oracle import int8_ref as R

pytestmark = pytest.mark.gpu
SEEDS = range(50)


def run(seed, tokens, rows, cols, bf16, calls=1):
    """A product of random codes into the middle of a wider Y, `calls` times over; compared bit for bit."""
    import post_weight_quantization_03_amd as g
    torch, dev = torch_dev()
    rng = np.random.default_rng(seed)
    w = rng.integers(0, 256, (rows, cols), dtype=np.uint8)
    ws = rng.uniform(1e-3, 2e-3, rows).astype(np.float32)
    wz = rng.integers(0, 256, rows, dtype=np.uint8)
    x = rng.standard_normal((tokens, cols)).astype(np.float32)
    q = g.gptq_quantize_tokens(to_dev(x))
    codes, scales, sums = R.quantize_tokens(x)
    assert np.array_equal(q.codes.cpu().numpy()[:, :cols], codes) and np.array_equal(q.sums.cpu().numpy(), sums)
    dt = torch.bfloat16 if bf16 else torch.float32
    want = torch.full((tokens + 1, rows + 3), 7.0, dtype=dt)
    want[:-1, 1:-2] = torch.from_numpy(R.product(codes, scales, w, ws, wz)).to(dt)
    args = to_dev(w).view(torch.int32), to_dev(ws), to_dev(wz)
    for _ in range(calls):
        Y = torch.full((tokens + 1, rows + 3), 7.0, dtype=dt, device=dev)
        g.gptq_int8_gemm(*args, q, Y[:-1, 1:-2])
        got = Y.cpu()
        wrong = int((got != want).sum())
        assert wrong == 0, f"{wrong} values differ, first at {(got != want).nonzero()[0].tolist()}"


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("tokens,rows,cols", LONG)
def test_long_products(tokens, rows, cols, bf16):
    say(f"product {tokens} x {rows} x {cols} bf16={bf16} ({LONG[tokens, rows, cols]})")
    run(tokens + rows + cols, tokens, rows, cols, bf16, calls=3)


@pytest.mark.parametrize("seed", SEEDS)
def test_sizes_over_the_whole_range(seed):
    tokens, rows, cols = random_size(seed)
    say(f"product {tokens} x {rows} x {cols}")
    run(seed, tokens, rows, cols, bool(seed % 2))
