"""GPU tests of gptq_kv_attention against the fp64 reference over the same codes and scales
(bounds: attnhelp.attention_bound)."""

import numpy as np
import pytest

from attnhelp import Paged, attention_bound, close, on_device, values
from gpuhelp import say, to_dev, torch_dev
from oracle import attn_ref as R

pytestmark = pytest.mark.gpu


def check(c, new, qh, bf16, causal=True, window=0, layout="plain", seed=31, qscale=1.0, sm_scale=None, lengths=None):
    """Runs one call with every output given, in the layout, and compares it with the reference."""
    import post_weight_quantization_03_amd as g
    torch, dev = torch_dev()
    rng = np.random.default_rng(seed)
    lengths = c.lengths if lengths is None else lengths
    plan, start = c.plan(new, lengths)
    q = values(rng, (int(start[-1]), qh, c.dim), bf16, qscale)
    out = on_device(np.full(q.shape, np.nan), bf16, layout)
    lse = torch.full(q.shape[:2], float("nan"), device=dev)
    st = to_dev(np.zeros(1, np.int32))
    g.gptq_kv_attention(on_device(q, bf16, layout), c.dev, plan, sm_scale, causal, window, out=out, lse=lse,
                        d_status=st)
    torch.cuda.synchronize()
    assert int(st) == 0
    scale = c.dim ** -0.5 if sm_scale is None else sm_scale
    got, got_lse = out.float().cpu().numpy(), lse.cpu().numpy()
    for b, n in enumerate(new):
        if n == 0:
            continue
        k, v = c.kv(b, lengths[b])
        rows = slice(start[b], start[b + 1])
        want, want_lse, more = R.attention(q[rows], k, v, scale, causal, window)
        more["lse"] = want_lse
        ob, lb = attention_bound(want, more, max(1, lengths[b]), c.dim, bf16, np.abs(v).max(initial=0))
        close(f"out[{b}]", got[rows], want, ob + 1e-38)
        empty = np.isneginf(want_lse)
        assert np.array_equal(np.isneginf(got_lse[rows]), empty)
        assert np.all(got[rows][empty] == 0)
        close(f"lse[{b}]", np.where(empty, 0, got_lse[rows]), np.where(empty, 0, want_lse), lb)
    return out, lse


LAYOUTS = ["plain", "slice", "odd", "heads first"]
FORMS = [
    # lengths, new, q heads, kv heads, dim, block
    ([1], [1], 1, 1, 64, 16),
    ([1, 2, 63, 64, 65], [1] * 5, 4, 4, 128, 64),
    ([43], [1], 32, 8, 128, 32),
    ([700, 3, 255, 256, 257], [1] * 5, 16, 1, 128, 16),
    ([300, 299], [1, 1], 14, 2, 64, 128),
    ([130, 18], [1, 1], 6, 2, 256, 64),
    ([90, 5, 31], [5, 5, 3], 12, 4, 64, 16),          # rows over two row tiles
    ([200, 64], [9, 2], 21, 3, 128, 32),              # 63 rows: two wide row tiles
    ([333], [25], 6, 2, 256, 16),
    ([150, 70, 64], [70, 70, 1], 4, 4, 128, 64),      # prompts: whole, of different lengths
    ([500, 131], [131, 131], 6, 2, 64, 128),          # chunks over earlier tokens, 393 rows
    ([300], [100], 4, 2, 256, 32),
    ([129, 40], [129, 0], 2, 1, 128, 16),             # a sequence without new tokens
    ([600, 257], [300, 257], 3, 1, 128, 128),         # 900 rows of one key head
]


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("mask", [(True, 0), (False, 0), (True, 20), (False, 70), (True, 1)])
def test_against_reference(form, bf16, mask):
    lengths, new, qh, kh, dim, block = form
    say(f"attention {form} bf16={bf16} mask={mask}")
    rng = np.random.default_rng(41)
    c = Paged(rng, lengths, kh, block, dim)
    i = FORMS.index(form) + 2 * bf16
    check(c, new, qh, bf16, *mask, layout=LAYOUTS[i % 4])


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("form", [([5000, 40, 1300], [1, 1, 1], 4, 2, 128, 64), ([3000], [2], 8, 8, 64, 16),
                                  ([2100, 10], [40, 10], 4, 1, 128, 32), ([1600], [4], 2, 1, 256, 128),
                                  ([2500, 90], [70, 70], 4, 2, 64, 128), ([3000, 700], [150, 20], 4, 2, 128, 64),
                                  ([900, 5000, 140], [130, 90, 140], 2, 2, 128, 16)])
def test_split_sequences(form, bf16):
    """Lengths that are split over workgroups and joined, with short ones in the same call."""
    lengths, new, qh, kh, dim, block = form
    say(f"split attention {form} bf16={bf16}")
    rng = np.random.default_rng(42)
    c = Paged(rng, lengths, kh, block, dim)
    import post_weight_quantization_03_amd as g
    plan, _ = c.plan(new)
    assert g.gptq_kv_attention_workspace_bytes(c.dev, plan, qh, g.GPTQ_BF16 if bf16 else g.GPTQ_F32) > 0
    a = check(c, new, qh, bf16)
    b = check(c, new, qh, bf16)
    torch, _ = torch_dev()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])  # the same bits run to run
    check(c, new, qh, bf16, window=700)


@pytest.mark.parametrize("new", [1, 5, 40, 200])
def test_rows_that_see_nothing(new):
    """More new tokens than the sequence holds, and empty sequences: rows without any token."""
    rng = np.random.default_rng(43)
    c = Paged(rng, [max(1, new // 2), 300, 1], 2, 16, 128)
    for bf16 in (True, False):
        check(c, [new] * 3, 4, bf16, lengths=[new // 2, 300, 0])
        check(c, [new] * 3, 4, bf16, causal=False, window=3, lengths=[new // 2, 0, 1])


@pytest.mark.parametrize("new", [1, 90])
@pytest.mark.parametrize("sm_scale", [0.0, -0.2, 3.0, 1e-30])
def test_score_scales(new, sm_scale):
    rng = np.random.default_rng(44)
    c = Paged(rng, [150], 2, 64, 64)
    check(c, [new], 2, True, sm_scale=sm_scale)
    check(c, [new], 2, False, sm_scale=sm_scale)


@pytest.mark.parametrize("new", [1, 90])
@pytest.mark.parametrize("qscale", [1e-30, 1e30, 0.0])
def test_query_sizes(new, qscale):
    """Queries far from 1 keep their digits; the softmax scale brings the scores back."""
    rng = np.random.default_rng(45)
    c = Paged(rng, [150], 2, 64, 64)
    sm = 0.125 / qscale if qscale else 1.0
    check(c, [new], 2, True, qscale=qscale, sm_scale=sm)
    check(c, [new], 2, False, qscale=qscale, sm_scale=sm)


@pytest.mark.parametrize("new", [1, 3, 90])
def test_wide_ranges_of_scores(new):
    """One key that dominates after many that do not, and the other way round."""
    import post_weight_quantization_03_amd as g
    torch, dev = torch_dev()
    rng = np.random.default_rng(46)
    for order in (1, -1):
        c = Paged(rng, [640], 1, 16, 64, spread=1.0)
        ramp = 2.0 ** np.linspace(-30, 6, 40)[::order]
        for b in range(40):
            c.ref.k_scales[c.table[0, b]] = 2.0 ** np.round(np.log2(ramp[b]))
            c.ref.v_scales[c.table[0, b]] = 2.0 ** np.round(np.log2(ramp[39 - b]))
        c.dev.k_scales.copy_(to_dev(c.ref.k_scales.astype(np.float32)))
        c.dev.v_scales.copy_(to_dev(c.ref.v_scales.astype(np.float32)))
        check(c, [new], 2, True, sm_scale=0.01)
        check(c, [new], 2, False, sm_scale=0.01)


@pytest.mark.parametrize("new", [1, 12, 100])
@pytest.mark.parametrize("which", ["k", "v"])
def test_nan_scales_reach_just_the_rows_that_see_their_block(new, which):
    """A block whose scale is NaN makes NaN of every row that sees a token of it, and of no other,
    wherever the block ends inside a tile."""
    import post_weight_quantization_03_amd as g
    torch, dev = torch_dev()
    rng = np.random.default_rng(47)
    c = Paged(rng, [200], 2, 16, 64)
    q = values(rng, (new, 4, 64), True)
    plan, _ = c.plan([new])
    # the window leaves some rows without the block's 16 tokens, the causal end others
    args = dict(window=60)
    good = g.gptq_kv_attention(on_device(q, True), c.dev, plan, **args)
    block = (200 - new) // 16 if new > 1 else 10
    page = int(c.table[0, block])
    getattr(c.dev, which + "_scales")[page, 0] = float("nan")
    got = g.gptq_kv_attention(on_device(q, True), c.dev, plan, **args)
    for i in range(new):
        p = 200 - new + i
        sees = block * 16 <= p and block * 16 + 15 > p - 60
        for h in range(4):
            if sees and h < 2:
                assert torch.isnan(got[i, h]).all()
            else:
                assert torch.equal(got[i, h], good[i, h])


@pytest.mark.parametrize("new", [1, 100])
def test_queries_that_are_not_finite_stay_in_their_row(new):
    import post_weight_quantization_03_amd as g
    torch, dev = torch_dev()
    rng = np.random.default_rng(48)
    c = Paged(rng, [200, 150], 2, 32, 128)
    q = values(rng, (2 * new, 4, 128), True)
    plan, _ = c.plan([new, new])
    good = g.gptq_kv_attention(on_device(q, True), c.dev, plan)
    x = on_device(q, True)
    x[0, 1, 3] = float("nan")
    x[new, 2, 0] = float("inf")
    got = g.gptq_kv_attention(x, c.dev, plan)
    assert torch.isnan(got[0, 1]).all() and torch.isnan(got[new, 2]).all()
    keep = torch.ones((2 * new, 4), dtype=torch.bool, device=dev)
    keep[0, 1] = keep[new, 2] = False
    assert torch.equal(got[keep], good[keep])


@pytest.mark.parametrize("new", [1, 100])
def test_rows_of_nobody_and_values_past_the_end_are_left_alone(new):
    """Rows that no sequence owns keep what they hold; codes, scales and table entries past a
    sequence's end have no influence."""
    import post_weight_quantization_03_amd as g
    torch, dev = torch_dev()
    rng = np.random.default_rng(49)
    c = Paged(rng, [133], 2, 64, 128)
    q = on_device(values(rng, (new + 9, 4, 128), True), True)
    plan, _ = c.plan([new], total=new + 9)
    out = torch.full_like(q, 7.0)
    lse = torch.full(q.shape[:2], 7.0, device=dev)
    g.gptq_kv_attention(q, c.dev, plan, out=out, lse=lse)
    assert torch.all(out[new:] == 7.0) and torch.all(lse[new:] == 7.0)
    last = int(c.table[0, 2])
    c.dev.k_codes[last, :, 5:] = 99
    c.dev.v_codes[last, :, 0, :, 5:] = -128
    c.dev.v_codes[last, :, 1:] = -128
    again = torch.full_like(q, 7.0)
    g.gptq_kv_attention(q, c.dev, plan, out=again)
    assert torch.equal(out, again)


@pytest.mark.parametrize("new", [1, 100])
def test_bad_tables_and_lengths_are_raised_and_hurt_no_other_sequence(new):
    import post_weight_quantization_03_amd as g
    torch, dev = torch_dev()
    rng = np.random.default_rng(50)
    c = Paged(rng, [150, 150], 2, 32, 64)
    q = on_device(values(rng, (2 * new, 4, 64), True), True)
    plan, _ = c.plan([new, new])
    good = g.gptq_kv_attention(q, c.dev, plan)
    for what, value in (("page", c.dev.pages), ("page", -1), ("page", 2 ** 31 - 1), ("length", 100000), ("length", -1)):
        table, length = c.table.copy(), np.array([150, 150], np.int32)
        if what == "page":
            table[0, 1] = value
        else:
            length[0] = value
        bad = g.KVBatch(plan.q_start, to_dev(length), to_dev(table), 2 * new, new, 150)
        st = to_dev(np.zeros(1, np.int32))
        got = g.gptq_kv_attention(q, c.dev, bad, d_status=st)
        assert int(st) == g.GPTQ_EINVAL
        assert torch.equal(got[new:], good[new:])


def test_another_stream_and_a_captured_graph():
    """The call on a stream of its own, and recorded in a graph whose replays follow lengths that
    change on the device."""
    import post_weight_quantization_03_amd as g
    torch, dev = torch_dev()
    rng = np.random.default_rng(51)
    c = Paged(rng, [3000], 2, 64, 128)
    q = on_device(values(rng, (1, 8, 128), True), True)
    start, length = to_dev(np.array([0, 1], np.int32)), to_dev(np.array([3000], np.int32))
    plan = g.KVBatch(start, length, to_dev(c.table), 1, 1, 3000)
    ws = torch.empty(g.gptq_kv_attention_workspace_bytes(c.dev, plan, 8, g.GPTQ_BF16), dtype=torch.uint8, device=dev)
    want = {}
    for n in (3000, 17, 1500):
        length.fill_(n)
        want[n] = g.gptq_kv_attention(q, c.dev, plan).clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = g.gptq_kv_attention(q, c.dev, plan, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want[1500])
    out = torch.empty_like(q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g.gptq_kv_attention(q, c.dev, plan, out=out, workspace=ws)
    for n in (17, 3000, 1500, 3000):
        length.fill_(n)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[n]), n
        assert torch.equal(g.gptq_kv_attention(q, c.dev, plan), want[n])


def test_cache_beyond_two_gibibytes():
    """Pages whose codes lie past 2^31 bytes, and a sequence over them that is split."""
    import post_weight_quantization_03_amd as g
    torch, dev = torch_dev()
    rng = np.random.default_rng(52)
    c = Paged(rng, [1000], 8, 64, 128)
    pages = (1 << 31) // (8 * 64 * 128) + 40
    big = g.KVCache.empty(pages, 8, 64, 128, dev)
    used = torch.from_numpy(c.table[0, :16].astype(np.int64)).to(dev)
    moved = used + (pages - c.dev.pages)
    for name in ("k_codes", "v_codes", "k_scales", "v_scales"):
        getattr(big, name)[moved] = getattr(c.dev, name)[used]
    for new in (1, 130):
        q = on_device(values(rng, (new, 8, 128), True), True)
        plan, _ = c.plan([new])
        far = g.KVBatch(plan.q_start, plan.kv_len, moved.to(torch.int32)[None], new, new, 1000)
        assert torch.equal(g.gptq_kv_attention(q, c.dev, plan), g.gptq_kv_attention(q, big, far))
