"""GPU tests of masked attention over the cache (visible first tokens beside a window, trees of new
tokens) against the fp64 reference over the same codes and scales (bounds: attnhelp.attention_bound),
and of the trees' masks, which are compared bit for bit."""

import numpy as np
import pytest

from attnhelp import Paged, attention_bound, close, on_device, values
from gpuhelp import say, to_dev, torch_dev
from oracle import mask_ref as M

pytestmark = pytest.mark.gpu
LAYOUTS = ["plain", "slice", "odd", "heads first"]


def free_unseen(c, sees):
    """Table entries of blocks that no token of a sequence sees go out of range, as if given away."""
    freed = 0
    for b, s in enumerate(sees):
        for k in range(-(-s.shape[1] // c.block)):
            if s.shape[0] and not s[:, k * c.block:(k + 1) * c.block].any():
                c.table[b, k] = -9
                freed += 1
    return freed


def check(c, new, qh, bf16, sees, window=0, sinks=0, causal=True, tree=None, layout="plain", lengths=None, seed=31):
    """Runs a call with every output given and compares it with the reference; sees [n, length] of each
    sequence."""
    import post_weight_quantization_03_amd as g
    torch, dev = torch_dev()
    rng = np.random.default_rng(seed)
    lengths = c.lengths if lengths is None else lengths
    kv = [c.kv(b, lengths[b]) for b in range(len(new))]
    freed = free_unseen(c, sees)
    plan, start = c.plan(new, lengths)
    q = values(rng, (int(start[-1]), qh, c.dim), bf16)
    out = on_device(np.full(q.shape, np.nan), bf16, layout)
    lse = torch.full(q.shape[:2], float("nan"), device=dev)
    st = to_dev(np.zeros(1, np.int32))
    made = None if tree is None else tree(plan)
    g.gptq_kv_attention(on_device(q, bf16, layout), c.dev, plan, None, causal, window, out=out, lse=lse, d_status=st,
                        sinks=sinks, tree=made)
    torch.cuda.synchronize()
    assert int(st) == 0, f"status {int(st)} ({freed} blocks given away)"
    got, got_lse = out.float().cpu().numpy(), lse.cpu().numpy()
    for b, n in enumerate(new):
        if n == 0:
            continue
        k, v = kv[b]
        rows = slice(start[b], start[b + 1])
        want, want_lse, more = M.attention(q[rows], k, v, c.dim ** -0.5, sees[b])
        more["lse"] = want_lse
        ob, lb = attention_bound(want, more, max(1, lengths[b]), c.dim, bf16, np.abs(v).max(initial=0))
        close(f"out[{b}]", got[rows], want, ob + 1e-38)
        empty = np.isneginf(want_lse)
        assert np.array_equal(np.isneginf(got_lse[rows]), empty)
        assert np.all(got[rows][empty] == 0)
        close(f"lse[{b}]", np.where(empty, 0, got_lse[rows]), np.where(empty, 0, want_lse), lb)
    return out, lse


def windows(new, lengths, window, sinks, causal=True):
    return [M.window_sees(n, t, window, sinks, causal) for n, t in zip(new, lengths)]


# lengths, new, q heads, kv heads, dim, block: as in the plain attention's tests, few rows and prompts
FORMS = [
    ([1], [1], 1, 1, 64, 16),
    ([1, 2, 63, 64, 65], [1] * 5, 4, 4, 128, 64),
    ([700, 3, 255, 256, 257], [1] * 5, 16, 1, 128, 16),
    ([300, 299], [1, 1], 14, 2, 64, 128),
    ([330, 18], [1, 1], 6, 2, 256, 64),
    ([290, 5, 31], [5, 5, 3], 12, 4, 64, 16),
    ([400, 64], [9, 2], 21, 3, 128, 32),
    ([333], [25], 6, 2, 256, 16),
    ([450, 70, 64], [70, 70, 1], 4, 4, 128, 64),
    ([700, 131], [131, 131], 6, 2, 64, 128),
    ([500], [100], 4, 2, 256, 32),
    ([429, 40], [129, 0], 2, 1, 128, 16),
    ([600, 257], [300, 257], 3, 1, 128, 128),
]


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("mask", [(1, 1), (20, 4), (70, 64), (33, 65), (64, 130), (200, 1)])
def test_sinks(form, bf16, mask):
    lengths, new, qh, kh, dim, block = form
    window, sinks = mask
    say(f"sinks {form} bf16={bf16} window={window} sinks={sinks}")
    c = Paged(np.random.default_rng(41), lengths, kh, block, dim)
    i = FORMS.index(form) + 2 * bf16
    check(c, new, qh, bf16, windows(new, lengths, window, sinks), window, sinks, layout=LAYOUTS[i % 4])


@pytest.mark.parametrize("new", [1, 7, 90])
def test_sinks_without_causality(new):
    c = Paged(np.random.default_rng(42), [400, 95], 2, 32, 64)
    check(c, [new, new], 4, True, windows([new, new], [400, 95], 50, 10, False), 50, 10, causal=False)


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("form", [
    ([9000, 40, 5300], [1, 1, 1], 4, 2, 128, 64, 3000, 5), ([6000], [2], 8, 8, 64, 16, 2500, 700),
    ([5100, 10], [40, 10], 4, 1, 128, 32, 1900, 64), ([4600], [4], 2, 1, 256, 128, 1000, 1),
    ([5500, 3000], [70, 70], 4, 2, 64, 128, 2000, 4), ([6000, 700], [150, 20], 4, 2, 128, 64, 2100, 300)])
def test_sinks_of_split_sequences(form, bf16):
    lengths, new, qh, kh, dim, block, window, sinks = form
    say(f"split sinks {form} bf16={bf16}")
    import post_weight_quantization_03_amd as g
    torch, _ = torch_dev()
    got = []
    for _ in range(2):
        c = Paged(np.random.default_rng(43), lengths, kh, block, dim)
        plan, _ = c.plan(new)
        assert g.gptq_kv_attention_workspace_bytes(c.dev, plan, qh, g.GPTQ_BF16 if bf16 else g.GPTQ_F32, True, window,
                                                   sinks) > 0
        got.append(check(c, new, qh, bf16, windows(new, lengths, window, sinks), window, sinks))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])  # the same bits run to run


def test_sinks_without_a_window_change_nothing():
    import post_weight_quantization_03_amd as g
    torch, _ = torch_dev()
    rng = np.random.default_rng(44)
    for new in (1, 80):
        c = Paged(rng, [200, 150], 2, 16, 128)
        plan, start = c.plan([new, new])
        q = on_device(values(rng, (2 * new, 4, 128), True), True)
        a = g.gptq_kv_attention(q, c.dev, plan)
        for window, sinks in ((0, 7), (200, 7), (1 << 40, 1 << 40)):
            assert torch.equal(a, g.gptq_kv_attention(q, c.dev, plan, window=window, sinks=sinks))
        # all tokens are sinks: as without a window
        b = g.gptq_kv_attention(q, c.dev, plan, window=3, sinks=200)
        assert torch.allclose(a.float(), b.float(), rtol=2.0 ** -7, atol=1e-3)


@pytest.mark.parametrize("new", [1, 5, 40, 200])
def test_rows_that_see_nothing(new):
    """More new tokens than the sequence holds, and empty sequences."""
    for bf16 in (True, False):
        c = Paged(np.random.default_rng(45), [max(1, new // 2), 300, 1], 2, 16, 128)
        lengths = [new // 2, 300, 0]
        sees = []
        for t in lengths:
            p, j = np.arange(t - new, t)[:, None], np.arange(t)
            sees.append((j <= p) & ((j > p - 3) | (j < 2)))
        check(c, [new] * 3, 4, bf16, sees, 3, 2, lengths=lengths)


def random_parents(rng, n):
    """Any earlier token as often as one of the last three; -1: none."""
    return np.array([rng.integers(-1, i) if rng.random() < 0.5 else max(-1, i - 1 - rng.integers(0, 4))
                     for i in range(n)])


def trees(rng, new, lengths, window=0, sinks=0):
    parents = [random_parents(rng, n) for n in new]
    sees = []
    for p, n, t in zip(parents, new, lengths):
        at, among = M.tree(p, t - n, window, sinks)
        sees.append(M.tree_sees(at, among, t - n, window, sinks))
    return np.concatenate(parents).astype(np.int32), sees


TREES = [
    ([1], [1], 1, 1, 64, 16),
    ([713], [13], 8, 8, 128, 64),
    ([100, 64, 5, 200], [5, 64, 5, 1], 4, 4, 128, 16),
    ([300, 131], [60, 63], 4, 1, 64, 32),
    ([333, 128], [65, 0], 2, 2, 128, 128),
    ([500], [129], 2, 1, 256, 16),
    ([400, 260], [200, 255], 4, 2, 128, 32),
    ([700], [300], 6, 2, 64, 64),
    ([900], [33], 7, 1, 256, 64),
    ([350], [350], 2, 1, 128, 16),
]


@pytest.mark.parametrize("form", TREES)
@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("mask", [(0, 0), (100, 4), (7, 70), (1, 0)])
def test_trees(form, bf16, mask):
    import post_weight_quantization_03_amd as g
    lengths, new, qh, kh, dim, block = form
    say(f"tree {form} bf16={bf16} mask={mask}")
    rng = np.random.default_rng(50)
    c = Paged(rng, lengths, kh, block, dim)
    parents, sees = trees(rng, new, lengths, *mask)
    i = TREES.index(form) + 2 * bf16
    check(c, new, qh, bf16, sees, *mask, tree=lambda plan: g.gptq_kv_tree(plan, to_dev(parents), *mask),
          layout=LAYOUTS[i % 4])


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("form", [([5000, 2000], [13, 40], 4, 2, 128, 64), ([4000, 90], [70, 70], 4, 2, 64, 128),
                                  ([3000], [200], 4, 2, 128, 16)])
@pytest.mark.parametrize("mask", [(0, 0), (1500, 4)])
def test_trees_of_split_sequences(form, bf16, mask):
    import post_weight_quantization_03_amd as g
    lengths, new, qh, kh, dim, block = form
    rng = np.random.default_rng(51)
    c = Paged(rng, lengths, kh, block, dim)
    parents, sees = trees(rng, new, lengths, *mask)
    check(c, new, qh, bf16, sees, *mask, tree=lambda plan: g.gptq_kv_tree(plan, to_dev(parents), *mask))


@pytest.mark.parametrize("form", [
    ([5000, 90, 2000, 64, 3000], [70, 70, 1, 64, 30], 4, 2, 128, 64), ([700, 6000, 300], [200, 150, 0], 6, 2, 64, 16),
    ([40 + 37 * i for i in range(64)], [1 + i % 40 for i in range(64)], 4, 1, 64, 32),
    ([1500, 400], [90, 90], 4, 4, 256, 128), ([3000, 1], [140, 1], 4, 2, 128, 16)])
@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("mask", [(0, 0), (900, 4)])
def test_trees_of_unequal_sequences(form, bf16, mask):
    """Batches of very different lengths over the prompt kernel's splits: run to run the same bits."""
    import post_weight_quantization_03_amd as g
    lengths, new, qh, kh, dim, block = form
    say(f"unequal trees of {len(new)} sequences, dim {dim} bf16={bf16} mask={mask}")
    torch, _ = torch_dev()
    got = []
    for _ in range(2):
        rng = np.random.default_rng(58)
        c = Paged(rng, lengths, kh, block, dim)
        parents, sees = trees(rng, new, lengths, *mask)
        got.append(check(c, new, qh, bf16, sees, *mask, tree=lambda plan: g.gptq_kv_tree(plan, to_dev(parents), *mask)))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])


@pytest.mark.parametrize("new,qh", [(9, 2), (100, 2), (140, 4)])
def test_any_pattern(new, qh):
    """Masks that are no trees: later tokens, not oneself, nothing at all; wider rows than needed and bits
    past the new tokens."""
    import post_weight_quantization_03_amd as g
    torch, dev = torch_dev()
    rng = np.random.default_rng(52)
    length, n = [new + 77, new], -(-new // 64) + 1
    c = Paged(rng, length, 2, 16, 128)
    among = [rng.random((new, new)) < 0.4 for _ in range(2)]
    among[1][3] = False
    bits = np.concatenate([M.words(a, n) for a in among])
    noise = np.full(2 * n * 64, ~np.uint64(0), dtype=np.uint64)[:n]
    for w in range(n):  # every bit from `new` on
        lo = new - 64 * w
        noise[w] = 0 if lo >= 64 else np.uint64((2 ** 64 - 1) ^ ((1 << max(lo, 0)) - 1))
    wide = torch.zeros((2 * new, n + 2), dtype=torch.int64, device=dev)
    wide[:, :n] = to_dev((bits | noise).view(np.int64))
    tree = g.KVTree(torch.zeros(2 * new, dtype=torch.int32, device=dev), wide[:, :n])
    sees = [M.tree_sees(np.zeros(new), a, t - new) for a, t in zip(among, length)]
    for bf16 in (True, False):
        check(c, [new, new], qh, bf16, sees, tree=lambda plan: tree)


@pytest.mark.parametrize("new", [3, 80])
def test_rows_that_no_sequence_has_stay(new):
    import post_weight_quantization_03_amd as g
    torch, dev = torch_dev()
    rng = np.random.default_rng(60)
    c = Paged(rng, [500, 3000], 2, 16, 128)
    total = 2 * new + 5
    lens = to_dev(np.array([500, 3000], np.int32))
    plan = g.KVBatch(to_dev(np.array([2, 2 + new, 2 + 2 * new], np.int32)), lens, to_dev(c.table), total, new, 3000)
    q = on_device(values(rng, (total, 4, 128), True), True)
    tree = g.gptq_kv_tree(plan, torch.full((total,), -1, dtype=torch.int32, device=dev), 100, 4)
    for kw in ({"window": 100, "sinks": 4}, {"tree": g.gptq_kv_tree(plan, torch.full_like(tree.positions, -1))},
               {"window": 100, "sinks": 4, "tree": tree}):
        out, lse = torch.full_like(q, 7.0), torch.full((total, 4), 7.0, device=dev)
        g.gptq_kv_attention(q, c.dev, plan, out=out, lse=lse, **kw)
        apart = [0, 1, *range(2 + 2 * new, total)]
        assert (out[apart] == 7).all() and (lse[apart] == 7).all()
        assert not (lse[2:2 + 2 * new] == 7).any()


def test_a_chain_is_plain_attention():
    import post_weight_quantization_03_amd as g
    torch, dev = torch_dev()
    rng = np.random.default_rng(53)
    for n, window in ((6, 0), (6, 40), (150, 0), (150, 100)):
        c = Paged(rng, [n + 300], 2, 32, 128)
        plan, _ = c.plan([n])
        q = on_device(values(rng, (n, 4, 128), True), True)
        tree = g.gptq_kv_tree(plan, to_dev(np.arange(-1, n - 1, dtype=np.int32)), window)
        a = g.gptq_kv_attention(q, c.dev, plan, window=window)
        b = g.gptq_kv_attention(q, c.dev, plan, window=window, tree=tree)
        assert torch.allclose(a.float(), b.float(), rtol=2.0 ** -7, atol=1e-3)


@pytest.mark.parametrize("mask", [(0, 0), (5, 0), (3, 40), (1, 1), (64, 9), (100000, 3)])
@pytest.mark.parametrize("new,lengths", [([1], [1]), ([13, 0, 64, 65], [40, 7, 64, 300]), ([255, 1], [300, 10]),
                                         ([700, 129], [701, 2000])])
def test_tree_masks(new, lengths, mask):
    """Bit for bit; rows that no sequence has stay as they were."""
    import post_weight_quantization_03_amd as g
    torch, dev = torch_dev()
    rng = np.random.default_rng(54)
    parents = [random_parents(rng, n) for n in new]
    total, count = sum(new) + 3, -(-max(new) // 64)
    start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32) + 1
    batch = g.KVBatch(to_dev(start), to_dev(np.asarray(lengths, np.int32)), to_dev(np.zeros((len(new), 40), np.int32)),
                      total, max(new), max(lengths))
    words = torch.full((total, count + 1), 77, dtype=torch.int64, device=dev)
    out = g.KVTree(torch.full((total,), 55, dtype=torch.int32, device=dev), words[:, :count])
    st = to_dev(np.zeros(1, np.int32))
    flat = np.concatenate([[9], *parents, [9, 9]]).astype(np.int32)
    got = g.gptq_kv_tree(batch, to_dev(flat), *mask, out=out, d_status=st)
    assert got is out and int(st) == 0
    want_p, want_w = np.full(total, 55), np.full((total, count + 1), 77, dtype=np.int64)
    for b, (p, n, t) in enumerate(zip(parents, new, lengths)):
        at, among = M.tree(p, t - n, *mask)
        want_p[start[b]:start[b + 1]] = at
        want_w[start[b]:start[b + 1], :count] = M.words(among, count).view(np.int64)
    assert np.array_equal(out.positions.cpu().numpy(), want_p) and np.array_equal(words.cpu().numpy(), want_w)


@pytest.mark.parametrize("before", [0, 3, 200])
@pytest.mark.parametrize("mask", [(0, 0), (1, 0), (70, 5), (64, 64), (3, 130), (130, 1), (129, 300), (500, 9)])
def test_masks_of_long_paths(before, mask):
    """Chains over several words, with gaps, cut by window and first tokens inside and between words."""
    import post_weight_quantization_03_amd as g
    rng = np.random.default_rng(59)
    chain = np.arange(-1, 319)
    gaps = np.maximum(np.arange(320) - rng.integers(1, 4, 320), -1)
    far = np.where(np.arange(320) % 65 == 64, np.arange(320) - 64, chain)
    start = np.arange(0, 961, 320, dtype=np.int32)
    batch = g.KVBatch(to_dev(start), to_dev(np.full(3, before + 320, np.int32)), to_dev(np.zeros((3, 8), np.int32)),
                      960, 320, before + 320)
    got = g.gptq_kv_tree(batch, to_dev(np.concatenate([chain, gaps, far]).astype(np.int32)), *mask)
    for b, parents in enumerate((chain, gaps, far)):
        at, among = M.tree(parents, before, *mask)
        rows = slice(start[b], start[b + 1])
        assert np.array_equal(got.positions[rows].cpu().numpy(), at)
        assert np.array_equal(got.mask[rows].cpu().numpy(), M.words(among, 5).view(np.int64))


@pytest.mark.parametrize("mask", [(0, 0), (300, 5)])
def test_a_long_chain_of_drafts(mask):
    """More tokens than fit in LDS."""
    import post_weight_quantization_03_amd as g
    n = 9000
    batch = g.KVBatch(to_dev(np.array([0, n], np.int32)), to_dev(np.array([n + 2], np.int32)),
                      to_dev(np.zeros((1, 200), np.int32)), n, n, n + 2)
    parents = np.arange(-1, n - 1)
    parents[[8191, 8192, 8500]] = [8000, 8191, 17]
    got = g.gptq_kv_tree(batch, to_dev(parents.astype(np.int32)), *mask)
    at, among = M.tree(parents, 2, *mask)
    assert np.array_equal(got.positions.cpu().numpy(), at)
    assert np.array_equal(got.mask.cpu().numpy(), M.words(among, -(-n // 64)).view(np.int64))


def test_index_data_out_of_range():
    """Parents, positions and lengths out of range raise the status, and other sequences are as they were."""
    import post_weight_quantization_03_amd as g
    torch, dev = torch_dev()
    rng = np.random.default_rng(55)
    new, lengths = [4, 4, 4], [50, 60, 70]
    c = Paged(rng, lengths, 2, 16, 64)
    plan, _ = c.plan(new)
    good = np.array([-1, 0, 0, 1] * 3, np.int32)
    q = on_device(values(rng, (12, 4, 64), True), True)
    tree = g.gptq_kv_tree(plan, to_dev(good), 20, 2)
    want = g.gptq_kv_attention(q, c.dev, plan, window=20, sinks=2, tree=tree)
    for bad in (1, 2, 99, -2, 2 ** 31 - 1, -2 ** 31):
        st, p = to_dev(np.zeros(1, np.int32)), good.copy()
        p[5] = bad
        t = g.gptq_kv_tree(plan, to_dev(p), 20, 2, d_status=st)
        assert int(st) == g.GPTQ_EINVAL
        keep = [0, 1, 2, 3, 8, 9, 10, 11]
        assert torch.equal(t.mask[keep], tree.mask[keep]) and torch.equal(t.positions[keep], tree.positions[keep])
    for bad in (0, 55, 60, 2 ** 31 - 1, -2 ** 31):
        st, at = to_dev(np.zeros(1, np.int32)), tree.positions.clone()
        at[5] = bad
        got = g.gptq_kv_attention(q, c.dev, plan, window=20, sinks=2, tree=g.KVTree(at, tree.mask), d_status=st)
        assert int(st) == g.GPTQ_EINVAL
        keep = [0, 1, 2, 3, 4, 6, 7, 8, 9, 10, 11]
        assert torch.equal(got[keep], want[keep])
    st = to_dev(np.zeros(1, np.int32))
    short = g.KVBatch(plan.q_start, to_dev(np.array([50, 3, 70], np.int32)), plan.block_table, 12, 4, 70)
    t = g.gptq_kv_tree(short, to_dev(good), 20, 2, d_status=st)
    assert int(st) == g.GPTQ_EINVAL and torch.equal(t.mask[8:], tree.mask[8:])


def test_lengths_out_of_range_among_unequal_trees():
    """A sequence whose length is out of range raises the status, and others are not affected."""
    import post_weight_quantization_03_amd as g
    torch, dev = torch_dev()
    rng = np.random.default_rng(59)
    new, lengths = [70, 70, 70], [900, 4000, 300]
    c = Paged(rng, lengths, 2, 16, 64)
    plan, _ = c.plan(new)
    parents, _ = trees(rng, new, lengths)
    q = on_device(values(rng, (210, 4, 64), True), True)
    tree = g.gptq_kv_tree(plan, to_dev(parents))
    want = g.gptq_kv_attention(q, c.dev, plan, tree=tree)
    for bad in (-1, 4001, 2 ** 31 - 1):
        st = to_dev(np.zeros(1, np.int32))
        wrong = g.KVBatch(plan.q_start, to_dev(np.array([900, 4000, bad], np.int32)), plan.block_table, 210, 70, 4000)
        got = g.gptq_kv_attention(q, c.dev, wrong, tree=tree, d_status=st)
        assert int(st) == g.GPTQ_EINVAL
        assert torch.equal(got[:140], want[:140])


@pytest.mark.parametrize("new", [6, 100])
def test_nan_scales_of_blocks_that_are_not_seen(new):
    """Blocks between the first tokens and the window, and drafted tokens of other branches, may hold
    anything: their scales do not reach a row."""
    import post_weight_quantization_03_amd as g
    torch, dev = torch_dev()
    rng = np.random.default_rng(56)
    c = Paged(rng, [new + 333], 2, 16, 128)
    parents, sees = trees(rng, [new], [new + 333], 60, 3)
    plan, _ = c.plan([new])
    q = on_device(values(rng, (new, 4, 128), True), True)
    tree = g.gptq_kv_tree(plan, to_dev(parents), 60, 3)
    a = g.gptq_kv_attention(q, c.dev, plan, window=60, sinks=3, tree=tree)
    pages = c.table[0, :-(-(new + 333) // 16)]
    unseen = [p for k, p in enumerate(pages) if not sees[0][:, 16 * k:16 * k + 16].any()]
    assert len(unseen) > 10
    for i, p in enumerate(unseen):
        for t in (c.dev.k_scales, c.dev.v_scales):
            t[p] = [float("nan"), float("inf")][i % 2]
    assert torch.equal(a, g.gptq_kv_attention(q, c.dev, plan, window=60, sinks=3, tree=tree))


@pytest.mark.parametrize("new,length", [(5, 3000), (90, 4000)])
def test_another_stream_and_replayed_graphs(new, length):
    """Two graphs with workspaces of their own, replayed in turn with eager calls between and other trees
    and lengths each time."""
    import post_weight_quantization_03_amd as g
    torch, dev = torch_dev()
    rng = np.random.default_rng(57)
    c = Paged(rng, [length + 50, length], 2, 32, 128)
    side = torch.cuda.Stream()
    graphs = []
    for _ in range(2):
        lens = to_dev(np.array([length + 50, length], np.int32))
        plan = g.KVBatch(to_dev(np.array([0, new, 2 * new], np.int32)), lens, to_dev(c.table), 2 * new, new,
                         length + 50)
        parents = to_dev(np.concatenate([random_parents(rng, new)] * 2).astype(np.int32))
        q = on_device(values(rng, (2 * new, 4, 128), True), True)
        out, tree = torch.empty_like(q), g.KVTree.empty(plan)
        need = g.gptq_kv_attention_workspace_bytes(c.dev, plan, 4, g.GPTQ_BF16, True, 2000, 4)
        space = torch.full((need + 64,), 255, dtype=torch.uint8, device=dev)

        def step():
            g.gptq_kv_tree(plan, parents, 2000, 4, out=tree)
            g.gptq_kv_attention(q, c.dev, plan, window=2000, sinks=4, tree=tree, out=out, workspace=space)

        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        graphs.append((graph, plan, lens, parents, q, out, space))
    for turn in range(3):
        for graph, plan, lens, parents, q, out, space in graphs:
            parents.copy_(to_dev(np.concatenate([random_parents(rng, new) for _ in range(2)]).astype(np.int32)))
            lens.copy_(to_dev(np.array([length + 50 - 7 * turn, length - 100 * turn], np.int32)))
            side.wait_stream(torch.cuda.current_stream())
            graph.replay()
            tree = g.gptq_kv_tree(plan, parents, 2000, 4, stream=side)
            eager = g.gptq_kv_attention(q, c.dev, plan, window=2000, sinks=4, tree=tree, stream=side)
            torch.cuda.synchronize()
            assert torch.equal(out, eager)
            assert (space[space.numel() - 64:] == 255).all()


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("form", FORMS)
def test_a_window_without_first_tokens(form, bf16):
    """The entry point with a mask of no first tokens and no tree: blocks behind the window are not looked up."""
    import post_weight_quantization_03_amd as g
    torch, dev = torch_dev()
    lengths, new, qh, kh, dim, block = form
    say(f"window alone {form} bf16={bf16}")
    c = Paged(np.random.default_rng(49), lengths, kh, block, dim)
    sees = windows(new, lengths, 21, 0)
    kv = [c.kv(b) for b in range(len(new))]
    free_unseen(c, sees)
    plan, start = c.plan(new)
    q = values(np.random.default_rng(50), (int(start[-1]), qh, dim), bf16)
    qd = on_device(q, bf16)
    out, st = torch.full_like(qd, float("nan")), to_dev(np.zeros(1, np.int32))
    a, mask = g.attn.gptq_attention(qh, dim ** -0.5, 1, 21), g.attn.gptq_kv_mask(0, None, 0, None)
    dt = g.GPTQ_BF16 if bf16 else g.GPTQ_F32
    need = g.lib().gptq_kv_masked_attention_workspace_bytes(c.dev.c, plan.c, dt, a, mask)
    work = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)
    s = qd.stride()
    assert g.lib().gptq_kv_masked_attention(c.dev.c, plan.c, a, mask, qd.data_ptr(), s[0], s[1], out.data_ptr(), s[0],
                                            s[1], None, dt, work.data_ptr(), need, st.data_ptr(),
                                            torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()
    assert int(st) == 0
    got = out.float().cpu().numpy()
    for b, n in enumerate(new):
        if n == 0:
            continue
        rows = slice(start[b], start[b + 1])
        want, want_lse, more = M.attention(q[rows], *kv[b], dim ** -0.5, sees[b])
        more["lse"] = want_lse
        bound = attention_bound(want, more, lengths[b], dim, bf16, np.abs(kv[b][1]).max(initial=0))[0]
        close(f"out[{b}]", got[rows], want, bound + 1e-38)


def test_positions_of_a_padded_batch_can_be_rotated():
    """Rows that no sequence has hold position 0 in the room that KVTree.empty makes."""
    import post_weight_quantization_03_amd as g
    torch, dev = torch_dev()
    c = Paged(np.random.default_rng(51), [100, 40], 2, 16, 64)
    plan, start = c.plan([5, 3], total=23)
    torch.full((23,), -123456, dtype=torch.int32, device=dev)  # what the room may be made of
    tree = g.gptq_kv_tree(plan, to_dev(np.full(23, -1, np.int32)), out=g.KVTree.empty(plan))
    assert tree.positions.tolist() == [95] * 5 + [37] * 3 + [0] * 15
    cos = torch.ones((100, 32), device=dev)
    q, st = torch.randn((23, 2, 64), device=dev), to_dev(np.zeros(1, np.int32))
    out = g.gptq_qk_norm_rope(q, None, tree.positions, g.Rope(cos, torch.zeros_like(cos)), d_status=st)[0]
    assert int(st) == 0 and torch.equal(out, q)
