"""The attention operators' fp64 references themselves (CPU): gradients against central
differences, the cache's error promise, and planted mistakes that the checks must catch."""

import numpy as np
import pytest

from oracle import attn_ref as R


def _tables(rng, positions, rot):
    a = rng.uniform(0, 6, (positions, rot // 2))
    return np.cos(a), np.sin(a)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot", [0, 16, 32])
@pytest.mark.parametrize("weight", [True, False])
def test_backward_against_differences(interleaved, rot, weight):
    rng = np.random.default_rng(3)
    t, h, d = 3, 2, 32
    x, dy = rng.standard_normal((t, h, d)), rng.standard_normal((t, h, d))
    w = rng.uniform(0.5, 1.5, d) if weight else None
    cos, sin = _tables(rng, 7, rot)
    pos = np.array([0, 5, 6])
    f = lambda x, w: float((R.norm_rope(x, w, cos, sin, pos, interleaved, 1e-3) * dy).sum())  # noqa: E731
    dx, dw = R.norm_rope_backward(dy, x, w, cos, sin, pos, interleaved, 1e-3)
    step = 1e-5
    # central differences: error step^2 / 6 times a third derivative of order 10, and 1e-16 / step
    for idx in [(0, 0, 0), (1, 1, 5), (2, 0, 17), (2, 1, 31)]:
        e = np.zeros_like(x)
        e[idx] = step
        assert abs((f(x + e, w) - f(x - e, w)) / (2 * step) - dx[idx]) < 1e-8
    if weight:
        for i in (0, 9, 31):
            e = np.zeros(d)
            e[i] = step
            assert abs((f(x, w + e) - f(x, w - e)) / (2 * step) - dw[i]) < 1e-8
    else:
        assert dw is None


def test_rotation_keeps_length_and_unrotated_part():
    rng = np.random.default_rng(5)
    x = rng.standard_normal((4, 3, 48))
    cos, sin = _tables(rng, 9, 32)
    pos = np.array([0, 2, 8, 3])
    for inter in (False, True):
        y = R.norm_rope(x, None, cos, sin, pos, inter)
        np.testing.assert_allclose((y ** 2).sum(-1), (x ** 2).sum(-1), rtol=1e-13)
        assert np.array_equal(y[..., 32:], x[..., 32:])
        back, _ = R.norm_rope_backward(y, None, None, cos, sin, pos, inter)
        np.testing.assert_allclose(back, x, atol=1e-14)
    # the two pairings are not the same rotation
    assert not np.allclose(R.norm_rope(x, None, cos, sin, pos, True), R.norm_rope(x, None, cos, sin, pos, False))


@pytest.mark.parametrize("amax,want", [(127.0, 0), (127.0000076, 1), (63.5, -1), (1.0, -6), (0.0, -100),
                                       (2.0 ** -140, -100), (3.4028234e38, 122), (2.0 ** -94, -100)])
def test_needed_scale(amax, want):
    assert R.needed_scale(amax) == 2.0 ** want
    assert amax <= 127 * R.needed_scale(amax)


def _empty(pages, heads, block, dim):
    rng = np.random.default_rng(1)
    return R.Cache(rng.integers(-128, 128, (pages, heads, block, dim)).astype(np.int8),
                   rng.integers(-128, 128, (pages, heads, block // 16, dim, 16)).astype(np.int8),
                   np.full((pages, heads), np.nan), np.full((pages, heads), 1e30))


def test_any_number_of_appends_stays_within_one_step():
    """Tokens whose size doubles now and then, appended one by one to a block of stale contents."""
    rng = np.random.default_rng(2)
    c = _empty(3, 2, 32, 16)
    table = [2, 0]
    x = rng.standard_normal((40, 2, 16)) * 2.0 ** (np.arange(40) // 3)[:, None, None]
    for i in range(40):
        c.append(x[i:i + 1], -x[i:i + 1], table, i)
        for is_v, sign in ((False, 1), (True, -1)):
            got = c.read(table, i + 1, is_v)
            scale = np.repeat((c.v_scales if is_v else c.k_scales)[table[:i // 32 + 1]], 32, 0)[:i + 1]
            assert np.all(np.abs(got - sign * x[:i + 1]) <= scale[..., None])
    assert np.all(c.k_scales[2] == R.needed_scale(np.abs(x[:32]).max((0, 2))))


def test_a_value_that_is_not_finite_poisons_its_block_and_head_only():
    c = _empty(2, 2, 16, 16)
    x = np.ones((3, 2, 16))
    x[1, 0, 3] = np.nan
    c.append(x, np.ones((3, 2, 16)), [1, 0], 0)
    assert np.isnan(c.k_scales[1, 0]) and c.k_scales[1, 1] == 2.0 ** -6 and np.all(c.v_scales[1] == 2.0 ** -6)
    c.append(np.ones((1, 2, 16)), np.ones((1, 2, 16)), [1, 0], 3)
    assert np.isnan(c.k_scales[1, 0])  # until the block is started afresh
    c.append(np.ones((1, 2, 16)), np.ones((1, 2, 16)), [1, 0], 0)
    assert c.k_scales[1, 0] == 2.0 ** -6


def test_attention_masks_and_empty_rows():
    rng = np.random.default_rng(4)
    q, k, v = (rng.standard_normal(s) for s in ((4, 2, 8), (3, 1, 8), (3, 1, 8)))
    out, lse, _ = R.attention(q, k, v, 0.3)  # four tokens, three places: the first sees nothing
    assert np.all(out[0] == 0) and np.all(np.isneginf(lse[0]))
    np.testing.assert_allclose(out[1], np.broadcast_to(v[0], (2, 8)))
    out, lse, _ = R.attention(q, k, v, 0.3, window=1)
    for i in (1, 2, 3):
        np.testing.assert_allclose(out[i], np.broadcast_to(v[i - 1], (2, 8)))
    full, _, _ = R.attention(q, k, v, 0.3, causal=False)
    assert np.all(full[0] != 0)


@pytest.mark.parametrize("plant", ["shift the mask", "forget the scale", "wrong head"])
def test_a_planted_mistake_shows(plant):
    """An attention with a mistake planted differs from the definition by far more than the bounds
    used on the device (which are below 1e-2)."""
    rng = np.random.default_rng(6)
    q, k, v = (rng.standard_normal(s) for s in ((5, 4, 16), (9, 2, 16), (9, 2, 16)))
    good, _, _ = R.attention(q, k, v, 0.25)
    if plant == "shift the mask":
        bad, _, _ = R.attention(q[:4], k[:8], v[:8], 0.25)
        bad, good = bad[:4], good[:4]
        bad = np.concatenate([bad[1:], bad[:1]])
    elif plant == "forget the scale":
        bad, _, _ = R.attention(q, k, v, 1.0)
    else:
        bad, _, _ = R.attention(q, k[:, ::-1], v[:, ::-1], 0.25)
    assert np.linalg.norm(bad - good) > 0.1 * np.linalg.norm(good)
