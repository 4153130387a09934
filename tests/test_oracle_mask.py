"""Pins of the masked attention's references: the plain window's reference, closed forms, planted mistakes."""

import numpy as np
import pytest

from oracle import attn_ref, mask_ref as M


@pytest.mark.parametrize("causal,window", [(True, 0), (True, 5), (False, 3)])
def test_without_sinks_it_is_the_window(causal, window):
    rng = np.random.default_rng(0)
    q, k, v = rng.standard_normal((7, 4, 8)), rng.standard_normal((20, 2, 8)), rng.standard_normal((20, 2, 8))
    a = attn_ref.attention(q, k, v, 0.3, causal, window)
    b = M.attention(q, k, v, 0.3, M.window_sees(7, 20, window, 0, causal))
    assert np.allclose(a[0], b[0], atol=1e-14) and np.allclose(a[1], b[1], atol=1e-14)


def test_sinks_are_the_first_tokens():
    sees = M.window_sees(3, 10, 2, 3)
    assert [np.flatnonzero(r).tolist() for r in sees] == [[0, 1, 2, 6, 7], [0, 1, 2, 7, 8], [0, 1, 2, 8, 9]]
    # never past the token's own place
    assert np.flatnonzero(M.window_sees(10, 10, 1, 5)[2]).tolist() == [0, 1, 2]


def test_a_chain_is_causal():
    at, among = M.tree([-1, 0, 1, 2], 6)
    assert at.tolist() == [6, 7, 8, 9]
    assert np.array_equal(M.tree_sees(at, among, 6), M.window_sees(4, 10))
    at, among = M.tree([-1, 0, 1, 2], 6, 3, 1)
    assert np.array_equal(M.tree_sees(at, among, 6, 3, 1), M.window_sees(4, 10, 3, 1))
    at, among = M.tree([-1, 0, 1, 2], 0, 2, 1)
    assert np.array_equal(M.tree_sees(at, among, 0, 2, 1), M.window_sees(4, 4, 2, 1))


def test_branches_do_not_see_each_other():
    at, among = M.tree([-1, 0, 0, 1, 2, -1], 10)
    assert at.tolist() == [10, 11, 11, 12, 12, 10]
    assert [np.flatnonzero(r).tolist() for r in among] == [[0], [0, 1], [0, 2], [0, 1, 3], [0, 2, 4], [5]]
    assert M.words(among, 2).tolist() == [[1, 0], [3, 0], [5, 0], [11, 0], [21, 0], [32, 0]]
    many = np.zeros((1, 70), dtype=bool)
    many[0, [0, 63, 64, 69]] = True
    assert M.words(many, 2).tolist() == [[1 + 2 ** 63, 1 + 32]]


def test_values_of_a_branch_are_its_own():
    """A tree's rows equal those of each path taken alone, and a causal mask does not."""
    rng = np.random.default_rng(1)
    parents, before = [-1, 0, 0, 2], 5
    q, k, v = rng.standard_normal((4, 1, 8)), rng.standard_normal((9, 1, 8)), rng.standard_normal((9, 1, 8))
    at, among = M.tree(parents, before)
    out = M.attention(q, k, v, 0.5, M.tree_sees(at, among, before))[0]
    path = [0, 1, 2, 3, 4, 5, 7, 8]  # the last token's: new tokens 0, 2, 3
    alone = attn_ref.attention(q[[0, 2, 3]], k[path], v[path], 0.5)[0]
    assert np.allclose(out[[0, 2, 3]], alone, atol=1e-14)
    assert np.abs(attn_ref.attention(q, k, v, 0.5)[0][3] - out[3]).max() > 1e-3
