"""The tree of drafted tokens that examples/decode_attention.py makes: what it keeps is a path of the tree."""

import os
import sys

import pytest

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.parametrize("drafts", [1, 2, 3, 4, 7, 8, 9, 12, 63, 64, 65, 1000])
def test_what_is_kept_is_a_longest_path(drafts):
    from decode_attention import half_tree
    parents, path = half_tree(drafts)
    assert len(parents) == drafts and all(-1 <= p < i for i, p in enumerate(parents))
    depth = []
    for p in parents:
        depth.append(depth[p] + 1 if p >= 0 else 0)
    assert parents[path[0]] == -1 and all(parents[b] == a for a, b in zip(path, path[1:]))
    assert len(path) == max(depth) + 1
