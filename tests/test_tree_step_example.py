"""GPU: adapters, rotary positions, paged cache, tree attention and the accepted
path together, as examples/tree_step.py uses them: the accepted nodes of a
verified tree, and the token after them, come out as the same tokens decoded
one by one.

Tolerance, in fp32: the two ways compute the same sums in other orders.  A
layer has four products in a row (projection, adapter, attention, output) of at
most 512 terms, each off by at most 512 * 2^-24 of its magnitudes on either
side; two layers: 2 * 2 * 4 * 512 * 2^-24 = 4.9e-4 of the rows' largest."""

import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("norm", [False, True])
def test_tree_step_matches_single_tokens(norm):
    import tree_step

    tree, single = tree_step.run(torch.float32, norm)
    assert tree.shape == (8, tree_step.HIDDEN) and bool(torch.isfinite(tree).all())
    off = float((tree - single).abs().max())
    assert off <= 2 * 2 * 4 * 512 * 2.0 ** -24 * float(single.abs().max()), off
    assert float((tree[0] - tree[1]).abs().max()) > 0.1  # different tokens do come out different
