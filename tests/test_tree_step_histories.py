"""GPU: examples/tree_step.py over a cache in 8 bits holds the same tokens whichever
way they came: at the last step of the two runs, the one whose drafted tree was
verified and the one forked at the prompt and decoded token by token, every
sequence's keys and values of the first layer are the same tokens' in the same order.

The two differ by roundings.  A first layer's key or value x depends on its token and
position alone, up to the order of sums in fp32 (512 terms: 512 * 2^-24 of the row's
largest, either run).  It is rounded when it is stored and again whenever its block's
exponent grows, from e1 to e2 > e1 and so on.  INT8 errs by half of 2^e each time, at
most 2^e in all for the last e, as those before are halves and less.  e4m3 errs by
2^-4 |x| once, as numbers in its normal range stay exact when the exponent grows, and
in its subnormal one like INT8, with steps of 2^-9 2^e: 2^-9 2^e in all."""

import os
import sys

import numpy as np
import pytest
import torch

from test_quantized_cache import f64, on_host

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def history(cache, table, context, q_start):
    """Of each sequence [2, L, heads, d] values and [2, L, heads, 1] exponents of its tokens, in order."""
    host, page = on_host(cache), cache[0].shape[2]
    block = page // host["k_exp"].shape[2]
    out = []
    table, lengths = table.cpu().numpy(), (context + q_start.diff()).tolist()
    for b, n in enumerate(lengths):
        pos = np.arange(n)
        at, row = table[b][pos // page], pos % page
        assert (at >= 0).all() and len(set(zip(at, row))) == n
        e = np.stack([host[x + "_exp"][at, :, row // block] for x in ("k", "v")])[..., None]
        out.append((np.stack([host[x][at, :, row] for x in ("k", "v")]) * 2.0 ** e, e))
    return out


@pytest.mark.parametrize("held", [torch.float8_e4m3fn, torch.int8])
@pytest.mark.parametrize("norm", [False, True])
def test_both_runs_hold_the_same_tokens(monkeypatch, norm, held):
    import tree_step

    calls, plain = [], tree_step.glsa.tree_attention_quantized

    def attention(q, cache, table, context, q_start, **kw):
        calls.append(history(cache, table, context, q_start))
        return plain(q, cache, table, context, q_start, **kw)

    monkeypatch.setattr(tree_step.glsa, "tree_attention_quantized", attention)
    tree_step.run(torch.float32, norm, held)
    assert len(calls) == tree_step.LAYERS * 7  # prompt, tree, token after it; three single steps, token after them
    tree, single = calls[2 * tree_step.LAYERS], calls[6 * tree_step.LAYERS]
    assert [x.shape[1] for x, _ in tree] == [x.shape[1] for x, _ in single] == [21 + 3 + 1, 40 + 2 + 1, 5 + 0 + 1]

    def bound(x, e, y, f):
        sums = 2 * 512 * 2.0 ** -24 * np.abs(x).max(-1, keepdims=True)
        if held == torch.int8:
            return 2.0 ** e + 2.0 ** f + 2 * sums
        # (|x| as held; the value before it was rounded is at most 1 / (1 - 2^-4) of it)
        return (np.abs(x) + np.abs(y)) * 2.0 ** -4 / (1 - 2.0 ** -4) + (2.0 ** e + 2.0 ** f) * 2.0 ** -9 + 2 * sums

    for (x, e), (y, f) in zip(tree, single):
        off = np.abs(x - y) / bound(x, e, y, f)
        assert off.max() <= 1, off.max()
        # other tokens in their places would show: every row, one place on
        moved = np.abs(x[:, 1:] - y[:, :-1]) > bound(x[:, 1:], e[:, 1:], y[:, :-1], f[:, :-1])
        assert moved.mean((2, 3)).min() > 0.2
