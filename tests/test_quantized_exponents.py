"""GPU: attention over a quantized cache whose blocks have the largest exponents.

A weight times its value's power of two, and that times a byte's number, may not
pass what fp32 holds: infinities would meet zeros, or each other, where every value
is finite.  Tolerances: those of test_quantized_cache, and for fp16 queries of more
than 32 rows a head (`few_bits`): a weight times its value's power of two enters as
one fp16 number, off by half a step: 2^-11 of itself down to 2^-14 and 2^-25 below,
where steps are all 2^-24.  The row's largest such product P is 2^12 at least in these
numbers, as it is put there whenever the reference of the weights moves, and others
only grow past it.  So a key is off by up to 2^-25 * 2^-12 P more, times its byte's
number: 2^-37 P sum |number| in all, where the weights add up to 1.  (It shows where a block
of a large power holds zeros, and so has no part in an element.)"""

import numpy as np
import pytest
import torch

from oracle import attention_oracle as ao
from oracle import cache_oracle as co
from test_quantized_cache import U, WEIGHT, Step, f64, ints, on_host

pytestmark = pytest.mark.gpu

ROWS = [([1, 3], 64, 8, 2), ([40, 33], 64, 8, 2), ([9, 20], 128, 8, 2), ([70, 30], 128, 8, 2), ([2, 1], 256, 8, 2),
        ([50, 64], 256, 4, 2)]  # nodes, d, hq, hk: one block of rows, two and more, and heads that only the wide kernel takes


def blocks(s, block, part, seed=0):
    """A random part of the cache's blocks [pages, heads, blocks], and their rows [pages, heads, page, 1]."""
    g = torch.Generator("cuda").manual_seed(seed)
    of = torch.rand(s.cache.v_exp.shape, generator=g, device="cuda") < part
    return of, of.repeat_interleave(block, 2)[..., None]


def few_bits(s):
    """2^-37 P sum |number| of every row and element of a step."""
    host, scale, group = on_host(s.cache), s.d ** -0.5, s.hq // s.hk
    q, k = f64(s.q).reshape(s.T, s.hq, s.d), co.values(host, "k")
    block = s.page // host["v_exp"].shape[2]
    out = np.zeros((s.T, s.hq, s.d))
    for b in range(s.B):
        at = ao.cache_rows_of(s.table[b], np.arange(s.context[b] + s.counts[b]), s.page, s.n_pages)
        page, row = at // s.page, at % s.page
        for h in range(s.hq):
            kv = h // group
            power = 2.0 ** np.clip(host["v_exp"][page, kv, row // block], co.LOW, co.TOP[host["fmt"]])
            held = np.abs(host["v"][page, kv, row])
            for i in range(s.counts[b]):
                seen = np.concatenate([np.ones(s.context[b], bool), s.sees[b][i]])
                score = scale * (k[page, kv, row][seen] @ q[s.q_start[b] + i, h])
                w = np.exp(score - score.max())
                out[s.q_start[b] + i, h] = 2.0 ** -37 * (w / w.sum() * power[seen]).max() * held[seen].sum(0)
    return out


def check_few_bits(s):
    """Step.check's bound on the output, and few_bits."""
    out, _ = s.run()
    host = on_host(s.cache)
    want, _, spread, z = ao.attend(f64(s.q).reshape(s.T, s.hq, s.d), co.values(host, "k"), co.values(host, "v"), s.table,
                                   s.context, s.q_start, s.sees, s.d ** -0.5)
    L, z = (max(s.context) + max(s.counts)), z[..., None]
    h, w = torch.finfo(s.dt).eps / 2, WEIGHT[s.dt]
    rel = 2 * ((3 * s.d + 2) * U * z + (4 + 2 * z) * U) + 4 * L * U + w + 8 * U
    off = h * np.abs(want) + (rel * spread + few_bits(s)) * (1 + h) + torch.finfo(s.dt).tiny * torch.finfo(s.dt).eps
    worst = np.abs(out - want) / off
    assert np.isfinite(out).all() and worst.max() <= 1, worst.max()


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows", range(len(ROWS)))
def test_zeros_under_the_largest_exponents(rows, dt, fmt):
    """Blocks of zeros, keys and values, whatever their exponent, are zeros."""
    counts, d, hq, hk = ROWS[rows]
    s = Step([150, 1400], counts, hq, hk, d, dt, fmt, block=4)
    for held, exps, seed in ((s.cache.k, s.cache.k_exp, 1), (s.cache.v, s.cache.v_exp, 2)):
        of, at = blocks(s, 4, 0.3, seed)
        held.view(torch.uint8).masked_fill_(at, 0)
        # (many fp16 rows: weights times powers are fp16 numbers, 2^10 is as far as fp16 values go)
        many = dt == "f16" and max(counts) * hq // hk > 32
        high = [10] if many and held is s.cache.v else [60, 100, 119, 120, 121, 127]
        pick = torch.randint(len(high), of.shape, generator=s.g, device="cuda")
        exps.copy_(torch.where(of, ints(high, torch.int8)[pick], exps))
    if many:
        check_few_bits(s)
    else:
        s.check(what=f"{counts}")


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("rows", range(len(ROWS)))
def test_values_of_the_largest_exponents(rows, dt, fmt):
    """Means of values up to the largest that a cache holds are finite, as they are."""
    counts, d, hq, hk = ROWS[rows]
    for low in (127, 60, -20):
        s = Step([150, 1400], counts, hq, hk, d, dt, fmt, block=4)
        s.cache.v_exp.copy_(torch.randint(low, 128, s.cache.v_exp.shape, generator=s.g, device="cuda").to(torch.int8))
        out = s.check(what=f"{counts} from {low}")
        assert np.isfinite(out).all() and np.abs(out).max() > 2.0 ** 110
