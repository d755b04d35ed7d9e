"""GPU: attention over a quantized cache where a workgroup walks many stages of
keys, with whole and partial last ones and with pages missing here and there, so
that which rows are keys differs from stage to stage.

65 sequences, most of them short: keys are then cut by the bounds, and there are
units enough that a sequence is one chunk (8 to 20 stages of 64 keys).  Tolerances:
those of test_quantized_cache, whose reference and inputs these are."""

import numpy as np
import pytest

from test_quantized_cache import Step

pytestmark = pytest.mark.gpu

# keys of the long sequences, context and nodes together: whole stages, one key more, some fewer
TOTALS = [8 * 64, 8 * 64 + 1, 11 * 64 - 5, 12 * 64, 12 * 64 + 33, 16 * 64 + 1, 17 * 64, 20 * 64 - 31]
HEADS = [  # d, hq, hk, nodes
    (64, 16, 4, 48), (64, 16, 4, 20), (128, 16, 4, 48), (128, 16, 4, 30), (48, 8, 4, 90), (256, 16, 8, 40),  # many rows
    (64, 16, 8, 2), (128, 16, 8, 4), (256, 16, 4, 3),                                                        # few
]


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("case", range(len(HEADS)))
def test_many_stages(case, dt, fmt):
    d, hq, hk, nodes = HEADS[case]
    rng = np.random.default_rng(case)
    contexts, counts = rng.integers(0, 40, 65), rng.integers(0, 4, 65).clip(0, nodes)
    long = rng.permutation(65)[:len(TOTALS)]
    for b, total in zip(long, TOTALS):
        counts[b] = nodes if total % 2 else max(1, nodes - 3)
        contexts[b] = total - counts[b]
    s = Step(contexts.tolist(), counts.tolist(), hq, hk, d, dt, fmt, block=8, seed=case, tree=case % 2 == 0)
    for b in long[1:]:  # (the first keeps all its pages)
        held = -(-int(contexts[b] + counts[b]) // 16)
        s.table[b][:held][rng.random(held) < 0.2] = -1
        s.table[b][held - 2 - b % 3] = -1
    s.poison_unused()
    s.check(what=f"{d} {hq} {hk} {nodes}")
