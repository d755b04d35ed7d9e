"""GPU: batches that serving has beside those of test_tree_attention.py, whose
reference and tolerances are taken: a piece of a prompt beside single tokens,
and the accepted path of more layers than one call of the library takes."""

import numpy as np
import pytest
import torch

import gemm_lora_shrink_amd as glsa
from oracle import attention_oracle as ao
from test_tree_attention import TYPES, Step, f64, ints

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("heads", [(8, 2, 128), (4, 4, 64), (4, 1, 256)], ids=lambda h: "x".join(map(str, h)))
@pytest.mark.parametrize("at", [0, 3, 6])
def test_a_prompt_beside_single_tokens(at, heads, dtype):
    counts, contexts = [1, 1, 1, 1, 1, 1, 1], [700, 0, 31, 1500, 64, 5, 128]
    counts[at] = 290
    s = Step(contexts, counts, *heads, TYPES[dtype], tree=False, seed=at)
    s.poison_unused()
    s.check()


@pytest.mark.parametrize("layers", [127, 128, 129, 257])
def test_kept_path_of_every_layer(layers):
    """Every layer's own rows move, those of the second and third call too."""
    hk, d, page, n = 2, 8, 7, 9
    contexts = [0, 37, 15]
    s = Step(contexts, [n] * 3, hk, hk, d, torch.bfloat16, page=page, seed=layers)
    path = np.array([[0, 3, 8], [1, 2, 4], [5, 6, 7]], np.int32)
    kept = np.array([3, 2, 3], np.int32)
    caches = [(torch.randn_like(s.k), torch.randn_like(s.v)) for _ in range(layers)]
    want = [[ao.keep(f64(c), s.table, contexts, path, kept) for c in pair] for pair in caches]
    glsa.keep_path([k for k, _ in caches], [v for _, v in caches], ints(s.table), ints(contexts), ints(path), ints(kept))
    for i, (pair, ref) in enumerate(zip(caches, want)):
        for c, r in zip(pair, ref):
            assert np.array_equal(f64(c), r), i
