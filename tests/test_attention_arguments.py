"""What the binding of include/lora_attention.h makes of its arguments before
they reach the library: strides of integer matrices."""

import pytest
import torch

import gemm_lora_shrink_amd as glsa
from gemm_lora_shrink_amd import attention as A

BAD = glsa.LORA_ERR_INVALID_ARG
HOST = -1  # the device index of host tensors


# ---- page tables and paths: rows that overlap ---------------------------------

def _overlapping(device="cpu"):
    row = torch.arange(8, dtype=torch.int32, device=device)
    return [row[:4].expand(3, 4), row.as_strided((3, 4), (2, 1))]  # one row for all, rows two apart


def test_integer_rows_that_overlap_are_refused():
    """The kernels step from row to row by the stride: with any other than the
    tensor's own they would read past its end."""
    for t in _overlapping():
        with pytest.raises(glsa.LoraError, match="overlap") as e:
            A._int_rows(t, "page_table", HOST, 3)
        assert e.value.status == BAD


def test_integer_rows_keep_their_own_stride():
    wide = torch.arange(24, dtype=torch.int32).view(3, 8)
    for t, ld, cols in ((wide, 8, 8), (wide[:, :5], 8, 5), (wide[:, 3:4], 8, 1), (wide[::2], 16, 8)):
        assert A._int_rows(t, "t", HOST, t.size(0)) == (t.data_ptr(), ld, cols)
    # a single row, or rows without columns, have no stride that matters
    assert A._int_rows(wide[:1].expand(1, 8), "t", HOST, 1)[1:] == (8, 8)
    assert A._int_rows(wide[:1, :1].expand(1, 1), "t", HOST, 1)[2] == 1
    assert A._int_rows(wide[:, :0], "t", HOST, 3)[2] == 0


@pytest.mark.gpu
def test_calls_with_overlapping_rows_are_refused():
    B, page, d = 3, 8, 64
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    k, v = (torch.zeros(4, 1, page, d, device="cuda") for _ in range(2))
    context, start = ints([5] * B), ints(range(B + 1))
    q = torch.zeros(B, d, device="cuda")
    good = ints([[0, 1, 2, 3]] * B)
    path, kept = ints([[0, 1, 2, 3]] * B), ints([2] * B)
    for t in _overlapping("cuda"):
        for call in (lambda: glsa.build_tree(None, start, context, max_nodes=1, n_tokens=B, page_table=t, n_pages=4,
                                             page_size=page),
                     lambda: glsa.tree_attention(q, k, v, t, context, start, max_nodes=1),
                     lambda: glsa.keep_path(k, v, t, context, path, kept),
                     lambda: glsa.keep_path(k, v, good, context, t, kept)):
            with pytest.raises(glsa.LoraError, match="overlap"):
                call()
    glsa.keep_path(k, v, good, context, path, kept)
