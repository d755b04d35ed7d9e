"""Arguments of the quantized cache's and the pages' calls at their edges: what
must be refused on the host, and what looks odd but is a call like any other."""

import numpy as np
import pytest
import torch

import gemm_lora_shrink_amd as glsa
from gemm_lora_shrink_amd import cache as C
from oracle import cache_oracle as co
from test_cache_abi import BAD, FAKE, OK, _attend, _keep

DEVICES = pytest.mark.gpu


def ints(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device="cuda")


def raw(tensors):
    return [t.clone().view(torch.uint8) for t in tensors]


@pytest.mark.parametrize("layers", [2, 128])
def test_keep_refuses_an_address_that_comes_twice(layers):
    """Keys, values or exponents of two layers, or of one, at one address: nothing is enqueued."""
    names = ("k", "v", "ke", "ve")
    pack = C.struct.Struct(f"@{layers}P").pack

    def lists():
        return {n: [FAKE + (i * layers + j) * 4096 for j in range(layers)] for i, n in enumerate(names)}

    for a, i, b, j in (("k", 0, "k", layers - 1), ("v", 1, "v", 0), ("ke", 0, "ke", 1), ("ve", layers - 1, "ve", 0),
                       ("ke", 0, "ve", 0), ("ke", 1, "ve", layers - 2), ("k", 0, "v", 0), ("k", 1, "ve", 0)):
        at = lists()
        at[a][i] = at[b][j]
        assert _keep(layers=layers, **{n: pack(*x) for n, x in at.items()}) == BAD
        assert b"twice" in glsa.lib().lora_last_error()


@DEVICES
def test_keep_refuses_exponents_that_come_twice():
    a, b = ([t.clone() for t in glsa.alloc_quantized_cache(4, 2, 8, 32, "cuda", dtype=torch.int8)] for _ in range(2))
    for t in a + b:
        t.copy_(torch.randint(-9, 9, t.shape, device="cuda").to(torch.int8))
    was = raw(a + b)
    args = ints([[0, 1], [2, 3]]), ints([7, 3]), ints([[2, 4], [1, 3]]), ints([2, 2])
    for caches in ([a, [*b[:2], a[2], b[3]]], [a, [*b[:3], a[3]]], [[*a[:3], a[2]]], [a, [*b[:2], a[3], b[3]]]):
        with pytest.raises(glsa.LoraError, match="twice"):
            glsa.keep_path_quantized(caches, *args)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(raw(a + b), was))
    glsa.keep_path_quantized([a, b], *args)
    torch.cuda.synchronize()
    assert not all(torch.equal(x, y) for x, y in zip(raw(a + b), was))


@DEVICES
@pytest.mark.parametrize("fmt", [torch.float8_e4m3fn, torch.int8])
def test_caches_of_no_pages(fmt):
    """Nothing is placed, nothing moves, and rows see no key: outputs of 0."""
    caches = [glsa.alloc_quantized_cache(0, 2, 16, 64, "cuda", dtype=fmt, block=8) for _ in range(3)]
    table, context = ints([[-1, -1, -1], [0, 5, -1]]), ints([7, 20])
    x = torch.randn(4, 8 * 64, device="cuda").bfloat16()
    glsa.store_quantized(x[:, :128], x[:, 128:256], caches[0], ints([0, 5, -1, 40]))
    glsa.keep_path_quantized(caches, table, context, ints([[0, 2], [1, 2]]), ints([2, 1]))
    lse = torch.zeros(4, 8, device="cuda")
    for nodes, counts in ((3, [3, 1]), (20, [1, 3])):  # one block of rows, and more
        out = torch.full_like(x, 5)
        ws = glsa.alloc_quantized_workspace(2, 4, nodes, 48, 8, 2, 64, "cuda")
        glsa.tree_attention_quantized(x, caches[0], table, context, ints(np.cumsum([0] + counts)), max_nodes=nodes,
                                      max_context=48, out=out, lse=lse, workspace=ws)
        assert not out.any() and bool((lse == -float("inf")).all())


def test_no_sequences_need_no_table():
    """An empty page table has no address, however many columns."""
    assert _attend(B=0, table=None, context=None, q_start=None) == OK
    assert _keep(B=0, table=None, context=None, path=None, kept=None) == OK
    assert _attend(B=0, table=None, n_table=-1) == BAD and _keep(B=0, table=None, n_table=-1, ld=4) == BAD
    assert _attend(B=1, table=None) == BAD and _keep(B=1, table=None) == BAD


@DEVICES
def test_calls_of_no_sequences():
    cache = glsa.alloc_quantized_cache(4, 2, 16, 64, "cuda")
    table, none = torch.empty(0, 9, dtype=torch.int32, device="cuda"), ints([])
    x = torch.randn(3, 8 * 64, device="cuda").half()
    out = torch.full_like(x, 5)
    glsa.tree_attention_quantized(x, cache, table, none, ints([0]), max_nodes=3, out=out)
    glsa.keep_path_quantized([cache], table, none, table, none)
    assert bool((out == 5).all())


@DEVICES
@pytest.mark.parametrize("page", [1, 3, 1 << 29, (1 << 30) + 1, 2 ** 31 - 1])
def test_lengths_near_2_to_31(page):
    """Columns are ceil(tokens / page_size) up to the largest lengths and pages."""
    top = 2 ** 31 - 1
    lengths = np.array([top, top - 1, 1 << 30, (1 << 30) + 1, page, min(page, top - 1) + 1, page - 1, 0, -5, -top - 1], np.int64)
    B, n = len(lengths), 60
    refs, table, missing = np.zeros(n, np.int64), np.full((B, 5), -1), ints([0])
    got_refs, got = ints(refs), ints(table)
    lacking = co.reserve(refs, table, lengths, page)
    glsa.reserve_pages(got_refs, got, ints(lengths), page_size=page, missing=missing)
    assert np.array_equal(got.cpu().numpy(), table) and np.array_equal(got_refs.cpu().numpy(), refs) and int(missing) == lacking == 0
    keep = lengths[[3, 5, 0, 2, 6, 1, 4, 8, 9, 7]]
    co.release(refs, table, range(B), keep, page)
    glsa.release_pages(got_refs, got, keep=ints(keep), page_size=page)
    assert np.array_equal(got.cpu().numpy(), table) and np.array_equal(got_refs.cpu().numpy(), refs)


def test_one_tensor_is_a_list_of_it():
    """Not a list of its pages, which would be copied as if their heads were pages."""
    x = torch.zeros(4, 4, 8)
    for listed in (C._listed(x), C._listed([x]), C._listed((x,))):
        assert len(listed) == 1 and listed[0] is x
    assert C._listed(()) == () and len(C._listed(glsa.alloc_quantized_cache(2, 1, 4, 16, "cpu"))) == 4


@DEVICES
def test_pages_of_one_tensor():
    x = torch.arange(4 * 4 * 8, device="cuda").view(4, 4, 8).float()
    want = x.clone()
    want[3] = want[1]
    glsa.copy_pages(x, ints([1]), ints([3]))
    assert torch.equal(x, want)
    refs, table = ints([0, 0, 0, 1]), ints([[3]])
    assert int(glsa.compact_pages(refs, table, tensors=x)) == 1
    want[0] = want[3]
    assert torch.equal(x, want) and table.tolist() == [[0]]
    to = ints([[7]])
    glsa.fork_sequences(refs, table, ints([0]), ints([0]), ints([3]), page_size=4, tensors=x, out_table=to)
    want[1] = want[0]
    assert torch.equal(x, want) and to.tolist() == [[1]]
