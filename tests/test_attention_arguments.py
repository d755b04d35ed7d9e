"""What the binding of include/lora_attention.h makes of its arguments before
they reach the library: strides of integer matrices, the streams of the
tensors it makes itself, and numbers past the 32 bits of the C ABI.  And the workspace of tree_attention, which a server
allocates once for its largest batch."""

import random
from contextlib import contextmanager
from types import SimpleNamespace

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


# ---- tensors that the binding makes: on the call's stream ----------------------

class _NoLibrary:
    """Every entry point succeeds and does nothing but keep its arguments."""

    def __getattr__(self, name):
        def call(*args):
            self.args = args
            return glsa.LORA_OK
        return call


@pytest.fixture
def no_library(monkeypatch):
    """The binding without a GPU, on host tensors."""
    monkeypatch.setattr(A, "_gpu", lambda t, name: HOST)
    monkeypatch.setattr(A, "_stream_of", lambda stream, dev: stream)
    monkeypatch.setattr(A, "_bound", _NoLibrary())
    monkeypatch.setattr(A, "_lib", lambda: A._bound)
    return A._bound


@pytest.fixture
def made_on(monkeypatch, no_library):
    """Lists the stream that each new tensor is made on."""
    streams, made = [None], []

    @contextmanager
    def stream(s):
        streams.append(s)
        yield
        streams.pop()

    def recorded(make):
        def call(*args, **kw):
            made.append(streams[-1])
            return make(*args, **kw)
        return call

    for name in ("empty", "zeros", "full"):
        monkeypatch.setattr(torch, name, recorded(getattr(torch, name)))
    monkeypatch.setattr(torch.cuda, "stream", stream)
    return made


def test_tensors_are_made_on_the_stream_of_the_call(made_on):
    """A fill on the current stream would not be ordered with the kernel on another."""
    side = SimpleNamespace(cuda_stream=1)
    ints = torch.tensor([0, 2], dtype=torch.int32)
    table, context = torch.tensor([[0]], dtype=torch.int32), torch.tensor([3], dtype=torch.int32)
    q, cache = torch.ones(2, 8), torch.ones(1, 1, 8, 8)
    glsa.build_tree(ints - 1, ints, context, max_nodes=2, page_table=table, n_pages=1, page_size=8, stream=side)
    assert made_on == [side] * 3
    del made_on[:]
    glsa.tree_attention(q, cache, cache, table, context, ints, max_nodes=2, stream=side)
    assert made_on == [side]
    del made_on[:]
    glsa.rope_table(4, 8, frequencies=[1.0] * 4, device="cpu", stream=side)
    assert made_on == [side]


@pytest.mark.gpu
def test_calls_on_a_stream_beside_a_busy_one():
    """Work queued on the current stream before a call on another one has no part
    in what the call gives."""
    B, n, hq, d, page = 2, 5, 2, 64, 8
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    parents, start, context = ints([-1, 0, 0, 2, 1] * B), ints([0, n, 2 * n]), ints([9, 20])
    pages = ints([[0, 1, 2, 3], [4, 5, 6, 7]])
    g = torch.Generator("cuda").manual_seed(0)
    q = torch.randn(B * n, hq * d, device="cuda", generator=g)
    k, v = (torch.randn(8, 1, page, d, device="cuda", generator=g) for _ in range(2))
    big = torch.ones(8192, 8192, device="cuda", dtype=torch.bfloat16)
    side = torch.cuda.Stream()

    def step(stream):
        mask, pos, rows = glsa.build_tree(parents, start, context, max_nodes=n, page_table=pages, n_pages=8,
                                          page_size=page, stream=stream)
        out = glsa.tree_attention(q, k, v, pages, context, start, max_nodes=n, mask=mask, stream=stream)
        return mask, pos, rows, out, glsa.rope_table(64, 32, stream=stream)

    want = [t.cpu() for t in step(None)]
    torch.cuda.synchronize()
    for _ in range(3):
        for _ in range(40):
            busy = big @ big  # some 40 ms of the current stream
        got = step(side)
        with torch.cuda.stream(side):
            got = [t.cpu() for t in got]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert bool((want[0] != 0).all() and (want[1] >= 0).all() and (want[2] >= 0).all()) and busy.numel()


# ---- one workspace for every batch ---------------------------------------------

FAKE = 0x10000  # an aligned, never dereferenced address


def _refusal(B, T, nodes, context, hq, hk, d, ws_bytes, dtype=2, status=BAD):
    """What a call with a workspace of ws_bytes says; without `out` it is refused
    for that at the latest, so nothing is launched."""
    cache = A._CACHE_FIELDS.pack(FAKE, FAKE, 0, 0, 0, 0, 0, 0, 4, 16)
    st = A._lib().lora_tree_attention(dtype, FAKE, hq * d, T, B, hq, hk, d, cache, FAKE, 4, 4, FAKE, FAKE, nodes, context,
                                      None, 0, 0.1, None, hq * d, None, FAKE, ws_bytes, None)
    assert st == status
    return glsa.lib().lora_last_error().decode()


def test_a_workspace_serves_every_smaller_call():
    """Fewer sequences or nodes are cut into more chunks, so what a call needs
    does not grow with its sizes; what is allocated for them must."""
    rng = random.Random(0)
    size = lambda most: min(most, int(2 ** rng.uniform(0, most.bit_length())))
    served = 0
    for _ in range(300):
        hk = rng.choice([1, 2, 8, 16, 40])
        heads = (hk * rng.choice([1, 2, 4, 7]), hk, rng.choice([8, 64, 80, 128, 256]))
        most = (size(256), size(8192), size(1024), size(131072))
        have = glsa.attention_workspace_bytes(*most, *heads)
        for _ in range(30):
            less = tuple(size(m) for m in most)
            said = _refusal(*less, *heads, have, rng.choice([0, 1, 2]))
            assert said == "out is null", f"{less} of {most}, {heads}: {said}"
            assert glsa.attention_workspace_bytes(*less, *heads) <= have
            served += _refusal(*less, *heads, 0) != "out is null"
    assert served > 1000  # calls that do need one


def test_a_workspace_has_a_bound():
    """Rows beyond what the sequences can have (a padded batch) take no room: at
    most 1024 chunks of 32 rows, 512 of 128 or 256 of 256 are in flight, and a
    sequence more than an even share of them."""
    for sizes in [(256, 8192, 512, 131072, 32, 8, 128), (1, 1 << 20, 1, 131072, 32, 8, 128), (64, 1 << 20, 1024, 1 << 20, 8, 1, 256)]:
        need = glsa.attention_workspace_bytes(*sizes)
        assert 0 < need <= 2 * 256 * 256 * (sizes[-1] + 2) * 4, sizes
    assert glsa.attention_workspace_bytes(256, 256, 1, 200, 32, 8, 128) == 0  # never more than one chunk


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_one_workspace_on_the_gpu(dtype):
    """Calls of many sizes in a workspace for the largest give what they give in
    one of their own; rows past the sequences' do not change that."""
    hq, hk, d, page, B, ctx = 8, 2, 64, 64, 24, 6000
    g = torch.Generator("cuda").manual_seed(3)
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    per = -(-(ctx + 40) // page)
    pages = torch.randperm(B * per, generator=g, device="cuda").to(torch.int32).view(B, per)
    k, v = (torch.empty(B * per, hk, page, d, device="cuda", dtype=dtype).normal_(generator=g) for _ in range(2))
    shared = glsa.alloc_attention_workspace(B, B * 40 + 100, 40, ctx, hq, hk, d, "cuda")
    some = 0
    for n_seqs, nodes, context, pad in [(24, 40, 6000, 0), (24, 1, 6000, 0), (3, 1, 6000, 0), (1, 1, 5000, 0), (2, 40, 6000, 0),
                                        (1, 9, 6000, 100), (3, 40, 5990, 100), (5, 3, 300, 7)]:
        T = n_seqs * nodes
        q = torch.empty(T + pad, hq * d, device="cuda", dtype=dtype).normal_(generator=g)
        args = (k, v, pages[:n_seqs], ints([context - 13 * b for b in range(n_seqs)]), ints([b * nodes for b in range(n_seqs + 1)]))
        kw = dict(max_nodes=nodes, max_context=context)
        own = glsa.alloc_attention_workspace(n_seqs, T, nodes, context, hq, hk, d, "cuda").fill_(0xFF)
        some += own.numel() > 0
        want = glsa.tree_attention(q[:T], *args, workspace=own, **kw)
        out = torch.full((T + pad, hq * d), 99.0, device="cuda", dtype=dtype)
        glsa.tree_attention(q, *args, out=out, workspace=shared.fill_(0xFF), **kw)
        assert torch.equal(out[:T], want) and bool((out[T:] == 99).all()) and bool(torch.isfinite(want).all())
    assert some > 5


# ---- numbers that the C ABI has 32 bits for --------------------------------------

def _attend_args(page=8, columns=4):
    ints = torch.tensor([0, 2], dtype=torch.int32)
    cache = torch.ones(1, 1, page, 8)
    return torch.ones(2, 8), cache, cache, torch.zeros(1, columns, dtype=torch.int32), ints[:1], ints


def test_a_wide_page_table_bounds_no_context_away(no_library):
    """The default max_context is what the table holds, as far as positions go: cut
    to its low 32 bits it made contexts of none."""
    for page, columns, nodes, want in [(8, 4, 2, 32), (4096, 1 << 20, 2, (1 << 31) - 3), (4096, 1 << 19, 7, (1 << 31) - 8),
                                       (4096, (1 << 19) - 1, 1, (1 << 31) - 4096)]:
        glsa.tree_attention(*_attend_args(page, columns), max_nodes=nodes)
        assert no_library.args[14:16] == (nodes, want)


@pytest.mark.parametrize("number", [1 << 32, (1 << 32) + 64, -(1 << 32) + 64, 1 << 31, 1 << 64])
def test_numbers_past_32_bits_are_refused(number):
    """ctypes would pass their low 32 bits on."""
    calls = [lambda: glsa.rope_frequencies(number), lambda: glsa.rope_table(4, number)]
    calls += [lambda i=i: glsa.attention_workspace_bytes(*[number if j == i else 64 for j in range(7)]) for i in range(7)]
    for call in calls:
        with pytest.raises(glsa.LoraError) as e:
            call()
        assert e.value.status == BAD


@pytest.mark.parametrize("number", [1 << 32, (1 << 32) + 64, -(1 << 32) + 64, 1 << 31])
def test_numbers_past_32_bits_are_refused_by_the_calls(number, no_library):
    q, cache, _, table, context, ints = _attend_args()
    for call in (lambda: glsa.tree_attention(q, cache, cache, table, context, ints, max_nodes=number),
                 lambda: glsa.tree_attention(q, cache, cache, table, context, ints, max_nodes=2, max_context=number),
                 lambda: glsa.build_tree(None, ints, context, max_nodes=number, n_tokens=2),
                 lambda: glsa.build_tree(None, ints, context, max_nodes=2, n_tokens=number, positions=ints),
                 lambda: glsa.build_tree(None, ints, context, max_nodes=2, n_tokens=2, page_table=table, n_pages=1,
                                         page_size=number),
                 lambda: glsa.rotary(q[:, :0], q[:, :0], ints, q, head_dim=number),
                 lambda: glsa.rope_table(1, 8, frequencies=[1.0] * 4, first=number << 32, device="cpu")):
        with pytest.raises(glsa.LoraError) as e:
            call()
        assert e.value.status == BAD


def test_cache_rows_take_the_caches_sizes(no_library):
    """Without them every row would come out as missing, and rotary would then place
    nothing in the cache."""
    _, _, _, table, context, ints = _attend_args()
    for sizes in ({}, dict(n_pages=4), dict(page_size=8)):
        with pytest.raises(glsa.LoraError, match="n_pages and page_size"):
            glsa.build_tree(None, ints, context, max_nodes=2, n_tokens=2, page_table=table, **sizes)
    glsa.build_tree(None, ints, context, max_nodes=2, n_tokens=2, page_table=table, n_pages=4, page_size=8)
    assert no_library.args[9:11] == (4, 8)
    glsa.build_tree(None, ints, context, max_nodes=2, n_tokens=2)


# ---- bounds past what a launch holds ---------------------------------------------

@pytest.mark.parametrize("sizes", [
    (65535, 4, 1 << 26, (1 << 31) - (1 << 26) - 2, 1024, 1024, 8),  # keys times workgroups pass 64 bits
    (65535, 4, 1 << 20, 4096, 32, 8, 128), (8192, 8192, 65536, 0, 16, 16, 256),
    (1, 4, 1 << 26, (1 << 31) - (1 << 26) - 2, 1, 1, 8),            # two chunks, too many rows to join in one launch
    (65535, 65535, 1, 100, 1024, 1024, 8)])
def test_bounds_past_a_launch_are_refused(sizes):
    """A launch holds fewer than 2^32 threads in a dimension of its grid."""
    for dtype in (0, 1, 2):
        assert "launch" in _refusal(*sizes, 1 << 60, dtype, glsa.LORA_ERR_UNSUPPORTED)


@pytest.mark.parametrize("sizes", [(256, 8192, 512, 131072, 32, 8, 128), (1, 1, 1, (1 << 31) - 2, 32, 8, 128),
                                   (4096, 8192, 512, 131072, 32, 8, 128), (65535, 65535, 1, 4096, 32, 8, 128),
                                   (1, 65536, 65536, 0, 64, 8, 128)])
def test_large_bounds_are_served(sizes):
    for dtype in (0, 1, 2):
        assert _refusal(*sizes, 1 << 60, dtype) == "out is null"


@pytest.mark.parametrize("T,hq,hk,d,rot,refused", [
    (1 << 28, 1, 1, 8, 8, True), (1 << 25, 32, 8, 256, 256, True), (1 << 25, 32, 8, 80, 20, True),
    (1 << 23, 32, 8, 256, 256, False), (1 << 22, 32, 8, 80, 20, False), (1 << 25, 32, 8, 64, 64, False)])
def test_rotations_past_a_launch_are_refused(T, hq, hk, d, rot, refused):
    cache = A._CACHE_FIELDS.pack(FAKE, FAKE, 0, 0, 0, 0, 0, 0, 4, 16)
    st = A._lib().lora_rotary(1, FAKE, hq * d, FAKE, hk * d, FAKE, hk * d, T, hq, hk, d, 0, rot, FAKE, 16, FAKE, FAKE, hq * d,
                              FAKE, hk * d, cache, None, None)  # without cache_rows: refused at the latest for that
    said = glsa.lib().lora_last_error().decode()
    assert (st, "launch" in said) == ((glsa.LORA_ERR_UNSUPPORTED, True) if refused else (BAD, False)), said
