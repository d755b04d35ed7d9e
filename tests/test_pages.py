"""GPU: the pool's calls and copy_pages against the reference, entry by entry.
Whole numbers and bytes: everything is equal."""

import numpy as np
import pytest
import torch

import gemm_lora_shrink_amd as glsa
from oracle import cache_oracle as co

pytestmark = pytest.mark.gpu


def ints(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device="cuda")


class Pool:
    """Sequences of the given lengths on random pages of a pool."""

    def __init__(self, lengths, page, n_pages, columns=None, seed=0, shared=0):
        rng = np.random.default_rng(seed)
        self.lengths, self.page = np.array(lengths, np.int32), page
        held = -(-self.lengths // page)
        columns = columns or max(int(held.max(initial=0)), 1)
        order = list(rng.permutation(n_pages))
        self.table = np.full((len(lengths), columns), -1, np.int32)
        for b, n in enumerate(held):
            for c in range(n):
                self.table[b, c] = self.table[b - 1, c] if b and c < shared and self.table[b - 1, c] >= 0 else order.pop()
        self.refs = np.zeros(n_pages, np.int32)
        for e in self.table[self.table >= 0]:
            self.refs[e] += 1

    def on_gpu(self):
        return ints(self.refs), ints(self.table)

    def tensors(self, seed=0):
        """Paged tensors of several kinds: a 16-bit cache, the same with its rows first, bytes,
        exponents, and a part of the heads of a wider cache."""
        g = torch.Generator("cuda").manual_seed(seed)
        n, page = len(self.refs), self.page
        wide = torch.randn(n, 4, page, 24, generator=g, device="cuda").half()
        return [torch.randn(n, 2, page, 40, generator=g, device="cuda").bfloat16(),
                torch.randn(n, page, 2, 40, generator=g, device="cuda").transpose(1, 2),
                torch.randint(0, 255, (n, 2, page, 16), generator=g, device="cuda").to(torch.uint8).view(torch.float8_e4m3fn),
                torch.randint(-9, 9, (n, 2, 3), generator=g, device="cuda").to(torch.int8), wide[:, 1:3], wide[:, 3:, :, :8],
                torch.randn(n, 5, generator=g, device="cuda")]


def raw(t):
    return t.contiguous().view(torch.uint8).cpu().numpy().reshape(t.size(0), -1)


def moved(before, pairs):
    out = before.copy()
    for of, to in pairs:
        out[to] = before[of]
    return out


@pytest.mark.parametrize("case", range(5))
def test_copy_pages(case):
    rng = np.random.default_rng(case)
    n, page = [(2, 1), (9, 8), (64, 16), (200, 24), (3000, 16)][case]
    p = Pool([], page, n)
    tensors = p.tensors(case)
    before = [raw(t) for t in tensors]
    order = rng.permutation(n)
    m = n // 2
    pairs = list(zip(order[:m], order[m:2 * m]))
    source, target = [a for a, _ in pairs] + [-1, 0, n], [b for _, b in pairs] + [0, -1, 0]
    glsa.copy_pages(tensors, ints(source), ints(target))
    for t, x in zip(tensors, before):
        assert np.array_equal(raw(t), moved(x, pairs))
    # a count from the GPU, and the tensors laid out once
    kept = glsa.PagedTensors(tensors)
    before = [raw(t) for t in tensors]
    glsa.copy_pages(kept, ints([b for _, b in pairs]), ints([a for a, _ in pairs]), count=ints([m // 2]))
    for t, x in zip(tensors, before):
        assert np.array_equal(raw(t), moved(x, [(b, a) for a, b in pairs[:m // 2]]))
    glsa.copy_pages(kept, ints([0]), ints([1]), count=ints([0]))
    glsa.copy_pages(kept, ints([]), ints([]))
    for t, x in zip(tensors, before):
        assert np.array_equal(raw(t), moved(x, [(b, a) for a, b in pairs[:m // 2]]))


def test_copy_pages_of_many_tensors_and_past_4_gib():
    n = 70000
    big = torch.zeros(n, 8, 64, 128, dtype=torch.uint8, device="cuda")  # 4.6 GB
    big[5], big[69999] = 3, 7
    small = [torch.full((n, 2), i, dtype=torch.int16, device="cuda") for i in range(130)]
    for t in small:
        t[5] = -1
    glsa.copy_pages([big, *small], ints([69999, 5]), ints([1, 69998]))
    assert bool((big[1] == 7).all()) and bool((big[69998] == 3).all()) and not big[2:5].any() and not big[69997].any()
    for i, t in enumerate(small):
        assert bool((t[69998] == -1).all()) and bool((t[[0, 1, 2, 69997, 69999]] == i).all())


@pytest.mark.parametrize("case", range(6))
def test_reserve(case):
    rng = np.random.default_rng(case)
    lengths, page, n = [([0], 16, 1), ([5, 0, 33], 8, 40), (list(range(0, 400, 3)), 16, 5000), ([7] * 2000, 4, 9000),
                        ([10, 20, 30], 8, 9), ([100000], 16, 20000)][case]
    columns = -(-(max(lengths) * 2 + 40) // page)
    p = Pool(lengths, page, n, columns, seed=case)
    want = p.lengths + rng.integers(-3, 40, len(lengths)).astype(np.int32)
    if case == 5:
        want[0] = 199000
    if case == 2:
        p.table[3, :2] = (-7, n)  # entries that name no page
        want[5] = 2 ** 31 - 1     # more than the table has columns
        want[6] = -4
    refs, table = p.on_gpu()
    missing = ints([77])
    n_missing = co.reserve(p.refs, p.table, want, page)
    ws = glsa.alloc_pages_workspace(n, len(lengths), "cuda").fill_(0xFF)
    glsa.reserve_pages(refs, table, ints(want), page_size=page, missing=missing, workspace=ws)
    assert np.array_equal(table.cpu().numpy(), p.table) and np.array_equal(refs.cpu().numpy(), p.refs)
    assert int(missing) == n_missing and (n_missing > 0 or case != 4)
    glsa.reserve_pages(refs, table, ints(want), page_size=page)  # once more changes nothing
    assert np.array_equal(table.cpu().numpy(), p.table) and np.array_equal(refs.cpu().numpy(), p.refs)


@pytest.mark.parametrize("case", range(6))
def test_fork(case):
    rng = np.random.default_rng(case)
    B, longest, page, n = [(1, 5, 16, 3), (4, 90, 8, 120), (64, 300, 16, 4000), (1500, 40, 4, 40000), (6, 50, 8, 45),
                           (3, 3000, 16, 2000)][case]
    p = Pool(rng.integers(0, longest + 1, B), page, n, -(-longest // page), seed=case, shared=2)
    p.lengths[0] = longest if case == 0 else p.lengths[0]
    parents = rng.integers(0, B, B)
    lengths = np.array([rng.integers(0, p.lengths[x] + 1) if rng.random() < 0.5 else p.lengths[x] for x in parents])
    children = rng.permutation(B)
    if case == 1:
        parents[1], children[2], lengths[3] = -1, B, -5
    if case == 2:
        parents[1], parents[2], children[3], lengths[4] = B, -7, -1, 10 ** 6  # longer than its parent and the table
        p.table[parents[6], 0] = -1
    refs, table = p.on_gpu()
    to = torch.full_like(table, 99)
    tensors = p.tensors()
    before = [raw(t) for t in tensors]
    new, missing = np.full_like(p.table, 99), ints([55])
    pairs, n_missing = co.fork(p.refs, p.table, new, parents, children, lengths, page)
    got = glsa.fork_sequences(refs, table, ints(parents), ints(children), ints(lengths), page_size=page, tensors=tensors,
                              out_table=to, missing=missing)
    assert got is to
    assert np.array_equal(to.cpu().numpy(), new) and np.array_equal(refs.cpu().numpy(), p.refs)
    assert np.array_equal(table.cpu().numpy(), p.table) and int(missing) == n_missing
    for t, x in zip(tensors, before):
        assert np.array_equal(raw(t), moved(x, pairs))
    assert case in (0, 4) or pairs


def test_fork_in_one_table_without_tensors():
    p = Pool([37, 12, 0, 0], 8, 20, 6)
    refs, table = p.on_gpu()
    pairs, _ = co.fork(p.refs, p.table, p.table, [0, 1], [2, 3], [37, 8], 8)
    glsa.fork_sequences(refs, table, ints([0, 1]), ints([2, 3]), ints([37, 8]), page_size=8)
    assert np.array_equal(table.cpu().numpy(), p.table) and np.array_equal(refs.cpu().numpy(), p.refs) and len(pairs) == 1
    glsa.fork_sequences(refs, table, ints([]), ints([]), ints([]), page_size=8)
    assert np.array_equal(table.cpu().numpy(), p.table)


@pytest.mark.parametrize("case", range(4))
def test_release(case):
    rng = np.random.default_rng(case)
    p = Pool(rng.integers(0, 200, 40), 16, 700, 14, seed=case, shared=3)
    rows, keep = [(None, None), ([3, 9, 3, -1, 40, 0], None), (list(range(40)), rng.integers(-5, 220, 40)),
                  (None, rng.integers(0, 100, 40))][case]
    refs, table = p.on_gpu()
    co.release(p.refs, p.table, range(40) if rows is None else rows, keep, 16)
    glsa.release_pages(refs, table, None if rows is None else ints(rows), keep=None if keep is None else ints(keep),
                       page_size=None if keep is None else 16)
    assert np.array_equal(table.cpu().numpy(), p.table) and np.array_equal(refs.cpu().numpy(), p.refs)


@pytest.mark.parametrize("case", range(6))
def test_compact(case):
    rng = np.random.default_rng(case)
    lengths, page, n = [([], 16, 5), ([40], 8, 5), (rng.integers(0, 300, 30), 16, 700), (rng.integers(1, 40, 3000), 4, 33000),
                        ([16], 16, 1), (rng.integers(0, 60, 9), 8, 4097)][case]
    p = Pool(lengths, page, n, -(-max([1, *lengths]) // page) + 1, seed=case, shared=2)
    if case == 2:
        co.release(p.refs, p.table, range(0, 30, 2), None, page)
        p.table[1, -1], p.table[3, -1] = -9, n + 5
    refs, table = p.on_gpu()
    tensors = p.tensors()
    before = [raw(t) for t in tensors]
    n_live, moves = co.compact(p.refs, p.table)
    ws = glsa.alloc_pages_workspace(n, 1, "cuda").fill_(0xFF)
    got = glsa.compact_pages(refs, table, tensors=tensors, workspace=ws)
    assert int(got) == n_live and np.array_equal(refs.cpu().numpy(), p.refs) and np.array_equal(table.cpu().numpy(), p.table)
    assert not p.refs[n_live:].any() and (p.refs[:n_live] > 0).all()
    for t, x in zip(tensors, before):
        assert np.array_equal(raw(t), moved(x, moves))


def test_pool_calls_replay_from_a_graph():
    """A step of beams captured: fork into another table, release, reserve, compact."""
    p = Pool([70, 33, 16, 5], 8, 90, 12)
    refs, table = p.on_gpu()
    start = refs.clone(), table.clone()
    tensors = glsa.PagedTensors(p.tensors())
    contents = [t.clone() for t in tensors.tensors]
    parents, children, lengths, more = ints([1, 0, 3, 0]), ints([0, 1, 2, 3]), ints([33, 70, 5, 64]), ints([40, 77, 9, 65])
    to, ws = torch.empty_like(table), glsa.alloc_pages_workspace(90, 4, "cuda")
    n_live, missing = ints([0]), ints([0])

    def step():
        glsa.fork_sequences(refs, table, parents, children, lengths, page_size=8, tensors=tensors, out_table=to, workspace=ws)
        glsa.release_pages(refs, table)
        glsa.reserve_pages(refs, to, more, page_size=8, missing=missing, workspace=ws)
        glsa.compact_pages(refs, to, tensors=tensors, n_live=n_live, workspace=ws)

    def reset():
        refs.copy_(start[0])
        table.copy_(start[1])
        to.fill_(5)
        for t, x in zip(tensors.tensors, contents):
            t.copy_(x)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in range(3):
        g = torch.Generator("cuda").manual_seed(seed)
        parents.copy_(torch.randint(0, 4, (4,), generator=g, device="cuda"))
        lengths.copy_(ints([70, 33, 16, 5])[parents.long()])
        more.copy_(lengths + 9)
        reset()
        step()
        want = [t.clone() for t in (refs, table, to, n_live, missing, *tensors.tensors)]
        reset()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip((refs, table, to, n_live, missing, *tensors.tensors), want):
            assert np.array_equal(raw(a.reshape(1, -1)), raw(b.reshape(1, -1)))
        assert int(n_live) == int((refs > 0).sum()) and int(missing) == 0


def test_forked_sequences_attend_as_copies_do():
    """A prompt in a quantized cache, forked: each beam goes on with tokens of its own and
    attends as if its whole past had been copied; then pages are given back and compacted."""
    hk, d, page, n_pages, B = 2, 64, 16, 60, 4
    g = torch.Generator("cuda").manual_seed(0)
    cache = glsa.alloc_quantized_cache(n_pages, hk, page, d, "cuda", block=8)
    refs, table = torch.zeros(n_pages, dtype=torch.int32, device="cuda"), torch.full((B, 6), -1, dtype=torch.int32, device="cuda")
    ws = glsa.alloc_pages_workspace(n_pages, B, "cuda")
    prompt, steps = 37, 20
    kv = torch.randn(prompt + B * steps, 2 * hk * d, generator=g, device="cuda").bfloat16()
    q = torch.randn(B * steps, 8 * d, generator=g, device="cuda").bfloat16()
    paged = glsa.PagedTensors(cache)

    def rows(n, start, context):
        return glsa.build_tree(None, start, context, max_nodes=max(n), n_tokens=sum(n), page_table=table, n_pages=n_pages,
                               page_size=page)[2]

    one = ints([prompt, 0, 0, 0])
    glsa.reserve_pages(refs, table, one, page_size=page, workspace=ws)
    glsa.store_quantized(kv[:prompt, :hk * d], kv[:prompt, hk * d:], cache,
                         rows([prompt, 0, 0, 0], ints([0, prompt, prompt, prompt, prompt]), ints([0] * 4)))
    glsa.fork_sequences(refs, table, ints([0, 0, 0]), ints([1, 2, 3]), ints([prompt] * 3), page_size=page, tensors=paged,
                        workspace=ws)
    assert refs[table[0, :2].long()].tolist() == [4, 4] and int((refs == 1).sum()) == 4
    context = torch.full((B,), prompt, dtype=torch.int32, device="cuda")
    start = ints([0, 1, 2, 3, 4])
    # the same beams, each in a cache that holds a copy of everything
    alone = glsa.alloc_quantized_cache(B * 6, hk, page, d, "cuda", block=8)
    own = torch.arange(B * 6, dtype=torch.int32, device="cuda").view(B, 6)
    for b in range(B):
        for c in range(3):
            for x, y in zip(alone, cache):
                x.view(torch.uint8)[b * 6 + c] = y.view(torch.uint8)[int(table[b, c])]
    outs = []
    for i in range(steps):
        new = kv[prompt + i * B:prompt + (i + 1) * B]
        glsa.reserve_pages(refs, table, context + 1, page_size=page, workspace=ws)
        if i == 11:
            glsa.compact_pages(refs, table, tensors=paged, workspace=ws)
        glsa.store_quantized(new[:, :hk * d], new[:, hk * d:], cache, rows([1] * B, start, context))
        at = own.gather(1, (context // page).long()[:, None])[:, 0] * page + context % page
        glsa.store_quantized(new[:, :hk * d], new[:, hk * d:], alone, at)
        for c, t in ((cache, table), (alone, own)):
            w = glsa.alloc_quantized_workspace(B, B, 1, 96, 8, hk, d, "cuda")
            outs.append(glsa.tree_attention_quantized(q[i * B:(i + 1) * B], c, t, context, start, max_nodes=1,
                                                      max_context=96, workspace=w))
        context += 1
    for a, b in zip(outs[::2], outs[1::2]):
        assert torch.equal(a, b)
    assert float((outs[-1][0] - outs[-1][1]).abs().max()) > 0.01
    glsa.release_pages(refs, table, ints([0, 2]))
    glsa.release_pages(refs, table, ints([1, 3]), keep=ints([10, 0]), page_size=page)
    assert int(refs.sum()) == 1 and int((table >= 0).sum()) == 1


def test_calls_of_nothing():
    """No sequences, no forks, no rows, no columns and an empty pool: nothing but the counts is written."""
    refs, table, none, missing = ints([0, 2, 0, 1]), ints([[1, 3], [1, -1]]), ints([]), ints([7])
    was = refs.clone(), table.clone()
    for t in (torch.empty(0, 5, dtype=torch.int32, device="cuda"), torch.empty(3, 0, dtype=torch.int32, device="cuda")):
        missing.fill_(7)
        glsa.reserve_pages(refs, t, torch.full((t.size(0),), 9, dtype=torch.int32, device="cuda"), page_size=4, missing=missing)
        assert int(missing) == 0
        glsa.release_pages(refs, t)
    missing.fill_(7)
    glsa.fork_sequences(refs, table, none, none, none, page_size=4, missing=missing)
    glsa.release_pages(refs, table, none)
    assert int(missing) == 0 and torch.equal(refs, was[0]) and torch.equal(table, was[1])
    missing.fill_(7)
    held = torch.full((2, 3), -1, dtype=torch.int32, device="cuda")
    glsa.reserve_pages(none, held, ints([1, 9]), page_size=4, missing=missing)
    assert int(missing) == 4 and bool((held == -1).all())
    assert int(glsa.compact_pages(none, held)) == 0


def test_calls_on_another_stream():
    """The calls follow the work of the stream that they are given, workspaces made within them too."""
    pool, s = Pool([70, 33, 0, 129], 16, 60), torch.cuda.Stream()
    refs, table = pool.on_gpu()
    tensors = pool.tensors()
    want_refs, want_table = refs.clone(), table.clone()
    want = [t.clone() for t in tensors]
    lengths, forks = ints([80, 40, 20, 130]), [ints(x) for x in ([0, 3], [2, 1], [37, 100])]

    def calls(refs, table, tensors, **kw):
        glsa.release_pages(refs, table, forks[1], **kw)
        glsa.fork_sequences(refs, table, *forks, page_size=16, tensors=tensors, **kw)
        glsa.reserve_pages(refs, table, lengths, page_size=16, **kw)
        return glsa.compact_pages(refs, table, tensors=tensors, **kw)

    live = int(calls(want_refs, want_table, want))
    torch.cuda.synchronize()
    late = refs.clone().zero_(), table.clone().fill_(-1)
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)
        late[0].copy_(refs)
        late[1].copy_(table)
    got = calls(*late, tensors, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert int(got) == live and torch.equal(late[0], want_refs) and torch.equal(late[1], want_table)
    held = sorted(set(want_table[want_table >= 0].tolist()))
    for a, b in zip(tensors, want):
        assert np.array_equal(raw(a)[held], raw(b)[held])
