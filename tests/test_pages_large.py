"""GPU: copies of more bytes than the last-level cache holds, which go past the
caches, with accesses of 16, 4 and 1 bytes, whole pages and pages in pieces, and
small pages beside them.  Bytes: everything is equal."""

import numpy as np
import pytest
import torch

import gemm_lora_shrink_amd as glsa

pytestmark = pytest.mark.gpu

N = 1600


def ints(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device="cuda")


def pages(seed):
    g = torch.Generator("cuda").manual_seed(seed)

    def bytes_of(*shape):
        return torch.randint(0, 256, (N, *shape), generator=g, device="cuda", dtype=torch.int32).to(torch.uint8)

    parts, odd = bytes_of(2, 64, 512), bytes_of(3, 41, 1001)
    return [bytes_of(120, 1024), bytes_of(60004), bytes_of(50001), parts[:, :, :48], odd[:, :2, :40, 3:1000], bytes_of(7),
            bytes_of(2, 16)]


def bound(tensors, pairs):
    return sum(2 * t[0].numel() * t.element_size() * pairs for t in tensors)


def test_copies_past_the_caches():
    tensors = pages(0)
    before = [t.clone() for t in tensors]
    order = np.random.default_rng(0).permutation(N)
    source, target = order[:N // 2], order[N // 2:]
    assert bound(tensors, N // 2) > 1 << 29
    glsa.copy_pages(tensors, ints(source), ints(target))
    for t, x in zip(tensors, before):
        x[torch.tensor(target, device="cuda")] = x[torch.tensor(source, device="cuda")]
        assert torch.equal(t, x)


@pytest.mark.parametrize("live", [3, N // 2 + 7])
def test_compacting_a_large_pool(live):
    """The bound on the moves decides how they are copied, however few there are."""
    tensors = pages(1)
    before = [t.clone() for t in tensors]
    held = np.sort(np.random.default_rng(1).permutation(N)[:live])
    refs = np.zeros(N, np.int32)
    refs[held] = 1
    got, table = ints(refs), ints(held[None])
    assert int(glsa.compact_pages(got, table, tensors=tensors)) == live
    assert got.tolist() == [1] * live + [0] * (N - live)
    now = table[0].long()
    assert sorted(now.tolist()) == list(range(live))
    for t, x in zip(tensors, before):
        assert torch.equal(t[now], x[torch.tensor(held, device="cuda")])
