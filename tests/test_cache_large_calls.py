"""GPU: stores of more tokens, and pools of more pages, than one round of a
workgroup takes.  Whole numbers and bytes: everything is equal to the reference."""

import numpy as np
import pytest
import torch

import gemm_lora_shrink_amd as glsa
from oracle import cache_oracle as co
from test_quantized_cache import TYPES, equal, f64, ints, made, on_host, rows_of

pytestmark = pytest.mark.gpu

PROMPTS = [  # contexts, counts, hk, d, page, block: more than 1024 tokens in all
    ([0, 5, 100], [700, 333, 64], 2, 32, 16, 16), ([3, 0, 17, 64], [1100, 1, 15, 16], 1, 48, 128, 128),
    ([1], [1040], 3, 16, 8, 1), (list(range(40)), [26 + b % 3 for b in range(40)], 5, 16, 24, 8),
]


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("case", range(len(PROMPTS)))
def test_store_of_prompts(case, dt, fmt):
    contexts, counts, hk, d, page, block = PROMPTS[case]
    g, rng = torch.Generator("cuda").manual_seed(case), np.random.default_rng(case)
    B, T = len(contexts), sum(counts)
    assert T > 1024
    per = max(-(-(c + n) // page) for c, n in zip(contexts, counts))
    n_pages = B * per + 3
    table = rng.permutation(n_pages)[:B * per].reshape(B, per)
    cache = made(n_pages, hk, page, d, fmt, block, g, rows_first=case % 2 == 0, spread=3)
    rows = torch.randn(T, 2 * hk * d + 8, generator=g, device="cuda") * torch.exp(2 * torch.randn(T, 1, generator=g, device="cuda"))
    rows[7], rows[600, 3::5], rows[1023, 1], rows[1024, hk * d] = 0, float("inf"), float("nan"), -float("inf")
    rows = rows.to(TYPES[dt])
    k, v = rows[:, :hk * d], rows[:, hk * d:2 * hk * d]
    at = rows_of(table, contexts, counts, page)
    of = at // block
    at[np.isin(of, rng.choice(of, T // 50))] = -1  # blocks that are not placed
    want = co.store(on_host(cache), f64(k).reshape(T, hk, d), f64(v).reshape(T, hk, d), at)
    glsa.store_quantized(k, v, cache, ints(at))
    equal(cache, want)


def compact(refs, table):
    """co.compact with the renaming of all pages at once."""
    n = int((refs > 0).sum())
    p = np.arange(len(refs))
    of, to = p[(p >= n) & (refs > 0)], p[(p < n) & (refs <= 0)]
    now = p.copy()
    now[of] = to
    refs[to], refs[of] = refs[of], 0
    table[:] = now[table]
    return n, of


@pytest.mark.parametrize("n", [65536, 65537, 200000])
def test_pools_of_many_pages(n):
    rng = np.random.default_rng(n)
    B, cols, page = 50, 700, 16
    held = rng.permutation(n)[:B * cols].reshape(B, cols).astype(np.int32)
    held[rng.random(held.shape) < 0.3] = -1
    held[0, :5], held[1, 0] = held[2, :5], n - 1 if n - 1 not in held else held[1, 0]
    refs = np.bincount(held[held >= 0], minlength=n).astype(np.int32)
    got_refs, table = ints(refs), ints(held)
    x = torch.arange(n, device="cuda", dtype=torch.int32)[:, None] * 3
    content = np.arange(n) * 3
    names = np.where(held >= 0, content[held], -1)
    # sequences grow, then the pool is compacted
    lengths = np.full(B, cols * page)
    missing = ints([9])
    lacking = co.reserve(refs, held, lengths, page)
    glsa.reserve_pages(got_refs, table, ints(lengths), page_size=page, missing=missing)
    assert int(missing) == lacking
    names = np.where(names >= 0, names, np.where(held >= 0, content[held], -1))
    assert np.array_equal(table.cpu().numpy(), held) and np.array_equal(got_refs.cpu().numpy(), refs)
    live, moves = compact(refs, held)
    assert int(glsa.compact_pages(got_refs, table, tensors=[x])) == live and live < n
    assert np.array_equal(table.cpu().numpy(), held) and np.array_equal(got_refs.cpu().numpy(), refs)
    assert np.array_equal(x[:, 0].cpu().numpy()[held], names)
    assert len(moves)


def test_moves_across_spans_of_a_large_pool():
    """Pages in use at both ends of a pool: the free ones between them are taken in order."""
    n = 300000
    rng = np.random.default_rng(0)
    used = np.unique(np.concatenate([rng.integers(0, 70000, 30000), rng.integers(200000, n, 60000), [0, n - 1, 65535, 65536]]))
    refs = np.zeros(n, np.int32)
    refs[used] = rng.integers(1, 4, len(used))
    table = rng.permutation(used)[None].astype(np.int32)
    got_refs, got = ints(refs), ints(table)
    x = torch.arange(n, device="cuda", dtype=torch.int32)[:, None] * 5
    names = table * 5
    live, moves = compact(refs, table)
    assert int(glsa.compact_pages(got_refs, got, tensors=[x])) == live and len(moves) > 65536 // 4
    assert np.array_equal(got.cpu().numpy(), table) and np.array_equal(got_refs.cpu().numpy(), refs)
    assert np.array_equal(x[:, 0].cpu().numpy()[table], names)
