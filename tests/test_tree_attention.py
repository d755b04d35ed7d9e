"""GPU: build_tree, tree_attention and keep_path against the fp64 reference.

Tolerances.  h = finfo.eps / 2 is half a step of the type, u = 2^-24.  With A
the softmax-weighted mean of |v| and z the row's largest scale * sum |q| |k|:
 - a score is a dot product of d terms in fp32: off by ds <= (d + 2) u z;
   every weight's exponential by 4 u, and by u times its argument (<= 2 z + ds
   in absolute value), which moves the weighted mean by at most
   2 (ds + (4 + 2 z) u) A;
 - weights of a product with 16-bit v are rounded to the type, h A (nothing in
   fp32);
 - the sums run over L keys: 2 L u A for the numerator and the denominator;
 - the output is rounded once: h |o|, or the type's smallest step; it is also
   put together from at most 64 parts, 8 u A.
The same terms without A bound lse."""

import math

import numpy as np
import pytest
import torch

import gemm_lora_shrink_amd as glsa
from oracle import attention_oracle as ao

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
U = 2.0 ** -24


def half_step(dt):
    return torch.finfo(dt).eps / 2


def f64(t):
    return t.detach().double().cpu().numpy()


def ints(v, dtype=torch.int32):
    return torch.tensor(np.asarray(v), dtype=dtype, device="cuda")


class Step:
    """A step's inputs: B sequences with the given contexts and node counts."""

    def __init__(self, contexts, counts, hq, hk, d, dt, *, page=16, seed=0, tree=True, spare=3, pad=0, q_scale=1.0,
                 rows_first=False):
        rng = np.random.default_rng(seed)
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.rng, self.g, self.dt, self.page, self.d, self.hq, self.hk = rng, g, dt, page, d, hq, hk
        self.context, self.counts, self.B = list(contexts), list(counts), len(contexts)
        self.q_start = np.concatenate([[0], np.cumsum(counts)]).astype(int)
        self.T = int(self.q_start[-1])
        per = max([-(-(c + n) // page) for c, n in zip(contexts, counts)] + [1]) + 1
        self.n_pages = self.B * per + spare
        self.table = rng.permutation(self.n_pages)[:self.B * per].reshape(self.B, per).astype(np.int32)
        shape = (self.n_pages, page, hk, d) if rows_first else (self.n_pages, hk, page, d)
        self.k, self.v = (torch.empty(shape, dtype=dt, device="cuda").normal_(0, 1, generator=g) for _ in range(2))
        if rows_first:
            self.k, self.v = self.k.transpose(1, 2), self.v.transpose(1, 2)
        self.rows = torch.empty(self.T, hq * d + pad, dtype=dt, device="cuda").normal_(0, q_scale, generator=g)
        self.q = self.rows[:, :hq * d]
        self.parents = None
        if tree:
            self.parents = [[int(rng.integers(-1, j)) if j else -1 for j in range(n)] for n in counts]
        self.sees = [ao.ancestors(self.parents[b]) if tree else np.tril(np.ones((n, n), bool))
                     for b, n in enumerate(counts)]
        self.max_nodes = max(list(counts) + [1])
        self.max_context = max(list(contexts) + [0])

    def mask(self):
        if self.parents is None:
            return None
        words = -(-self.max_nodes // 64)
        out = np.zeros((self.T, words), np.uint64)
        for b in range(self.B):
            for i in range(self.counts[b]):
                for j in np.nonzero(self.sees[b][i])[0]:
                    out[self.q_start[b] + i, j // 64] |= np.uint64(1) << np.uint64(j % 64)
        return ints(out.view(np.int64), torch.int64)

    def used_rows(self):
        """[n_pages, page] booleans: rows of some sequence's context or nodes."""
        used = np.zeros(self.n_pages * self.page, bool)
        for b in range(self.B):
            r = ao.cache_rows_of(self.table[b], np.arange(self.context[b] + self.counts[b]), self.page, self.n_pages)
            used[r[r >= 0]] = True
        return used.reshape(self.n_pages, self.page)

    def poison_unused(self, value=float("nan")):
        unused = torch.from_numpy(~self.used_rows()).cuda()
        for c in (self.k, self.v):
            c.masked_fill_(unused[:, None, :, None], value)

    def workspace(self, fill=None, nodes=None, ctx=None):
        ws = glsa.alloc_attention_workspace(self.B, self.T, nodes or self.max_nodes,
                                            self.max_context if ctx is None else ctx, self.hq, self.hk, self.d, "cuda")
        return ws.fill_(0xFF) if fill is None else ws.fill_(fill)  # every float a NaN: nothing may rely on it

    def run(self, **kw):
        lse = torch.full((self.T, self.hq), 99.0, device="cuda")
        out = torch.full((self.T, self.hq * self.d), 99.0, dtype=self.dt, device="cuda")
        a = dict(max_nodes=self.max_nodes, max_context=self.max_context, mask=self.mask(), out=out, lse=lse)
        a.update(kw)
        if "workspace" not in a:
            a["workspace"] = self.workspace(nodes=a["max_nodes"], ctx=a["max_context"])
        got = glsa.tree_attention(self.q, self.k, self.v, ints(self.table), ints(self.context), ints(self.q_start), **a)
        assert got is a["out"]
        return f64(out).reshape(self.T, self.hq, self.d), f64(lse)

    def check(self, got=None, scale=None, what="", **kw):
        out, lse = got or self.run(**({} if scale is None else dict(scale=scale)), **kw)
        sc = self.d ** -0.5 if scale is None else scale
        want, want_lse, spread, z = ao.attend(f64(self.q).reshape(self.T, self.hq, self.d), f64(self.k), f64(self.v),
                                              self.table, self.context, self.q_start, self.sees, sc)
        L = np.zeros(self.T)
        for b in range(self.B):
            L[self.q_start[b]:self.q_start[b + 1]] = self.context[b] + self.counts[b]
        h, w = half_step(self.dt), 0.0 if self.dt == torch.float32 else half_step(self.dt)
        z, L = z[..., None], L[:, None, None]
        ds = (self.d + 2) * U * z
        rel = 2 * (ds + (4 + 2 * z) * U) + 2 * L * U + w + 8 * U
        off = h * np.abs(want) + rel * spread * (1 + h) + torch.finfo(self.dt).tiny * torch.finfo(self.dt).eps
        nan = np.isnan(want)
        assert np.array_equal(np.isnan(out), nan), f"{what}: NaN in other places"
        over = (np.abs(out - want) > off) & ~nan
        assert not over.any(), f"{what}: {over.sum()} of {over.size} off, worst {np.max((np.abs(out - want) / off)[~nan]):.3g}"
        empty = np.isinf(want_lse)
        assert np.array_equal(lse[empty], want_lse[empty])
        ok = ~empty & ~np.isnan(want_lse)
        off = (ds + (4 + 2 * z) * U + 2 * L * U)[..., 0] + 4 * U * np.abs(want_lse, where=ok, out=np.zeros_like(lse)) + 8 * U
        assert np.all(np.abs(lse - want_lse)[ok] <= off[ok]), f"{what}: lse"
        return out


# ---- masks, positions, cache rows -------------------------------------------

@pytest.mark.parametrize("nodes", [1, 5, 64, 65, 200, 1024])
def test_build_tree(nodes):
    rng = np.random.default_rng(nodes)
    counts = [nodes, 0, max(1, nodes // 2), 1]
    s = Step([0, 7, 130, 31], counts, 1, 1, 8, torch.float32, page=6, seed=nodes)
    flat = np.concatenate([p for p in s.parents] + [[]]).astype(np.int32)
    if nodes > 4:  # a parent that is no earlier node counts as none
        flat[3], flat[4] = 3, nodes + 9
        s.sees[0] = ao.ancestors([int(p) if p < j else -1 for j, p in enumerate(flat[:nodes])])
    table = s.table.copy()
    table[2, -2:] = [-1, s.n_pages]
    words = -(-nodes // 64) + 1  # a wider row than needed
    mask = torch.full((s.T, words), -1, dtype=torch.int64, device="cuda")
    got, pos, rows = glsa.build_tree(ints(flat), ints(s.q_start), ints(s.context), max_nodes=nodes,
                                     page_table=ints(table), n_pages=s.n_pages, page_size=6, mask=mask)
    assert got is mask
    bits = np.unpackbits(mask.cpu().numpy().view(np.uint8).reshape(s.T, -1), axis=1, bitorder="little").astype(bool)
    for b in range(s.B):
        a, e = s.q_start[b], s.q_start[b + 1]
        n = e - a
        assert np.array_equal(bits[a:e, :n], s.sees[b]) and not bits[a:e, n:].any()
        assert np.array_equal(pos[a:e].cpu().numpy(), s.context[b] + s.sees[b].sum(1) - 1)
        assert np.array_equal(rows[a:e].cpu().numpy(),
                              ao.cache_rows_of(table[b], s.context[b] + np.arange(n), 6, s.n_pages))


def test_build_chain():
    counts = [130, 1, 0, 64]
    s = Step([5, 0, 3, 64], counts, 1, 1, 8, torch.float32, tree=False)
    mask, pos, rows = glsa.build_tree(None, ints(s.q_start), ints(s.context), max_nodes=130, n_tokens=s.T)
    assert mask is None and rows is None
    want = np.concatenate([c + np.arange(n) for c, n in zip(s.context, counts)])
    assert np.array_equal(pos.cpu().numpy(), want)
    mask = torch.full((s.T, 3), 77, dtype=torch.int64, device="cuda")
    glsa.build_tree(None, ints(s.q_start), ints(s.context), max_nodes=130, n_tokens=s.T, mask=mask)
    bits = np.unpackbits(mask.cpu().numpy().view(np.uint8).reshape(s.T, -1), axis=1, bitorder="little").astype(bool)
    for b, n in enumerate(counts):
        a = s.q_start[b]
        assert np.array_equal(bits[a:a + n, :n], np.tril(np.ones((n, n), bool))) and not bits[a:a + n, n:].any()


# ---- attention ----------------------------------------------------------------

HEADS = [(1, 1, 8), (4, 4, 64), (8, 2, 128), (32, 8, 128), (6, 2, 80), (16, 1, 64), (3, 1, 256), (2, 2, 200), (40, 1, 128)]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("heads", HEADS, ids=lambda h: "x".join(map(str, h)))
@pytest.mark.parametrize("tree", [True, False], ids=["tree", "chain"])
def test_ragged_batches(heads, dtype, tree):
    """Contexts and node counts of every kind side by side, unused rows NaN."""
    s = Step([0, 1, 15, 16, 33, 130, 517, 64], [3, 1, 7, 0, 20, 2, 5, 1], *heads, TYPES[dtype], page=16, tree=tree,
             seed=heads[0] + heads[2])
    s.poison_unused()
    s.check(what=f"{heads} {dtype}")


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("page", [1, 3, 8, 24, 64, 100, 1000])
def test_page_sizes(page, dtype):
    s = Step([99, 300, 63, 0], [4, 1, 9, 2], 8, 2, 128, TYPES[dtype], page=page, seed=page)
    s.poison_unused()
    s.check()


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("nodes,group", [(1, 1), (1, 8), (2, 8), (9, 4), (17, 2), (33, 1), (64, 4), (65, 2), (100, 3), (200, 1)])
def test_node_counts(nodes, group, dtype):
    s = Step([200, 31], [nodes, max(1, nodes - 1)], 2 * group, 2, 64, TYPES[dtype], seed=nodes)
    s.poison_unused()
    s.check()


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("contexts,counts,hq,hk", [([9000], [1], 4, 1), ([20011], [5], 8, 2), ([4097, 0, 2500], [3, 2, 40], 4, 2),
                                                   ([6000], [70], 4, 1)])
def test_long_contexts(contexts, counts, hq, hk, dtype):
    """Contexts that are split over workgroups and joined."""
    s = Step(contexts, counts, hq, hk, 128, TYPES[dtype], seed=counts[0])
    s.poison_unused()
    s.check()


@pytest.mark.parametrize("dtype", list(TYPES))
def test_long_chain(dtype):
    """A piece of a prompt: more tokens than a tree may have nodes."""
    s = Step([70, 0], [1100, 257], 2, 1, 64, TYPES[dtype], tree=False, seed=4)
    s.poison_unused()
    s.check()


@pytest.mark.parametrize("dtype", list(TYPES))
def test_large_scores(dtype):
    """Scores in the hundreds: the running maximum matters, most weights vanish."""
    s = Step([400, 1000], [6, 3], 8, 2, 128, TYPES[dtype], seed=5, q_scale=30.0)
    s.check()
    s.check(scale=-0.02)
    s.check(scale=0.0)


@pytest.mark.parametrize("dtype", list(TYPES))
def test_rows_that_see_nothing(dtype):
    s = Step([0, 0, 40], [4, 70, 5], 8, 2, 64, TYPES[dtype], seed=6)
    for b, i in ((0, 0), (0, 3), (1, 69), (1, 10), (2, 4)):
        s.sees[b][i] = False  # no node, not even itself
    s.poison_unused()
    out = s.check()
    assert np.all(out[0] == 0) and np.all(out[3] == 0) and np.all(out[4 + 69] == 0)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("ctx,n", [(50, 9), (0, 40), (1500, 70)])
def test_masked_values_do_not_matter(value, dtype, ctx, n):
    """A node whose k and v hold no numbers is felt by the nodes that see it alone."""
    s = Step([ctx], [n], 8, 2, 128, TYPES[dtype], seed=7)
    bad = n // 2
    s.sees[0] = np.tril(np.ones((n, n), bool))
    s.sees[0][::2, bad] = False
    row = int(ao.cache_rows_of(s.table[0], [ctx + bad], s.page, s.n_pages)[0])
    s.k[row // s.page, :, row % s.page], s.v[row // s.page, :, row % s.page] = float("nan"), value
    s.poison_unused(value)
    out = s.check()
    assert np.isnan(out[bad + 1 - bad % 2]).all() and not np.isnan(out[::2]).any()


@pytest.mark.parametrize("dtype", list(TYPES))
def test_infinite_values_that_are_seen(dtype):
    """v may be infinite in single places where k is ordinary: they reach the
    rows that see them, with their sign, and no other column."""
    s = Step([0], [12], 4, 2, 64, TYPES[dtype], seed=8)
    row = int(ao.cache_rows_of(s.table[0], [5], s.page, s.n_pages)[0])
    s.v[row // s.page, :, row % s.page, 3], s.v[row // s.page, :, row % s.page, 9] = float("inf"), -float("inf")
    out, lse = s.run()
    sees = s.sees[0][:, 5]
    assert np.all(out[sees][..., 3] == np.inf) and np.all(out[sees][..., 9] == -np.inf)
    s.v.masked_fill_(torch.isinf(s.v), 0.0)
    clean, _ = s.run()
    other = np.ones(64, bool)
    other[[3, 9]] = False
    assert np.array_equal(out[..., other], clean[..., other]) and np.array_equal(out[~sees], clean[~sees])


@pytest.mark.parametrize("dtype", list(TYPES))
def test_missing_pages_are_masked(dtype):
    s = Step([200, 90, 30], [5, 3, 2], 8, 2, 64, TYPES[dtype], seed=9, page=16)
    s.table[0, 3], s.table[0, 12], s.table[1, 0] = -1, s.n_pages, 2 ** 31 - 1
    s.table[2, :] = -(2 ** 31)  # nothing at all
    s.poison_unused()
    out = s.check()
    assert np.all(out[8:] == 0)


def test_table_shorter_than_the_context():
    """Positions past the table's columns are masked too."""
    s = Step([100], [3], 4, 1, 64, torch.float16, seed=10)
    s.table = np.ascontiguousarray(s.table[:, :4])
    s.check(max_context=100)


@pytest.mark.parametrize("dtype", list(TYPES))
def test_strides(dtype):
    """Padded q rows, out with its own stride, caches of either order, a wide page table."""
    s = Step([77, 300], [6, 2], 8, 2, 128, TYPES[dtype], pad=24, rows_first=True, seed=11)
    s.poison_unused()
    s.check()
    big = torch.zeros(s.T, 8 * 128 + 8, dtype=s.dt, device="cuda")
    lse = torch.zeros(s.T, 8, device="cuda")
    wide = torch.full((s.B, s.table.shape[1] + 5), -7, dtype=torch.int32, device="cuda")
    wide[:, :s.table.shape[1]] = ints(s.table)
    glsa.tree_attention(s.q, s.k, s.v, wide[:, :s.table.shape[1]], ints(s.context), ints(s.q_start), max_nodes=6,
                        max_context=300, mask=s.mask(), out=big[:, :1024], lse=lse, workspace=s.workspace())
    s.check((f64(big[:, :1024]).reshape(s.T, 8, 128), f64(lse)))
    assert torch.all(big[:, 1024:] == 0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_out_in_place_of_q_and_loose_bounds(dtype):
    s = Step([700, 5], [9, 4], 8, 2, 64, TYPES[dtype], seed=12)
    want = s.run()
    loose = s.run(max_nodes=64, max_context=5000)
    s.check(loose)
    default = s.run(max_context=None, workspace=s.workspace(ctx=s.table.shape[1] * s.page))
    s.check(default)
    kept = s.q.clone()
    lse = torch.zeros(s.T, 8, device="cuda")
    glsa.tree_attention(s.q, s.k, s.v, ints(s.table), ints(s.context), ints(s.q_start), max_nodes=9, max_context=700,
                        mask=s.mask(), out=s.q, lse=lse, workspace=s.workspace())
    assert np.array_equal(f64(s.q).reshape(want[0].shape), want[0]) and not torch.equal(s.q, kept)


def test_unsound_device_values_are_cut():
    """Counts past max_nodes or the rows, negative ones and contexts past
    max_context are cut; rows of no sequence are left alone."""
    s = Step([40, 40, 40], [5, 5, 5], 2, 1, 64, torch.float32, seed=13, tree=False)
    out = torch.full((15, 128), 99.0, device="cuda")
    glsa.tree_attention(s.q, s.k, s.v, ints(s.table), ints([-3, 1000, 40]), ints([0, 9, 9, 40]), max_nodes=5,
                        max_context=40, out=out, workspace=s.workspace())
    assert torch.all(out[5:9] == 99) and torch.all(out[14:] == 99)
    s.q_start, s.context = np.array([0, 5]), [0]
    s.B, s.T, s.counts, s.q, s.sees, s.table = 1, 5, [5], s.q[:5], s.sees[:1], s.table[:1]
    want, _, _, _ = ao.attend(f64(s.q).reshape(5, 2, 64), f64(s.k), f64(s.v), s.table, [0], [0, 5], s.sees, 0.125)
    assert np.allclose(f64(out[:5]).reshape(5, 2, 64), want, atol=1e-5)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_far_pages(dtype):
    """Element offsets past 32 bits."""
    dt, d, page = TYPES[dtype], 128, 16
    n_pages = (1 << 32) // (page * d) + 64  # over 2^32 elements
    s = Step([50], [3], 2, 1, d, dt, page=page, seed=14)
    small_k, small_v, table = s.k, s.v, s.table.copy()
    k = torch.empty(n_pages, 1, page, d, dtype=dt, device="cuda")
    v = torch.empty(n_pages, 1, page, d, dtype=dt, device="cuda")
    far = n_pages - 1 - np.arange(table.shape[1]) * 3
    for c, big in ((small_k, k), (small_v, v)):
        big[torch.from_numpy(far).cuda()] = c[torch.from_numpy(table[0]).long().cuda()]
    want = s.run()
    s.k, s.v, s.table = k, v, far[None].astype(np.int32)
    got = s.run()
    assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])
    # and the rotation's rows and the kept path go there too
    rows = torch.randn(2, 3 * d, device="cuda").to(dt)
    place = ints([n_pages * page - 5, n_pages * page - 17])
    if n_pages * page < 2 ** 31:
        glsa.rotary(rows[:, :d], rows[:, d:2 * d], ints([0, 0]), glsa.rope_table(1, d), head_dim=d, v=rows[:, 2 * d:],
                    k_cache=k, v_cache=v, cache_rows=place)
        assert torch.equal(v[n_pages - 1, 0, page - 5], rows[0, 2 * d:])
        assert torch.equal(k[n_pages - 2, 0, page - 1], rows[1, d:2 * d])
        glsa.keep_path(k, v, ints([[n_pages - 2]]), ints([2]), ints([[13]]), ints([1]))
        assert torch.equal(k[n_pages - 2, 0, 2], rows[1, d:2 * d])


def test_same_bits_every_time():
    """Splits are joined in order: the result does not depend on the schedule."""
    s = Step([9000, 300], [6, 2], 8, 2, 128, torch.bfloat16, seed=15)
    a, b = s.run(), s.run()
    assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])


def test_refusals_of_the_binding():
    s = Step([40], [4], 4, 2, 64, torch.bfloat16, seed=16)
    ok = dict(max_nodes=4, max_context=40, mask=s.mask(), workspace=s.workspace())
    args = [s.q, s.k, s.v, ints(s.table), ints(s.context), ints(s.q_start)]
    glsa.tree_attention(*args, **ok)

    def bad(at=None, value=None, status=glsa.LORA_ERR_INVALID_ARG, **kw):
        a = list(args)
        if at is not None:
            a[at] = value
        with pytest.raises(glsa.LoraError) as e:
            glsa.tree_attention(*a, **dict(ok, **kw))
        assert e.value.status == status
    bad(0, s.q.float())
    bad(0, s.q[:, :100])
    bad(1, s.k[0])
    bad(2, s.v.half())
    bad(2, s.v[:, :1])
    bad(3, ints(s.table).long())
    bad(3, ints(s.table)[:, ::2])
    bad(4, ints([40, 1]))
    bad(5, ints([0, 2, 4]))
    bad(mask=s.mask()[:2])
    bad(mask=s.mask().int())
    bad(out=torch.empty(4, 128, dtype=torch.bfloat16, device="cuda"))
    bad(lse=torch.empty(3, device="cuda"))
    bad(max_nodes=0)
    bad(max_nodes=100)  # the mask has too few words
    bad(workspace=torch.empty(8, device="cuda"))
    # a call that needs a workspace does not run without one
    if glsa.attention_workspace_bytes(1, 4, 4, 100000, 4, 2, 64):
        bad(max_context=100000, workspace=None)
        bad(max_context=100000, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))


# ---- the accepted path --------------------------------------------------------

@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("hk,d,page,layers", [(2, 64, 16, 1), (8, 128, 16, 3), (1, 256, 5, 2), (3, 80, 1, 2), (2, 8, 7, 130)])
def test_keep_path(hk, d, page, layers, dtype):
    rng = np.random.default_rng(d)
    n = 150
    contexts = [0, 37, 15, 200, 8, 64, 3]
    s = Step(contexts, [n] * 7, hk, hk, d, TYPES[dtype], page=page, seed=d)
    path = np.stack([np.sort(rng.permutation(n)[:70]) for _ in range(7)]).astype(np.int32)
    path[1] = np.arange(70)                 # nothing to move
    path[2] = n - 70 + np.arange(70)        # everything, each row onto the next one's source
    path[3, 5] = path[3, 4]                 # ends before an entry that does not ascend
    path[4, 0] = -1                         # or is negative: nothing
    path[6] = 1 + np.arange(70)             # one row up
    kept = np.array([70, 70, 70, 70, 70, 0, 99], np.int32)
    s.table[0, 0] = -1                      # destinations without a page
    s.table[0, -2] = s.n_pages
    caches = [(torch.randn_like(s.k), torch.randn_like(s.v).transpose(1, 2).contiguous().transpose(1, 2)) for _ in range(layers)]
    want = [[ao.keep(f64(c), s.table, contexts, path, kept) for c in pair] for pair in caches[:3]]
    wide = ints(np.concatenate([path, np.zeros_like(path[:, :3])], 1))
    glsa.keep_path([k for k, _ in caches], [v for _, v in caches], ints(s.table), ints(contexts), wide[:, :70], ints(kept))
    for pair, ref in zip(caches, want):
        for c, r in zip(pair, ref):
            assert np.array_equal(f64(c), r)


def test_keep_path_refusals():
    s = Step([4], [4], 1, 1, 64, torch.float16)
    ok = [s.k, s.v, ints(s.table), ints([4]), ints([[1, 2]]), ints([2])]
    for at, value in ((0, [s.k, s.k]), (1, s.v.float()), (2, ints(s.table).long()), (3, ints([4, 4])), (4, ints([1, 2])),
                      (5, ints([2]).long()), (0, []), (0, s.k.cpu())):
        a = list(ok)
        a[at] = value
        with pytest.raises(glsa.LoraError):
            glsa.keep_path(*a)
    glsa.keep_path(*ok)


# ---- streams and graphs ---------------------------------------------------------

def test_on_another_stream_and_in_a_graph():
    """A whole step (tree, rotation into the cache, attention, kept path) on a
    side stream, then captured and replayed with other inputs in place."""
    hq, hk, d, page, n = 8, 2, 128, 16, 12
    s = Step([300, 44], [n, n], hq, hk, d, torch.bfloat16, page=page, seed=20, spare=0)
    parents = ints(np.concatenate(s.parents))
    table, start = ints(s.table), ints(s.q_start)
    rows0 = torch.randn(s.T, (hq + 2 * hk) * d, device="cuda").bfloat16()
    k0, v0 = s.k.clone(), s.v.clone()
    context = ints(s.context)
    rows, out = rows0.clone(), torch.empty(s.T, hq * d, dtype=torch.bfloat16, device="cuda")
    rope = glsa.rope_table(1024, d)
    path, kept = ints([[0, 3, 7], [1, 2, 9]]), ints([3, 2])
    mask = torch.empty(s.T, 1, dtype=torch.int64, device="cuda")
    pos, place = (torch.empty(s.T, dtype=torch.int32, device="cuda") for _ in range(2))
    ws = glsa.alloc_attention_workspace(2, s.T, n, 1000, hq, hk, d, "cuda")
    q, k, v = rows[:, :hq * d], rows[:, hq * d:(hq + hk) * d], rows[:, (hq + hk) * d:]

    def step(stream):
        glsa.build_tree(parents, start, context, max_nodes=n, page_table=table, n_pages=s.n_pages, page_size=page,
                        mask=mask, positions=pos, cache_rows=place, stream=stream)
        glsa.qk_norm_rotary(q, k, None, None, pos, rope, head_dim=d, v=v, k_cache=s.k, v_cache=s.v, cache_rows=place,
                            stream=stream)
        glsa.tree_attention(q, s.k, s.v, table, context, start, max_nodes=n, max_context=1000, mask=mask, out=out,
                            workspace=ws, stream=stream)
        glsa.keep_path(s.k, s.v, table, context, path, kept, stream=stream)

    def reset(ctx, factor):
        rows.copy_(rows0 * factor)
        s.k.copy_(k0)
        s.v.copy_(v0)
        context.copy_(ints(ctx))
        out.fill_(float("nan"))

    inputs = [([300, 44], 1.0), ([123, 0], 0.5), ([17, 250], 2.0), ([300, 44], 1.0)]
    eager = []
    for ctx, f in inputs:
        reset(ctx, f)
        step(None)
        eager.append([t.clone() for t in (out, s.k, s.v, rows, mask)])
    side = torch.cuda.Stream()
    for (ctx, f), want in zip(inputs, eager):
        reset(ctx, f)
        side.wait_stream(torch.cuda.current_stream())
        step(side)
        torch.cuda.current_stream().wait_stream(side)
        assert all(torch.equal(a, b) for a, b in zip((out, s.k, s.v, rows, mask), want))
    graph = torch.cuda.CUDAGraph()
    reset(*inputs[0])
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step(None)
    for (ctx, f), want in zip(inputs, eager):
        reset(ctx, f)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((out, s.k, s.v, rows, mask), want))
