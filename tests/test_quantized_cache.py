"""GPU: store_quantized, tree_attention_quantized and keep_path_quantized against
the fp64 reference.

The store and the kept path are exact: exponents and bytes are equal, as every
step of them is a product with a power of two and one rounding.

Tolerances of the attention.  h = finfo.eps / 2 is half a step of the type, u =
2^-24.  With A the softmax-weighted mean of |v| and z the row's largest scale *
sum |q| |k| (keys and values as the cache holds them, which enter exactly):
 - q enters as up to three numbers of 8 bits that add up to it, so a score is a
   sum of 3 d exact products in fp32: off by ds <= (3 d + 2) u z; every weight's
   exponential by 4 u, and by u times its argument (<= 2 z + ds in absolute
   value), which moves the weighted mean by at most 2 (ds + (4 + 2 z) u) A;
 - a weight enters the product with the values as one bf16 number, one fp16
   number (or two bf16 ones) or, for fp32, three bf16 ones, each off by half a
   step of what the ones before it left: w = 2^-8, 2^-11, 2^-24 of itself, w A;
 - the sums run over L keys and three numbers a weight: 4 L u A for the
   numerator and the denominator;
 - the output is rounded once: h |o|, or the type's smallest step; it is also
   put together from at most 64 parts, 8 u A;
 - fp32 and bf16 numbers below 2^-126 may count as 0: a weight, relative to the
   row's largest, leaves out up to 2^-126 |v|, a weight times its value's power of
   two up to 2^-126 of a byte's number (at most 448), for each of the L keys.  It
   shows only where outputs are themselves that small (value exponents near -126).
The same terms without A bound lse."""

import math

import numpy as np
import pytest
import torch

import gemm_lora_shrink_amd as glsa
from oracle import attention_oracle as ao
from oracle import cache_oracle as co

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
FORMATS = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}
WEIGHT = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
U = 2.0 ** -24
E4M3 = co.e4m3_numbers()


def f64(t):
    return t.detach().double().cpu().numpy()


def ints(v, dtype=torch.int32):
    return torch.tensor(np.asarray(v), dtype=dtype, device="cuda")


def numbers(t):
    """float64 numbers of a cache tensor's bytes."""
    raw = t.view(torch.uint8).cpu().numpy()
    return E4M3[raw] if t.dtype == torch.float8_e4m3fn else raw.view(np.int8).astype(np.float64)


def on_host(cache):
    fmt = "e4m3" if cache[0].dtype == torch.float8_e4m3fn else "int8"
    return dict(k=numbers(cache[0]), v=numbers(cache[1]), k_exp=cache[2].cpu().numpy().astype(int),
                v_exp=cache[3].cpu().numpy().astype(int), fmt=fmt)


def equal(cache, want, where=None):
    """The cache holds what the reference does (at the rows of `where` [pages, page])."""
    got = on_host(cache)
    for name in ("k", "v"):
        a, b = got[name], want[name]
        same = (a == b) | (np.isnan(a) & np.isnan(b))
        if where is not None:
            same |= ~where[:, None, :, None]
        assert same.all(), f"{name}: {(~same).sum()} bytes differ, first at {np.argwhere(~same)[0]}"
        assert np.array_equal(got[name + "_exp"], want[name + "_exp"]), f"{name}_exp differs"


def made(n_pages, hk, page, d, fmt, block, g, rows_first=False, spread=1):
    """A cache of random bytes (no NaN) and exponents that make values of about 1."""
    shape = (n_pages, page, hk, d) if rows_first else (n_pages, hk, page, d)
    out = []
    for _ in range(2):
        x = torch.randn(shape, generator=g, device="cuda") * (100 if fmt == "e4m3" else 32)
        x = x.clamp(-co.LARGEST[fmt], co.LARGEST[fmt])
        x = (x if fmt == "e4m3" else x.round()).to(FORMATS[fmt])
        out.append(x.transpose(1, 2) if rows_first else x)
    mid = -7 if fmt == "e4m3" else -5
    for _ in range(2):
        out.append(torch.randint(mid - spread, mid + spread + 1, (n_pages, hk, page // block), generator=g,
                                 device="cuda").to(torch.int8))
    return glsa.QuantizedCache(*out)


def rows_of(table, contexts, counts, page):
    return np.concatenate([[table[b][(c + j) // page] * page + (c + j) % page for j in range(n)]
                           for b, (c, n) in enumerate(zip(contexts, counts))] + [[]]).astype(int)


# ---- store ------------------------------------------------------------------

STORES = [  # contexts, counts, hk, d, page, block
    ([0], [1], 1, 16, 16, 16), ([5, 16, 31, 0], [1, 1, 1, 1], 8, 128, 16, 16), ([3, 60], [70, 5], 2, 64, 32, 8),
    ([7, 0, 9], [40, 0, 33], 3, 80, 24, 24), ([2], [200], 1, 256, 128, 128), ([1, 2], [9, 17], 2, 48, 8, 1),
    ([0, 100], [130, 3], 5, 112, 16, 2), ([12], [300], 2, 32, 96, 32), ([j for j in range(40)], [1] * 40, 2, 128, 16, 4),
]


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("case", range(len(STORES)))
def test_store(case, dt, fmt):
    contexts, counts, hk, d, page, block = STORES[case]
    g = torch.Generator("cuda").manual_seed(case)
    rng = np.random.default_rng(case)
    B, T = len(contexts), sum(counts)
    per = max(-(-(c + n) // page) for c, n in zip(contexts, counts)) + 1
    n_pages = B * per + 2
    table = rng.permutation(n_pages)[:B * per].reshape(B, per)
    cache = made(n_pages, hk, page, d, fmt, block, g, rows_first=case % 2 == 1, spread=3)
    # fused rows; sizes from token to token and of some channels, a token of zeros, infinities and NaN
    rows = torch.randn(T, 3 * hk * d + 8 * (case % 3), generator=g, device="cuda")
    rows *= torch.exp(2 * torch.randn(T, 1, generator=g, device="cuda"))
    rows[:, ::7] *= 16
    if T > 4:
        rows[1] = 0
        rows[2, hk * d::5] = math.inf
        rows[3, hk * d + 1::9] = math.nan
        rows[4, hk * d + 2::4] = -math.inf
    rows = rows.to(TYPES[dt])
    k, v = rows[:, hk * d:2 * hk * d], rows[:, 2 * hk * d:3 * hk * d]
    at = rows_of(table, contexts, counts, page)
    want = co.store(on_host(cache), f64(k).reshape(T, hk, d), f64(v).reshape(T, hk, d), at)
    glsa.store_quantized(k, v, cache, ints(at))
    equal(cache, want)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_store_range(fmt):
    """Zeros, the smallest and the largest numbers, and values at the exponents' borders."""
    g = torch.Generator("cuda").manual_seed(5)
    big = torch.finfo(torch.float32).max
    most = co.LARGEST[fmt]
    sizes = [0.0, 1e-45, 1e-38, 2.0 ** -126, most, math.nextafter(most, 1e9), most * 2.0 ** -140, most * 2.0 ** 119, big,
             most * 2.0 ** -126, 1.0, 2.0, 1.9999, math.inf, 2.0 ** 121, 2.0 ** 100 * most]
    T = len(sizes)
    cache = made(T, 1, 4, 32, fmt, 4, g)
    x = (torch.rand(T, 32, generator=g, device="cuda") * 2 - 1)
    x[:, 3] = 1.0
    x = x.double() * torch.tensor([min(s, big) for s in sizes], dtype=torch.float64, device="cuda")[:, None]
    x[13, 5] = math.inf
    x = x.float()
    at = np.arange(T) * 4
    want = co.store(on_host(cache), f64(x)[:, None], f64(-x)[:, None], at)
    glsa.store_quantized(x, -x, cache, ints(at))
    equal(cache, want)
    assert bool(torch.isfinite(torch.from_numpy(co.values(on_host(cache), "k")).float()).all())


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_store_token_by_token(fmt):
    """A block that grows by tokens of changing size holds what the reference does at each step."""
    g = torch.Generator("cuda").manual_seed(1)
    cache = made(3, 2, 16, 64, fmt, 16, g)
    want = on_host(cache)
    for t in range(20):
        x = (torch.randn(1, 2 * 64, generator=g, device="cuda") * 2.0 ** (t % 7)).bfloat16()
        y = (torch.randn(1, 2 * 64, generator=g, device="cuda") * 2.0 ** -(t % 5)).bfloat16()
        at = [[2, 0][t // 16] * 16 + t % 16]
        want = co.store(want, f64(x).reshape(1, 2, 64), f64(y).reshape(1, 2, 64), at)
        glsa.store_quantized(x, y, cache, ints(at))
        equal(cache, want)


def test_store_exponents_beyond_their_range():
    g = torch.Generator("cuda").manual_seed(2)
    for fmt in ("e4m3", "int8"):
        cache = made(4, 1, 8, 16, fmt, 8, g)
        for e in cache[2:]:
            e[0], e[1], e[2], e[3] = -128, 127, -127, 120
        x = torch.randn(4, 16, generator=g, device="cuda")
        at = [1, 9, 18, 27]
        want = co.store(on_host(cache), f64(x)[:, None], f64(x)[:, None], at)
        glsa.store_quantized(x, x, cache, ints(at))
        equal(cache, want)


def test_store_rows_that_are_not_placed():
    g = torch.Generator("cuda").manual_seed(3)
    cache = made(4, 2, 16, 32, "e4m3", 8, g)
    x = torch.randn(6, 64, generator=g, device="cuda").half()
    at = [-1, 5, 6, 64, 2 ** 31 - 1, 20]
    want = co.store(on_host(cache), f64(x).reshape(6, 2, 32), f64(x).reshape(6, 2, 32), at)
    glsa.store_quantized(x, x, cache, ints(at))
    equal(cache, want)
    before = on_host(cache)
    glsa.store_quantized(x[:0], x[:0], cache, ints(at)[:0])
    equal(cache, before)


# ---- attention ----------------------------------------------------------------

class Step:
    """A step's inputs: B sequences with the given contexts and node counts."""

    def __init__(self, contexts, counts, hq, hk, d, dt, fmt, *, page=16, block=None, seed=0, tree=True, pad=0, q_scale=1.0,
                 rows_first=False, spread=2):
        rng = np.random.default_rng(seed)
        g = torch.Generator("cuda").manual_seed(seed)
        self.rng, self.g, self.dt, self.page, self.d, self.hq, self.hk = rng, g, TYPES[dt], page, d, hq, hk
        self.context, self.counts, self.B = list(contexts), list(counts), len(contexts)
        self.q_start = np.concatenate([[0], np.cumsum(counts)]).astype(int)
        self.T = int(self.q_start[-1])
        per = max([-(-(c + n) // page) for c, n in zip(contexts, counts)] + [1]) + 1
        self.n_pages = self.B * per + 3
        self.table = rng.permutation(self.n_pages)[:self.B * per].reshape(self.B, per).astype(np.int32)
        self.cache = made(self.n_pages, hk, page, d, fmt, block or page, g, rows_first, spread)
        self.rows = (torch.randn(self.T, hq * d + pad, generator=g, device="cuda") * q_scale).to(self.dt)
        self.q = self.rows[:, :hq * d]
        self.parents = [[int(rng.integers(-1, j)) if j else -1 for j in range(n)] for n in counts] if tree else None
        self.sees = [ao.ancestors(self.parents[b]) if tree else np.tril(np.ones((n, n), bool))
                     for b, n in enumerate(counts)]
        self.max_nodes, self.max_context = max(list(counts) + [1]), max(list(contexts) + [0])

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
        used = np.zeros(self.n_pages * self.page, bool)
        for b in range(self.B):
            r = ao.cache_rows_of(self.table[b], np.arange(self.context[b] + self.counts[b]), self.page, self.n_pages)
            used[r[r >= 0]] = True
        return used.reshape(self.n_pages, self.page)

    def poison_unused(self):
        """What no sequence holds: NaN bytes (e4m3) or the largest (int8), exponents at their top."""
        used = torch.from_numpy(self.used_rows()).cuda()
        for c in self.cache[:2]:
            c.view(torch.uint8).masked_fill_(~used[:, None, :, None], 0x7f)
        block = self.page // self.cache[2].shape[2]
        of_block = used.view(self.n_pages, -1, block).any(-1)
        for e in self.cache[2:]:
            e.masked_fill_(~of_block[:, None], 127)

    def workspace(self, nodes=None, ctx=None):
        ws = glsa.alloc_quantized_workspace(self.B, self.T, nodes or self.max_nodes,
                                            self.max_context if ctx is None else ctx, self.hq, self.hk, self.d, "cuda")
        return ws.fill_(0xFF)

    def run(self, **kw):
        lse = torch.full((self.T, self.hq), 99.0, device="cuda")
        out = torch.full((self.T, self.hq * self.d), 99.0, dtype=self.dt, device="cuda")
        a = dict(max_nodes=self.max_nodes, max_context=self.max_context, mask=self.mask(), out=out, lse=lse)
        a.update(kw)
        if "workspace" not in a:
            a["workspace"] = self.workspace(a["max_nodes"], a["max_context"])
        got = glsa.tree_attention_quantized(self.q, self.cache, ints(self.table), ints(self.context), ints(self.q_start), **a)
        assert got is a["out"]
        return f64(got).reshape(self.T, self.hq, self.d), f64(a["lse"])

    def check(self, got=None, scale=None, what="", **kw):
        out, lse = got or self.run(**({} if scale is None else dict(scale=scale)), **kw)
        sc = self.d ** -0.5 if scale is None else scale
        host = on_host(self.cache)
        want, want_lse, spread, z = ao.attend(f64(self.q).reshape(self.T, self.hq, self.d), co.values(host, "k"),
                                              co.values(host, "v"), self.table, self.context, self.q_start, self.sees, sc)
        L = np.zeros(self.T)
        for b in range(self.B):
            L[self.q_start[b]:self.q_start[b + 1]] = self.context[b] + self.counts[b]
        h, w = torch.finfo(self.dt).eps / 2, WEIGHT[self.dt]
        z, L = z[..., None], L[:, None, None]
        ds = (3 * self.d + 2) * U * z
        rel = 2 * (ds + (4 + 2 * z) * U) + 4 * L * U + w + 8 * U
        off = h * np.abs(want) + rel * spread * (1 + h) + torch.finfo(self.dt).tiny * torch.finfo(self.dt).eps
        off = off + L * 2.0 ** -126 * (np.nanmax(np.abs(co.values(host, "v"))) + 448)
        nan = np.isnan(want)
        assert np.array_equal(np.isnan(out), nan), f"{what}: NaN in other places"
        over = (np.abs(out - want) > off) & ~nan
        assert not over.any(), f"{what}: {over.sum()} of {over.size} off, worst {np.max((np.abs(out - want) / off)[~nan]):.3g}"
        empty = np.isneginf(want_lse)
        assert np.array_equal(lse[empty], want_lse[empty])
        ok = ~empty & ~np.isnan(want_lse)
        off = (ds + (4 + 2 * z) * U + 4 * L * U)[..., 0] + 4 * U * np.abs(want_lse, where=ok, out=np.zeros_like(lse)) + 8 * U
        assert np.all(np.abs(lse[ok] - want_lse[ok]) <= off[ok]), f"{what}: lse"
        return out


CASES = [  # contexts, counts, hq, hk, d, options
    ([100], [1], 32, 8, 128, {}), ([0, 1, 63, 64, 65, 129], [1, 1, 1, 1, 1, 1], 8, 2, 64, dict(page=8, block=4)),
    ([300, 5, 40], [7, 3, 1], 8, 8, 80, dict(page=24, block=8)), ([1500, 31], [2, 2], 16, 2, 256, dict(page=32, block=1)),
    ([700, 0], [33, 64], 8, 2, 128, dict(page=64, block=32)), ([0, 0, 17], [50, 1, 0], 4, 4, 48, dict(block=2)),
    ([2100], [40], 32, 8, 128, dict(page=128, block=128, tree=False)), ([90, 600], [128, 65], 4, 1, 64, {}),
    ([515], [70], 6, 2, 240, dict(page=40, block=8)), ([10], [200], 4, 2, 112, dict(tree=False)),
    ([33, 4000], [1, 1], 32, 1, 128, dict(tree=False, rows_first=True)), ([64, 64], [9, 9], 12, 4, 16, dict(page=5, block=5)),
    ([777, 3], [12, 30], 16, 4, 256, dict(tree=False, page=16, block=16)),
]


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_attention(case, dt, fmt):
    contexts, counts, hq, hk, d, more = CASES[case]
    s = Step(contexts, counts, hq, hk, d, dt, fmt, seed=case, pad=8 * (case % 2), **more)
    s.poison_unused()
    s.check(what=f"{contexts} {counts}")


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
def test_many_units(dt, fmt):
    """More sequences than chunks are cut for by their lengths, and chains of several row tiles with units enough."""
    rng = np.random.default_rng(0)
    contexts = rng.integers(0, 300, 300)
    contexts[17] = 1500
    s = Step(contexts.tolist(), [1 + b % 2 for b in range(300)], 2, 1, 64, dt, fmt, tree=False, block=8)
    s.poison_unused()
    s.check(what="many sequences")
    s = Step([0, 100, 33, 5, 0, 64, 1, 9], [70, 64, 5, 66, 80, 1, 0, 90], 64, 16, 64, dt, fmt, tree=False)
    s.poison_unused()
    s.check(what="long chains")


@pytest.mark.parametrize("ctx", [None, 9000, 1000000])
@pytest.mark.parametrize("counts", [[1] * 6, [9, 40, 2, 17, 33, 0], [70, 64, 1, 90, 3, 80]])
def test_chunks_of_unlike_lengths(counts, ctx):
    """Sequences of many chunks next to ones of one and of none, under bounds that they reach or stay far below."""
    s = Step([5000, 3, 700, 64, 0, 2100], counts, 8, 2, 64, "bf16", "e4m3", block=4)
    s.poison_unused()
    s.check(**({} if ctx is None else dict(max_context=ctx)))


@pytest.mark.parametrize("B", [63, 64, 65])
def test_chunks_of_many_sequences(B):
    rng = np.random.default_rng(B)
    contexts, counts = rng.integers(0, 80, B), rng.integers(0, 3, B)
    contexts[B - 1], counts[B - 1], counts[0] = 3000, 2, 0
    s = Step(contexts.tolist(), counts.tolist(), 4, 1, 64, "f16", "int8", tree=False)
    s.poison_unused()
    s.check(max_context=5000)


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
def test_scores_far_apart(dt):
    """Large queries: one key takes all, sums stay exact enough; and negative or no scale."""
    s = Step([200, 900], [5, 40], 8, 2, 64, dt, "e4m3", q_scale=30.0)
    s.check(what="large")
    s.check(scale=-0.05, what="negative")
    s.check(scale=0.0, what="none")


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
def test_exponents_far_apart(dt, fmt):
    """Blocks whose scales differ by many powers of two, and exponents at and past their ends."""
    for counts in ([1, 3], [40, 33]):
        s = Step([150, 400], counts, 8, 2, 64, dt, fmt, block=4, spread=6)
        s.cache.v_exp[::3] -= 60
        s.cache.v_exp[1::5] = -128
        s.cache.k_exp[1::4] = -127
        s.check(what=f"{counts}")


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("counts", [[1, 3, 2], [40, 3, 64]])
def test_rows_that_see_nothing(dt, counts):
    s = Step([0, 0, 70], counts, 8, 2, 64, dt, "e4m3")
    for b in (0, 1):
        s.sees[b][counts[b] - 1] = False
        s.sees[b][0] = False
    s.table[2][:] = -1  # no page at all
    s.poison_unused()
    out = s.check()
    assert not out[s.q_start[1] - 1].any() and not out[s.q_start[2]:].any()


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("counts", [[1, 1], [6, 50]])
def test_missing_pages_are_masked(dt, counts):
    s = Step([200, 333], counts, 8, 2, 128, dt, "int8")
    s.table[0][3], s.table[1][0], s.table[1][7] = -1, s.n_pages, 2 ** 31 - 1
    s.poison_unused()
    s.check()


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("counts", [[4, 7], [20, 64]])
def test_nan_reaches_the_rows_that_see_it(dt, counts):
    """A NaN byte of a node's value or key: NaN for its descendants, nothing for the others."""
    s = Step([50, 190], counts, 8, 2, 64, dt, "e4m3")
    for b, node in ((0, 1), (1, counts[1] // 2)):
        pos = s.context[b] + node
        page, row = s.table[b][pos // 16], pos % 16
        s.cache.v.view(torch.uint8)[page, b, row, 5] = 0xff
        if b:
            s.cache.k.view(torch.uint8)[page, 0, row, 9] = 0x7f
    out = s.check()
    assert np.isnan(out).any() and not np.isnan(out).all()


def test_rows_of_no_sequence_are_left():
    s = Step([60, 20], [5, 9], 8, 2, 64, "bf16", "e4m3")
    q = torch.cat([s.rows, s.rows[:6]])
    out = torch.full_like(q, 7.0)
    mask = torch.cat([s.mask(), s.mask()[:6]])
    ws = glsa.alloc_quantized_workspace(2, q.size(0), 9, 60, 8, 2, 64, "cuda")
    glsa.tree_attention_quantized(q, s.cache, ints(s.table), ints(s.context), ints(s.q_start), max_nodes=9, max_context=60,
                                  mask=mask, out=out, workspace=ws)
    assert bool((out[14:] == 7).all())
    ref, _ = s.run()
    assert np.array_equal(f64(out[:14]).reshape(ref.shape), ref)


def test_bounds_of_a_step_are_cut_to_the_calls():
    """More nodes, contexts or rows than the call allows are not read."""
    s = Step([100, 50], [4, 6], 8, 2, 64, "f16", "e4m3", tree=False)
    out = torch.full_like(s.q, 7.0)
    ws = glsa.alloc_quantized_workspace(2, s.T, 4, 70, 8, 2, 64, "cuda")
    glsa.tree_attention_quantized(s.q, s.cache, ints(s.table), ints(s.context), ints(s.q_start), max_nodes=4, max_context=70,
                                  out=out, workspace=ws)
    assert bool((out[8:] == 7).all())
    s.context, s.counts = [70, 50], [4, 4]
    q_start = [0, 4, 8]
    host = on_host(s.cache)
    ref, *_ = ao.attend(f64(s.q[:8]).reshape(8, 8, 64), co.values(host, "k"), co.values(host, "v"), s.table, s.context,
                        q_start, [np.tril(np.ones((4, 4), bool))] * 2, 0.125)
    got = f64(out[:8]).reshape(8, 8, 64)
    assert np.max(np.abs(got - ref)) <= 2 * 2.0 ** -11 * np.max(np.abs(ref))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_out_may_be_q_and_workspace_larger(dt):
    s = Step([900, 40], [1, 20], 8, 2, 128, dt, "e4m3")
    ref, _ = s.run()
    ws = glsa.alloc_quantized_workspace(16, 64, 64, 4096, 8, 2, 128, "cuda").fill_(0xFF)
    got, _ = s.run(out=s.q, workspace=ws)
    assert np.array_equal(got, ref)


def test_page_offsets_past_32_bits():
    """A cache of more than 4 GiB: pages behind it are read and written where they are."""
    n_pages, hk, page, d = 70000, 8, 64, 128  # 4.6 GB of keys
    cache = glsa.alloc_quantized_cache(n_pages, hk, page, d, "cuda", block=32)
    g = torch.Generator("cuda").manual_seed(0)
    table = np.array([[69999, 3, 68001], [12, 69998, 0]], np.int32)
    contexts, counts = [100, 70], [60, 20]
    T = sum(counts)
    for b in range(2):
        n = contexts[b]
        x = torch.randn(n, 2 * hk * d, generator=g, device="cuda").bfloat16()
        glsa.store_quantized(x[:, :hk * d], x[:, hk * d:], cache, ints(rows_of(table[b:b + 1], [0], [n], page)))
    x = torch.randn(T, 2 * hk * d, generator=g, device="cuda").bfloat16()
    at = rows_of(table, contexts, counts, page)
    glsa.store_quantized(x[:, :hk * d], x[:, hk * d:], cache, ints(at))
    used = sorted(set(table.flatten().tolist()))
    small = glsa.QuantizedCache(*(t.view(torch.uint8)[used].view(t.dtype) for t in cache))
    where = np.searchsorted(used, table).astype(np.int32)
    q = torch.randn(T, 32 * d, generator=g, device="cuda").bfloat16()
    outs = []
    for c, t in ((cache, table), (small, where)):
        ws = glsa.alloc_quantized_workspace(2, T, 60, 100, 32, hk, d, "cuda")
        outs.append(glsa.tree_attention_quantized(q, c, ints(t), ints(contexts), ints([0, 60, 80]), max_nodes=60,
                                                  max_context=100, workspace=ws))
    assert torch.equal(*outs) and bool(torch.isfinite(outs[0]).all()) and float(outs[0].float().abs().max()) > 0.1
    path, kept = ints([[1, 30, 59], [0, 5, 19]]), ints([3, 2])
    glsa.keep_path_quantized([cache], ints(table), ints(contexts), path, kept)
    glsa.keep_path_quantized([small], ints(where), ints(contexts), path, kept)
    for a, b in zip(cache, small):
        assert torch.equal(a.view(torch.uint8)[used], b.view(torch.uint8))


def test_a_million_tokens():
    """One long sequence: a key near its end that the first head's query stands by is found, the other heads see all."""
    page, d, n, far = 128, 64, 1_000_000, 999_990
    per = -(-(n + 1) // page)
    g = torch.Generator("cuda").manual_seed(0)
    cache = made(per, 1, page, d, "e4m3", 32, g)
    table = torch.randperm(per, generator=g, device="cuda").to(torch.int32)[None]
    q = torch.randn(1, 4 * d, generator=g, device="cuda")
    cache.k.view(torch.uint8)[table[0, far // page], 0, far % page] = torch.where(q[0, :d] < 0, 0xfe, 0x7e).to(torch.uint8)
    ws = glsa.alloc_quantized_workspace(1, 1, 1, n, 4, 1, d, "cuda")
    out = glsa.tree_attention_quantized(q, cache, table, ints([n]), ints([0, 1]), max_nodes=1, max_context=n, workspace=ws)
    at = torch.arange(n + 1, device="cuda")
    pages = table[0].long()[at // page]
    k, v = (torch.ldexp(t.view(torch.uint8)[pages, 0, at % page].view(t.dtype).double(),
                        e[pages, 0, at % page // 32].double()[:, None]) for t, e in zip(cache[:2], cache[2:]))
    w = torch.softmax((q.double().view(4, d) @ k.t()) / 8, -1)
    assert float(w[0, far]) > 0.9 and float(w[1:].max()) < 0.1
    assert bool(((out.double().view(4, d) - w @ v).abs() <= 4 * (n + 1) * U * (w @ v.abs())).all())


# ---- the kept path ------------------------------------------------------------

KEEPS = [  # contexts, nodes, path, kept, hk, d, page, block
    ([20, 0, 33], 16, [[1, 4, 9, 15], [0, 1, 2, 3], [3, 5, 6, 7]], [4, 3, 1], 8, 128, 16, 16),
    ([5, 16, 47], 40, [[0, 2, 17, 39], [5, 20, 21, 39], [1, 2, 3, 4]], [4, 4, 0], 3, 48, 16, 4),
    ([7, 90], 30, [[2, 1, 5, 6], [4, 8, 8, 9]], [4, 4], 2, 256, 24, 8),   # paths that stop ascending
    ([3], 12, [[0, 1, 2, 3, 4, 5, 6, 7, 8, 9, 10, 11]], [12], 1, 80, 8, 1),
    ([2, 9, 11], 12, [[2, 3, 4, 5, 6, 7, 8, 9, 10, 11]] * 3, [10, 9, 10], 5, 64, 8, 8),
]


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("case", range(len(KEEPS)))
def test_keep(case, fmt):
    contexts, nodes, path, kept, hk, d, page, block = KEEPS[case]
    g = torch.Generator("cuda").manual_seed(case)
    rng = np.random.default_rng(case)
    B, path = len(contexts), np.array(path, np.int32)
    per = -(-(max(contexts) + nodes) // page)
    n_pages = B * per + 1
    table = rng.permutation(n_pages)[:B * per].reshape(B, per).astype(np.int32)
    caches = [made(n_pages, hk, page, d, fmt, block, g, rows_first=case % 2 == 0, spread=4) for _ in range(3)]
    want = [co.keep(on_host(c), table, contexts, path, kept) for c in caches]
    # behind the kept rows a cache holds nothing
    dead = np.zeros((n_pages, page), bool)
    for b in range(B):
        for pos in range(contexts[b] + kept[b], contexts[b] + nodes):
            dead[table[b][pos // page], pos % page] = True
    glsa.keep_path_quantized(caches, ints(table), ints(contexts), ints(path), ints(kept))
    for c, w in zip(caches, want):
        equal(c, w, ~dead)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("n_path,block", [(64, 16), (65, 4), (100, 16), (200, 1)])
def test_keep_long_paths(n_path, block, fmt):
    g, rng = torch.Generator("cuda").manual_seed(n_path), np.random.default_rng(n_path)
    contexts, nodes, page, B = [5, 64, 0], 260, 16, 3
    path = np.stack([np.sort(rng.choice(nodes, n_path, replace=False)) for _ in range(B)]).astype(np.int32)
    path[1, :30] = np.arange(30)      # the first nodes stay where they are
    path[1, 30:] = np.sort(rng.choice(np.arange(30, nodes), n_path - 30, replace=False))
    path[2, 50] = path[2, 49]         # ends there
    kept = [n_path, n_path - 1, n_path]
    per = -(-(max(contexts) + nodes) // page)
    table = rng.permutation(B * per + 1)[:B * per].reshape(B, per).astype(np.int32)
    table[0, 3] = -1
    cache = made(B * per + 1, 3, page, 48, fmt, block, g, False, spread=4)
    want = co.keep(on_host(cache), table, contexts, path, kept)
    live = np.zeros((B * per + 1, page), bool)
    for b in range(B):
        for pos in range(contexts[b] + (50 if b == 2 else kept[b])):
            if table[b][pos // page] >= 0:
                live[table[b][pos // page], pos % page] = True
    glsa.keep_path_quantized([cache], ints(table), ints(contexts), ints(path), ints(kept))
    equal(cache, want, live)


def test_keep_with_missing_pages_and_many_layers():
    g = torch.Generator("cuda").manual_seed(0)
    caches = [made(8, 2, 8, 32, "int8", 8, g, spread=4) for _ in range(70)]  # more than a launch takes
    table = np.array([[0, 1, -1, 3], [9, 5, 6, 7]], np.int32)
    contexts, path, kept = [6, 3], np.array([[1, 4, 11, 20], [0, 4, 9, 12]], np.int32), [4, 4]
    want = [co.keep(on_host(c), table, contexts, path, kept) for c in (caches[0], caches[69])]
    glsa.keep_path_quantized(caches, ints(table), ints(contexts), ints(path), ints(kept))
    live = np.zeros((8, 8), bool)
    for b in range(2):
        for pos in range(contexts[b] + 4):
            if 0 <= table[b][pos // 8] < 8:
                live[table[b][pos // 8], pos % 8] = True
    equal(caches[0], want[0], live)
    equal(caches[69], want[1], live)


# ---- together -----------------------------------------------------------------

@pytest.mark.parametrize("nodes", [1, 40])
def test_step_replays_from_a_graph(nodes):
    """Store, attention and kept path captured; every replay equals the eager calls."""
    s = Step([120, 700, 31], [nodes, 1, min(nodes, 9)], 8, 2, 64, "bf16", "e4m3", block=8)
    kv = torch.empty(s.T, 2 * 2 * 64, device="cuda", dtype=torch.bfloat16)
    table, context, q_start, mask = ints(s.table), ints(s.context), ints(s.q_start), s.mask()
    rows = ints(rows_of(s.table, s.context, s.counts, 16))
    path, kept = ints([[0]] * 3), ints([1, 0, 1])
    ws, out = s.workspace(), torch.zeros_like(s.q)

    def step():
        glsa.store_quantized(kv[:, :128], kv[:, 128:], s.cache, rows)
        glsa.tree_attention_quantized(s.q, s.cache, table, context, q_start, max_nodes=s.max_nodes,
                                      max_context=s.max_context, mask=mask, out=out, workspace=ws)
        glsa.keep_path_quantized([s.cache], table, context, path, kept)

    start = [t.clone() for t in s.cache]

    def again(seed):
        for t, x in zip(s.cache, start):
            t.view(torch.uint8).copy_(x.view(torch.uint8))
        kv.copy_(torch.randn(kv.shape, generator=torch.Generator("cuda").manual_seed(seed), device="cuda"))
        out.zero_()

    again(0)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (1, 2, 3):
        again(seed)
        step()
        want = [out.clone()] + [t.clone() for t in s.cache]
        again(seed)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip([out, *s.cache], want):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_calls_on_another_stream():
    s = Step([400, 90], [1, 12], 8, 2, 64, "f16", "int8")
    want, want_lse = s.run()
    lse, out = torch.zeros(s.T, 8, device="cuda"), torch.zeros_like(s.q)
    args = s.q, s.cache, ints(s.table), ints(s.context), ints(s.q_start)
    more = dict(max_nodes=12, max_context=400, mask=s.mask(), workspace=s.workspace())
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    glsa.tree_attention_quantized(*args, out=out, lse=lse, stream=side, **more)
    side.synchronize()
    assert np.array_equal(f64(out).reshape(want.shape), want) and np.array_equal(f64(lse), want_lse)


@pytest.mark.parametrize("nodes", [1, 40])
def test_replays_follow_the_lengths(nodes):
    """Two graphs, each with a workspace of its own, replayed with contexts and nodes that change between: every
    replay cuts the keys anew, as the eager call does."""
    s = Step([900, 3000, 31, 0], [nodes, nodes, min(nodes, 9), 1], 8, 2, 64, "f16", "int8", tree=False)
    table, context, q_start = ints(s.table), ints(s.context), ints(s.q_start)
    outs = [torch.zeros_like(s.q) for _ in range(3)]
    spaces = [s.workspace(nodes, 3000) for _ in range(3)]

    def call(i):
        glsa.tree_attention_quantized(s.q, s.cache, table, context, q_start, max_nodes=nodes, max_context=3000, out=outs[i],
                                      workspace=spaces[i])

    call(2)
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for i, graph in enumerate(graphs):
        with torch.cuda.graph(graph):
            call(i)
    for contexts, counts in (([900, 3000, 31, 0], [nodes, nodes, min(nodes, 9), 1]), ([3, 1, 0, 7], [1, 0, 1, 0]),
                             ([0, 0, 3000, 2999], [0, nodes, 1, nodes]), ([0] * 4, [0] * 4), ([64, 700, 1, 1], [1, 1, nodes, 0])):
        context.copy_(ints(contexts))
        q_start.copy_(ints(np.concatenate([[0], np.cumsum(counts)])))
        for o in outs:
            o.fill_(5)
        call(2)
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], outs[2]) and torch.equal(outs[1], outs[2])
        assert bool((outs[2][sum(counts):] == 5).all()) and not bool((outs[2][:sum(counts)] == 5).all(1).any())


def test_a_cache_listed_twice_is_refused():
    g = torch.Generator("cuda").manual_seed(0)
    a, b = (made(4, 2, 8, 32, "int8", 8, g) for _ in range(2))
    was = [t.clone() for t in (*a, *b)]
    args = ints([[0, 1], [2, 3]]), ints([7, 3]), ints([[2, 4], [1, 3]]), ints([2, 2])
    for caches in ([a, b, a], [a, (b[0], a[1], b[2], b[3])]):
        with pytest.raises(glsa.LoraError):
            glsa.keep_path_quantized(caches, *args)
    torch.cuda.synchronize()
    assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip((*a, *b), was))


def test_another_gpu_than_the_current_one_is_refused(monkeypatch):
    s = Step([9, 3], [1, 1], 4, 2, 64, "bf16", "e4m3", tree=False)
    table, context, q_start = ints(s.table), ints(s.context), ints(s.q_start)
    kv, rows, refs = torch.zeros(2, 128, device="cuda", dtype=torch.bfloat16), ints([0, 16]), ints([0] * s.n_pages)
    out, ws = torch.full_like(s.q, 3), s.workspace()
    was = [t.clone() for t in s.cache]
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: s.q.get_device() + 1)
    calls = (lambda: glsa.store_quantized(kv, kv, s.cache, rows),
             lambda: glsa.tree_attention_quantized(s.q, s.cache, table, context, q_start, max_nodes=1, max_context=9, out=out,
                                                   workspace=ws),
             lambda: glsa.keep_path_quantized([s.cache], table, context, rows.view(2, 1), rows),
             lambda: glsa.copy_pages(list(s.cache), rows, rows), lambda: glsa.reserve_pages(refs, table, context, page_size=16),
             lambda: glsa.fork_sequences(refs, table, rows, rows, rows, page_size=16),
             lambda: glsa.release_pages(refs, table), lambda: glsa.compact_pages(refs, table))
    for call in calls:
        with pytest.raises(glsa.LoraError, match="not the current one"):
            call()
    monkeypatch.undo()
    torch.cuda.synchronize()
    assert bool((out == 3).all()) and all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(s.cache, was))
