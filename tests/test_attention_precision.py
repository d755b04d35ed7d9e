"""GPU: tree_attention where one key stands far above thousands of others and
its value is zero (an attention sink), so that the small weights together make
the output.

Tolerances as in test_tree_attention.py: h = finfo.eps / 2, u = 2^-24, A the
softmax-weighted mean of |v|, z the largest scale * sum |q| |k|; scores,
exponentials, sums and parts in fp32 give 2 ((d + 2) u z + (4 + 2 z) u) A +
2 L u A + 8 u A, the weights of a product with 16-bit values h A and the
output's rounding h |o|, or the type's smallest step (an output of a few small
weights may be subnormal in fp16; with values of 256 none here is).  An fp16 weight below 2^-14 is off by up to half its
smallest step, 2^-25, instead of h times itself; the row's weights are measured
so that the largest is at least 2^12, so those are off by 2^-37 sum |v| of the
output at most."""

import math

import pytest
import torch

import gemm_lora_shrink_amd as glsa

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
U = 2.0 ** -24


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("size", [1.0, 256.0])
@pytest.mark.parametrize("heads,d", [(4, 64), (40, 128), (136, 64), (40, 256)])  # the rows of each kernel
@pytest.mark.parametrize("gap,spread", [(14.0, 0.0), (16.0, 0.0), (17.5, 0.0), (17.5, 1.0), (20.0, 0.0), (23.0, 1.0)])
@pytest.mark.parametrize("B,L,place", [(1, 256, 0), (1100, 4096, 0), (1100, 4096, 2501), (1, 32768, -1)])
def test_many_small_weights(B, L, place, gap, spread, heads, d, size, dtype):
    """B sequences on the same pages: so many that the keys of each are one chunk, or
    one sequence that is cut into chunks."""
    dt, page = TYPES[dtype], 64
    g = torch.Generator("cuda").manual_seed(int(gap * 2) + d)
    k = torch.zeros(L, d, device="cuda", dtype=dt)
    v = torch.empty(L, d, device="cuda", dtype=dt).normal_(0.5 * size, size, generator=g)
    k[:, 0].normal_(0.0, 1.0, generator=g).mul_(spread)
    k[place, 0], v[place] = gap, 0.0
    q = torch.zeros(heads, d, device="cuda", dtype=dt)
    q[:, 0] = 1 + torch.arange(heads, device="cuda") / 1024
    pages = torch.randperm(L // page, generator=g, device="cuda")
    caches = []
    for c in (k, v):
        cache = torch.empty(L // page, 1, page, d, device="cuda", dtype=dt)
        cache[pages, 0] = c.view(-1, page, d)
        caches.append(cache)
    table = pages.to(torch.int32).repeat(B, 1)
    lse = torch.empty(B, heads, device="cuda")
    out = glsa.tree_attention(q.view(1, -1).repeat(B, 1), *caches, table, torch.full_like(table[:, 0], L - 1),
                              torch.arange(B + 1, dtype=torch.int32, device="cuda"), max_nodes=1, max_context=L - 1,
                              scale=1.0, lse=lse,
                              workspace=glsa.alloc_attention_workspace(B, B, 1, L - 1, heads, 1, d, "cuda"))
    assert torch.equal(out, out[:1].expand_as(out)) and torch.equal(lse, lse[:1].expand_as(lse))
    q64, k64, v64 = (t.double().cpu() for t in (q, k, v))
    s = q64 @ k64.T
    w = torch.softmax(s, -1)
    want, A, z = w @ v64, w @ v64.abs(), (q64.abs() @ k64.abs().T).amax(-1, keepdim=True)
    h = torch.finfo(dt).eps / 2
    rel = 2 * ((d + 2) * U * z + (4 + 2 * z) * U) + 2 * L * U + 8 * U + (0.0 if dtype == "f32" else h)
    off = h * want.abs() + rel * A * (1 + h) + torch.finfo(dt).tiny * torch.finfo(dt).eps
    if dtype == "f16":
        off += 2.0 ** -37 * v64.abs().sum(0)
    worst = float(((out[0].view(heads, d).double().cpu() - want).abs() / off).max())
    assert worst <= 1.0, worst
    near = (lse[0].double().cpu() - torch.logsumexp(s, -1)).abs()
    assert float((near / (rel[:, 0] + 4 * U * (math.log(L) + z[:, 0]))).max()) <= 1.0


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("heads,d", [(4, 64), (40, 128), (136, 64), (40, 256)])
@pytest.mark.parametrize("power", [14, 15, 16, 17, 18, 19, 22, 30, 60])
def test_scores_whose_units_are_large(power, heads, d, dtype):
    """Scores so large that a step of fp32 passes the range of the weights: the key
    with the largest one is all that is left, whichever tile it is in."""
    dt, L, page = TYPES[dtype], 512, 64
    k = torch.zeros(L, d, device="cuda", dtype=dt)
    k[:, 0] = torch.randperm(L, generator=torch.Generator().manual_seed(power)).cuda() % 251  # exact in every type
    k[77, 0] = 252.0
    v = torch.randn(L, d, device="cuda", generator=torch.Generator("cuda").manual_seed(power)).to(dt)
    q = torch.zeros(1, heads * d, device="cuda", dtype=dt)
    q[0, ::d] = 16.0
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    lse = torch.empty(1, heads, device="cuda")
    cache = [c.view(L // page, 1, page, d) for c in (k, v)]
    out = glsa.tree_attention(q, *cache, ints([list(range(L // page))]), ints([L - 1]), ints([0, 1]), max_nodes=1,
                              max_context=L - 1, scale=2.0 ** power, lse=lse,
                              workspace=glsa.alloc_attention_workspace(1, 1, 1, L - 1, heads, 1, d, "cuda"))
    # one weight and its value, over that weight: the weight's and the output's rounding
    # to the type, and three in fp32 (exponential, reciprocal, product)
    h = torch.finfo(dt).eps / 2
    off = (8 * U if dtype == "f32" else 2 * h + 8 * U) * v[77].double().abs()
    assert bool(((out.view(heads, d).double() - v[77].double()).abs() <= off).all())
    assert torch.allclose(lse, torch.full_like(lse, 16.0 * 252.0 * 2.0 ** power), rtol=8 * U)
