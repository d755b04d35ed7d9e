"""GPU: the rotation's table, rotary and qk_norm_rotary against the fp64
reference.

Tolerances.  A rounding is off by at most half a step, h = finfo.eps / 2 of
the value.  One output is a c - b s: its fp32 roundings are at most 3 of
2^-24 (|a| + |b|) (|c|, |s| <= 1 up to the table's magnitude), then one
rounding h to the type, or the type's smallest step where it is subnormal.
The norm's factor r = 1 / sqrt(mean + eps): a sum of d squares in chains of
at most 32 additions, halved by the root, the division, the root itself and
the two products, within 24 roundings of 2^-24."""

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


def tiny(dt):
    f = torch.finfo(dt)
    return f.tiny * f.eps  # the smallest step


def f64(t):
    return t.detach().double().cpu().numpy()


def make(T, hq, hk, d, dt, seed, pad=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rows = torch.empty(T, (hq + 2 * hk) * d + pad, dtype=dt, device="cuda").normal_(0, 1, generator=g)
    return rows, rows[:, :hq * d], rows[:, hq * d:(hq + hk) * d], rows[:, (hq + hk) * d:(hq + 2 * hk) * d], g


@pytest.mark.parametrize("scaling", [None, dict(type="linear", factor=4.0), dict(type="ntk", factor=4.0),
                                     dict(type="llama3", factor=8.0, original_max_position=8192),
                                     dict(type="yarn", factor=16.0, original_max_position=4096)])
@pytest.mark.parametrize("rot,n,first", [(128, 300, 0), (20, 77, 1000000), (6, 1, 2 ** 31 - 1), (256, 1025, 131000)])
def test_table(scaling, rot, n, first):
    f, magnitude = glsa.rope_frequencies(rot, 500000.0, scaling)
    got = f64(glsa.rope_table(n, rot, base=500000.0, scaling=scaling, first=first))
    a = ao.rope_angles(first + np.arange(n), f)
    want = np.concatenate([np.cos(a), np.sin(a)], 1) * magnitude
    # the angle: both sides round the product and the frequency in 64 bits (4
    # roundings of 2^-53 of the angle between them)
    off = U * np.abs(want) + magnitude * np.concatenate([a, a], 1) * 4 * 2.0 ** -53 + 1e-15
    assert np.all(np.abs(got - want) <= off), np.max(np.abs(got - want) / off)


def test_table_of_own_frequencies_and_no_rows():
    f = [0.5, 0.25, 0.0]
    got = f64(glsa.rope_table(9, 6, frequencies=f, magnitude=2.0))
    a = ao.rope_angles(np.arange(9), f)
    assert np.allclose(got, 2.0 * np.concatenate([np.cos(a), np.sin(a)], 1), rtol=1e-6, atol=1e-7)
    assert glsa.rope_table(0, 6).shape == (0, 6)


def run(norm, q, k, pos, table, d, **kw):
    if norm:
        return glsa.qk_norm_rotary(q, k, kw.pop("qw"), kw.pop("kw"), pos, table, head_dim=d, eps=1e-5, **kw)
    kw.pop("qw"), kw.pop("kw")
    return glsa.rotary(q, k, pos, table, head_dim=d, **kw)


def check(got, x, w, norm, table, pos, layout, dt, what):
    """got against the reference on heads x [T, h, d] (fp64)."""
    if norm:
        x = ao.norm_heads(x, w, 1e-5)
    want, mag = ao.rotate_heads(x, table, pos, layout)
    scale = max(1.0, np.max(np.abs(table)))
    off = half_step(dt) * np.abs(want) + (24 if norm else 4) * U * mag * scale * (1 + half_step(dt)) + tiny(dt)
    there = ~np.isnan(want)
    bad = np.abs(got - want)[there] > off[there]
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} elements off, worst {np.max((np.abs(got - want) / off)[there]):.3g}"
    return there


SHAPES = [  # T, hq, hk, d, rot, page, padding of the rows
    (1, 1, 1, 8, 2, 16, 0), (3, 4, 1, 64, 64, 16, 0), (67, 32, 8, 128, 128, 16, 0), (5, 8, 8, 80, 80, 7, 8),
    (33, 16, 2, 80, 20, 24, 16), (2, 5, 5, 256, 64, 1, 0), (129, 6, 2, 96, 48, 64, 8), (700, 32, 8, 128, 32, 16, 0),
    (1500, 16, 8, 64, 64, 16, 0), (9, 3, 1, 24, 6, 5, 8), (13, 2, 2, 48, 16, 16, 0),
]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("norm", [False, True], ids=["rotary", "norm"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_rows_and_cache(shape, norm, layout, dtype):
    T, hq, hk, d, rot, page, pad = shape
    dt = TYPES[dtype]
    rows, q, k, v, g = make(T, hq, hk, d, dt, T + d, pad)
    x = f64(rows)[:, :(hq + 2 * hk) * d].reshape(T, hq + 2 * hk, d)
    before = rows.clone()
    table_t = glsa.rope_table(50, rot, scaling=dict(type="yarn", factor=4.0, original_max_position=32))
    table = f64(table_t)
    pos = torch.randint(0, 50, (T,), dtype=torch.int32, device="cuda", generator=g)
    if T > 2:
        pos[1], pos[2] = -1, 50  # padding
    n_pages = -(-T // page) + 1
    shapes = (n_pages, hk, page, d)
    kc, vc = (torch.full(shapes, 7.0, dtype=dt, device="cuda") for _ in range(2))
    place = torch.randperm(n_pages * page, generator=g, device="cuda")[:T].to(torch.int32)
    if T > 4:
        place[3], place[4] = -1, n_pages * page  # not cached
    w = [torch.empty(d, dtype=dt, device="cuda").normal_(1, 0.3, generator=g) for _ in range(2)]
    w64 = [f64(a) for a in w]
    q_out = torch.full((T, hq * d), 5.0, dtype=dt, device="cuda")
    more = dict(layout=layout, qw=w[0], kw=w[1])
    got_q, got_k = run(norm, q, k, pos, table_t, d, q_out=q_out, v=v, k_cache=kc, v_cache=vc, cache_rows=place, **more)
    assert got_q is q_out and got_k is None
    assert torch.equal(rows, before)  # inputs are left
    p = pos.cpu().numpy()
    there = check(f64(q_out).reshape(T, hq, d), x[:, :hq], w64[0], norm, table, p, layout, dt, "q")
    assert np.all(f64(q_out).reshape(T, hq, d)[~there] == 5.0)
    # the cache: k turned, v as it is, everything else untouched
    at = place.cpu().numpy()
    placed = (at >= 0) & (at < n_pages * page) & (p >= 0) & (p < 50)
    kf, vf = (f64(c).transpose(0, 2, 1, 3).reshape(-1, hk, d) for c in (kc, vc))
    check(kf[at[placed]], x[placed, hq:hq + hk], w64[1], norm, table, p[placed], layout, dt, "k in the cache")
    assert np.array_equal(vf[at[placed]], x[placed, hq + hk:])
    rest = np.ones(n_pages * page, bool)
    rest[at[placed]] = False
    assert np.all(kf[rest] == 7.0) and np.all(vf[rest] == 7.0)
    # in place, without a cache: the same bits
    run(norm, q, k, pos, table_t, d, **more)
    assert torch.equal(q[there.any((1, 2))], q_out[there.any((1, 2))])
    assert np.array_equal(f64(k).reshape(T, hk, d)[placed], kf[at[placed]])
    out_of_table = ~((p >= 0) & (p < 50))
    assert np.array_equal(f64(rows)[out_of_table], f64(before)[out_of_table])
    assert torch.equal(rows[:, (hq + hk) * d:], before[:, (hq + hk) * d:])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_cache_with_rows_first_and_k_out(dtype):
    """A cache [pages, rows, heads, d] is passed as its transpose; k_out beside it."""
    dt = TYPES[dtype]
    T, hq, hk, d, page = 21, 4, 2, 128, 8
    rows, q, k, v, g = make(T, hq, hk, d, dt, 5)
    table = glsa.rope_table(40, d)
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    place = torch.randperm(4 * page, generator=g, device="cuda")[:T].to(torch.int32)
    kc, vc = (torch.zeros(4, page, hk, d, dtype=dt, device="cuda") for _ in range(2))
    k_out, q_out = torch.empty_like(k).contiguous(), torch.empty_like(q).contiguous()
    glsa.rotary(q, k, pos, table, head_dim=d, q_out=q_out, k_out=k_out, v=v, k_cache=kc.transpose(1, 2),
                v_cache=vc.transpose(1, 2), cache_rows=place)
    at = place.long()
    assert torch.equal(kc.view(-1, hk * d)[at], k_out) and torch.equal(vc.view(-1, hk * d)[at], v)
    check(f64(k_out).reshape(T, hk, d), f64(k).reshape(T, hk, d), None, False, f64(table), pos.cpu().numpy(), "half", dt, "k_out")


def test_norm_of_zero_large_and_tiny_heads():
    """A head of zeros gives zeros; heads near the type's ends stay finite."""
    d = 64
    q = torch.zeros(3, 2 * d, device="cuda")
    q[1], q[2] = 1e15, 1e-15
    k = torch.zeros(3, d, device="cuda")
    table = glsa.rope_table(1, d)
    pos = torch.zeros(3, dtype=torch.int32, device="cuda")
    glsa.qk_norm_rotary(q, k, None, None, pos, table, head_dim=d, eps=1e-6)
    assert torch.all(q[0] == 0) and torch.all(k == 0)
    assert torch.allclose(q[1], torch.ones_like(q[1]), atol=1e-6)
    assert torch.allclose(q[2], torch.full_like(q[2], 1e-12), rtol=1e-5)


def test_nan_stays_in_its_head():
    T, hq, hk, d = 2, 4, 2, 128
    rows, q, k, v, g = make(T, hq, hk, d, torch.bfloat16, 6)
    q[0, 130] = float("nan")
    table = glsa.rope_table(4, d)
    pos = torch.zeros(T, dtype=torch.int32, device="cuda")
    glsa.qk_norm_rotary(q, k, None, None, pos, table, head_dim=d)
    nan = torch.isnan(q).view(T, hq, d)
    assert nan[0, 1].all() and not nan[0, [0, 2, 3]].any() and not nan[1].any() and not torch.isnan(k).any()


def test_many_tokens():
    """The largest launches, whose lane groups walk several heads."""
    T, hq, hk, d = 5001, 32, 8, 128
    rows, q, k, v, g = make(T, hq, hk, d, torch.bfloat16, 8)
    table = glsa.rope_table(8192, d)
    pos = torch.randint(0, 8192, (T,), dtype=torch.int32, device="cuda", generator=g)
    some = torch.randperm(T, generator=g, device="cuda")[:64]
    x = f64(rows[some]).reshape(64, hq + 2 * hk, d)
    glsa.rotary(q, k, pos, table, head_dim=d)
    p = pos[some].cpu().numpy()
    check(f64(q[some]).reshape(64, hq, d), x[:, :hq], None, False, f64(table), p, "half", torch.bfloat16, "q")
    check(f64(k[some]).reshape(64, hk, d), x[:, hq:hq + hk], None, False, f64(table), p, "half", torch.bfloat16, "k")
    assert np.array_equal(f64(v[some]).reshape(64, hk, d), x[:, hq + hk:])


def test_refusals_of_the_binding():
    T, hq, hk, d = 4, 2, 1, 64
    rows, q, k, v, g = make(T, hq, hk, d, torch.float16, 9)
    table = glsa.rope_table(4, d)
    pos = torch.zeros(T, dtype=torch.int32, device="cuda")
    kc = torch.zeros(2, hk, 4, d, dtype=torch.float16, device="cuda")
    cached = dict(v=v, k_cache=kc, v_cache=kc.clone(), cache_rows=pos)
    call = lambda *a, **kw: glsa.rotary(*a, **dict(dict(head_dim=d), **kw))
    before = rows.clone()
    for args, kw in [((q, k, pos.long(), table), {}), ((q, k, pos[:3], table), {}), ((q, k, pos, table.half()), {}),
                     ((q, k.float(), pos, table), {}), ((q, k[:3], pos, table), {}), ((q, k, pos, table), dict(head_dim=48)),
                     ((q, k, pos, table), dict(layout="both")), ((q, k, pos, table.cpu()), {}),
                     ((q, k, pos, table), dict(v=v)), ((q, k, pos, table), dict(cached, v=None)),
                     ((q, k, pos, table), dict(cached, cache_rows=pos[:2])),
                     ((q, k, pos, table), dict(cached, v_cache=kc.float())),
                     ((q, k, pos, table), dict(cached, k_cache=kc[:, :, :, :32])),
                     ((q, k, pos, table), dict(q_out=torch.empty(T, d, dtype=torch.float16, device="cuda")))]:
        with pytest.raises(glsa.LoraError):
            call(*args, **kw)
    with pytest.raises(glsa.LoraError):
        glsa.qk_norm_rotary(q, k, torch.ones(32, dtype=torch.float16, device="cuda"), None, pos, table, head_dim=d)
    torch.cuda.synchronize()
    assert torch.equal(rows, before)
