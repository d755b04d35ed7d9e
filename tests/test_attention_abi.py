"""CPU tests of include/lora_attention.h: the library exports what the header
declares, the rotation's frequencies follow their formulas, and bad arguments
are rejected on the host before anything reaches the GPU."""

import ctypes
import math
import os
import re

import pytest
import torch

import gemm_lora_shrink_amd as glsa
from gemm_lora_shrink_amd import attention as A

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BAD, NOT = glsa.LORA_ERR_INVALID_ARG, glsa.LORA_ERR_UNSUPPORTED
FAKE = 0x10000  # an aligned, never dereferenced address


def test_library_exports_every_declared_symbol():
    src = open(os.path.join(ROOT, "include", "lora_attention.h")).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    names = sorted(set(re.findall(r"\b(lora_[a-z_0-9]+)\s*\(", src)))
    assert {"lora_rotary", "lora_tree_attention", "lora_keep_path"} <= set(names)
    for n in names:
        assert hasattr(A._lib(), n), f"{n} is declared but not exported"
    assert int(re.search(r"#define LORA_MAX_TREE_NODES (\d+)", src).group(1)) == A.MAX_TREE_NODES
    assert int(re.search(r"#define LORA_MAX_KEEP_LAYERS (\d+)", src).group(1)) == A.MAX_KEEP_LAYERS


# ---- frequencies -------------------------------------------------------------

def test_plain_and_linear_and_ntk_frequencies():
    f, m = glsa.rope_frequencies(64, 10000.0)
    assert m == 1.0 and len(f) == 32
    for i in range(32):
        assert math.isclose(f[i], 10000.0 ** (-i / 32), rel_tol=1e-14)
    g, m = glsa.rope_frequencies(64, 10000.0, dict(type="linear", factor=4.0))
    assert m == 1.0 and all(math.isclose(a, b / 4, rel_tol=1e-15) for a, b in zip(g, f))
    g, _ = glsa.rope_frequencies(64, 10000.0, dict(type="ntk", factor=4.0))
    # the fastest pair is unchanged, the slowest is slowed by the whole factor
    assert g[0] == 1.0 and math.isclose(g[-1], f[-1] / 4, rel_tol=1e-12)


def test_llama3_frequencies_by_turns():
    L, s = 8192, 8.0
    f, _ = glsa.rope_frequencies(128, 500000.0)
    g, m = glsa.rope_frequencies(128, 500000.0, dict(type="llama3", factor=s, original_max_position=L))
    assert m == 1.0
    kinds = set()
    for a, b in zip(f, g):
        turns = L * a / (2 * math.pi)
        if turns >= 4:
            assert b == a
            kinds.add("fast")
        elif turns <= 1:
            assert math.isclose(b, a / s, rel_tol=1e-15)
            kinds.add("slow")
        else:
            assert a / s < b < a
            kinds.add("between")
    assert kinds == {"fast", "slow", "between"}


def test_yarn_frequencies_and_magnitude():
    f, _ = glsa.rope_frequencies(128, 10000.0)
    g, m = glsa.rope_frequencies(128, 10000.0, dict(type="yarn", factor=4.0, original_max_position=4096))
    assert math.isclose(m, 0.1 * math.log(4.0) + 1.0, rel_tol=1e-15)
    kept = [(b - a / 4) / (a - a / 4) for a, b in zip(f, g)]  # 1: unchanged, 0: slowed
    assert kept[0] == 1.0 and abs(kept[-1]) < 1e-12 and all(a >= b - 1e-12 for a, b in zip(kept, kept[1:]))
    assert glsa.rope_frequencies(128, 10000.0, dict(type="yarn", factor=4.0, original_max_position=4096,
                                                    magnitude=1.5))[1] == 1.5


@pytest.mark.parametrize("args,status", [
    ((0, 1e4, None), BAD), ((3, 1e4, None), BAD), ((258, 1e4, None), BAD), ((64, 0.0, None), BAD),
    ((64, math.inf, None), BAD), ((64, math.nan, None), BAD),
    ((64, 1e4, dict(type="linear", factor=0.0)), BAD), ((64, 1e4, dict(type="linear", factor=math.nan)), BAD),
    ((64, 1e4, dict(type="llama3", factor=8.0)), BAD),  # no original context
    ((64, 1e4, dict(type="llama3", factor=8.0, original_max_position=8192, low=4.0, high=4.0)), BAD),
    ((64, 1.0, dict(type="yarn", factor=8.0, original_max_position=8192)), BAD),
    ((2, 1e4, dict(type="ntk", factor=8.0)), NOT),
    ((64, 1e4, dict(type="yarn", factor=8.0, original_max_position=8192, magnitude=-1.0)), BAD),
    ((64, 1e4, dict(type="spiral")), BAD), ((64, 1e4, dict(factor=2.0)), BAD),
    ((64, 1e4, dict(type="linear", factr=2.0)), BAD),
])
def test_frequencies_refused(args, status):
    with pytest.raises(glsa.LoraError) as e:
        glsa.rope_frequencies(*args)
    assert e.value.status == status


# ---- the C ABI ---------------------------------------------------------------

def _cache(**kw):
    a = dict(k=FAKE, v=FAKE, k_page=1024, k_head=512, k_row=64, v_page=1024, v_head=512, v_row=64, n_pages=4, page_size=8)
    a.update(kw)
    return A._CACHE_FIELDS.pack(*(a[x] or 0 for x in ("k", "v", "k_page", "k_head", "k_row", "v_page", "v_head", "v_row",
                                                      "n_pages", "page_size")))


def _table(**kw):
    a = dict(freq=(ctypes.c_double * 32)(), rot=64, magnitude=1.0, first=0, n=8, table=FAKE)
    a.update(kw)
    return A._lib().lora_rope_table(a["freq"], a["rot"], a["magnitude"], a["first"], a["n"], a["table"], None)


@pytest.mark.parametrize("kw", [dict(freq=None), dict(rot=63), dict(rot=512), dict(first=-1), dict(n=-1),
                                dict(first=1 << 31, n=1), dict(n=(1 << 31) + 1), dict(table=None)])
def test_rope_table_refused(kw):
    assert _table(**kw) == BAD and glsa.lib().lora_last_error()


def test_rope_table_limits():
    assert _table(table=FAKE + 4) == NOT
    assert _table(n=0) == glsa.LORA_OK


def _rotary(norm=False, cache=None, **kw):
    a = dict(dt=1, q=FAKE, ldq=512, k=FAKE, ldk=128, v=None, ldv=128, T=4, hq=8, hk=2, d=64, layout=0, rot=64, qw=FAKE,
             kw=FAKE, eps=1e-6, table=FAKE, n=16, positions=FAKE, q_out=FAKE, ldqo=512, k_out=FAKE, ldko=128, rows=None)
    a.update(kw)
    head = [a[x] for x in ("dt", "q", "ldq", "k", "ldk", "v", "ldv", "T", "hq", "hk", "d", "layout", "rot")]
    tail = [a[x] for x in ("table", "n", "positions", "q_out", "ldqo", "k_out", "ldko")] + [
        cache, a["rows"], None]
    if norm:
        return A._lib().lora_qk_norm_rotary(*head, a["qw"], a["kw"], a["eps"], *tail)
    return A._lib().lora_rotary(*head, *tail)


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("kw,status", [
    (dict(dt=5), BAD), (dict(T=-1), BAD), (dict(d=0), BAD), (dict(d=60), NOT), (dict(d=264), NOT), (dict(hq=-1), BAD),
    (dict(hk=1025), NOT), (dict(hq=0, hk=0), BAD), (dict(layout=2), BAD), (dict(rot=0), BAD), (dict(rot=7), BAD),
    (dict(rot=66), BAD), (dict(n=0), BAD), (dict(table=None), BAD), (dict(positions=None), BAD),
    (dict(table=FAKE + 4), NOT), (dict(q=None), BAD), (dict(q=FAKE + 2), NOT), (dict(ldq=256), BAD), (dict(ldq=516), NOT),
    (dict(q_out=None), BAD), (dict(ldqo=1024), BAD), (dict(k=None), BAD), (dict(k_out=None), BAD), (dict(ldko=256), BAD),
    (dict(cache=_cache(), v=FAKE), BAD),                          # no cache_rows
    (dict(cache=_cache(), rows=FAKE), BAD),                       # no v
    (dict(cache=_cache(), rows=FAKE, v=FAKE, ldv=64), BAD),
    (dict(cache=_cache(k=None), rows=FAKE, v=FAKE), BAD),
    (dict(cache=_cache(v=FAKE + 8), rows=FAKE, v=FAKE), NOT),
    (dict(cache=_cache(page_size=0), rows=FAKE, v=FAKE), BAD),
    (dict(cache=_cache(n_pages=-1), rows=FAKE, v=FAKE), BAD),
    (dict(cache=_cache(n_pages=1 << 30), rows=FAKE, v=FAKE), NOT),
    (dict(cache=_cache(k_row=60), rows=FAKE, v=FAKE), NOT),
    (dict(cache=_cache(v_head=-8), rows=FAKE, v=FAKE), BAD),
    (dict(cache=_cache(), rows=FAKE, v=FAKE, hk=0), BAD),
    (dict(T=1 << 29), NOT),
])
def test_rotary_refused(norm, kw, status):
    assert _rotary(norm, **kw) == status
    assert glsa.lib().lora_last_error()


@pytest.mark.parametrize("kw,status", [(dict(eps=-1.0), BAD), (dict(eps=math.nan), BAD), (dict(eps=math.inf), BAD),
                                       (dict(qw=FAKE + 2), NOT), (dict(kw=FAKE + 8), NOT)])
def test_norm_refused(kw, status):
    assert _rotary(True, **kw) == status


def test_rotary_of_no_tokens_is_a_no_op():
    assert _rotary(T=0, q=None, k=None, table=None) == glsa.LORA_OK
    assert _rotary(True, T=0) == glsa.LORA_OK


def _build(**kw):
    a = dict(parents=FAKE, T=8, B=2, q_start=FAKE, context=FAKE, nodes=4, table=FAKE, ld=4, n_table=4, n_pages=9, page=16,
             mask=FAKE, words=1, positions=FAKE, rows=FAKE)
    a.update(kw)
    return A._lib().lora_build_tree(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), BAD), (dict(B=-1), BAD), (dict(B=70000), NOT), (dict(nodes=0), BAD), (dict(nodes=1025, words=17), NOT),
    (dict(words=0), BAD), (dict(nodes=65), BAD), (dict(mask=FAKE + 4), NOT), (dict(table=None), BAD), (dict(ld=3), BAD),
    (dict(n_table=-1), BAD), (dict(page=0), BAD), (dict(n_pages=-1), BAD), (dict(n_pages=1 << 30), NOT),
    (dict(q_start=None), BAD), (dict(context=None), BAD),
])
def test_build_tree_refused(kw, status):
    assert _build(**kw) == status and glsa.lib().lora_last_error()


def test_build_tree_no_ops():
    assert _build(T=0, q_start=None) == glsa.LORA_OK and _build(B=0, context=None) == glsa.LORA_OK
    assert _build(mask=None, positions=None, rows=None) == glsa.LORA_OK


def _attend(cache="", **kw):
    a = dict(dt=2, q=FAKE, ldq=512, T=8, B=2, hq=8, hk=2, d=64, table=FAKE, ld=4, n_table=4, context=FAKE, q_start=FAKE,
             nodes=4, ctx=60, mask=FAKE, words=1, scale=0.125, out=FAKE, ldo=512, lse=None, ws=FAKE, ws_bytes=1 << 40)
    a.update(kw)
    v = list(a.values())
    c = _cache() if cache == "" else cache
    return A._lib().lora_tree_attention(*v[:8], c, *v[8:], None)


@pytest.mark.parametrize("kw,status", [
    (dict(dt=3), BAD), (dict(T=-1), BAD), (dict(B=-1), BAD), (dict(B=1 << 20), NOT), (dict(hq=7), BAD), (dict(hk=0), BAD),
    (dict(hq=0), BAD), (dict(d=12), NOT), (dict(d=320), NOT), (dict(nodes=0), BAD), (dict(nodes=1025, words=17), NOT),
    (dict(ctx=-1), BAD), (dict(ctx=(1 << 31) - 1), NOT), (dict(words=0), BAD), (dict(mask=FAKE + 4), NOT),
    (dict(scale=math.nan), BAD), (dict(scale=math.inf), BAD), (dict(table=None), BAD), (dict(ld=2), BAD),
    (dict(context=None), BAD), (dict(q_start=None), BAD), (dict(cache=None), BAD), (dict(cache=_cache(v=None)), BAD),
    (dict(cache=_cache(k_page=1028)), NOT), (dict(cache=_cache(v_page=1 << 31)), NOT), (dict(q=None), BAD), (dict(q=FAKE + 8), NOT), (dict(ldq=504), BAD),
    (dict(out=None), BAD), (dict(ldo=516), NOT), (dict(ldo=1024), BAD),
    (dict(nodes=1 << 26, mask=None), NOT),
])
def test_tree_attention_refused(kw, status):
    assert _attend(**kw) == status
    assert glsa.lib().lora_last_error()


def test_tree_attention_of_nothing_is_a_no_op():
    assert _attend(T=0, q=None, out=None) == glsa.LORA_OK
    assert _attend(B=0, context=None, q_start=None) == glsa.LORA_OK


def test_workspace_sizes():
    # one sequence with a long context is split, whatever its bounds; bad sizes need nothing
    n = glsa.attention_workspace_bytes
    for sizes in [(1, 1, 1, 100, 32, 8, 128), (256, 256, 1, 4096, 32, 8, 128), (1, 64, 64, 32768, 32, 8, 128),
                  (3, 100, 64, 0, 4, 4, 256), (1, 1, 1, (1 << 31) - 2, 1, 1, 8)]:
        assert n(*sizes) >= 0 and n(*sizes) % 256 == 0
    assert n(-1, 1, 1, 1, 1, 1, 8) == 0 and n(1, 1, 1, 1, 3, 2, 8) == 0 and n(1, 1, 0, 1, 1, 1, 8) == 0


def _keep(cache="", k=(FAKE, FAKE), v=(FAKE, FAKE), **kw):
    a = dict(dt=1, layers=2, hk=2, d=64, B=2, table=FAKE, ld=4, n_table=4, context=FAKE, path=FAKE, ldp=4, n_path=4,
             kept=FAKE)
    a.update(kw)
    x = list(a.values())
    layers = [(ctypes.c_void_p * 2)(*p) if p else None for p in (k, v)]
    return A._lib().lora_keep_path(x[0], _cache() if cache == "" else cache, *layers, *x[1:], None)


@pytest.mark.parametrize("kw,status", [
    (dict(dt=9), BAD), (dict(layers=-1), BAD), (dict(layers=129), NOT), (dict(hk=0), BAD), (dict(d=4), NOT),
    (dict(B=-1), BAD), (dict(n_path=-1), BAD), (dict(n_path=1025, ldp=1025), NOT), (dict(ldp=3), BAD), (dict(ld=3), BAD),
    (dict(table=None), BAD), (dict(context=None), BAD), (dict(path=None), BAD), (dict(kept=None), BAD),
    (dict(cache=None), BAD), (dict(k=None), BAD), (dict(v=None), BAD), (dict(k=(FAKE, 0)), BAD), (dict(v=(FAKE + 8, FAKE)), NOT),
    (dict(cache=_cache(page_size=0)), BAD), (dict(cache=_cache(k_row=60)), NOT),
])
def test_keep_path_refused(kw, status):
    assert _keep(**kw) == status and glsa.lib().lora_last_error()


def test_keep_path_no_ops():
    assert _keep(layers=0) == _keep(B=0) == _keep(n_path=0) == glsa.LORA_OK


# ---- the binding, which must not let host tensors through ---------------------

def test_binding_refuses_host_tensors():
    q, k = torch.zeros(2, 128), torch.zeros(2, 64)
    pos, table = torch.zeros(2, dtype=torch.int32), torch.zeros(4, 64)
    cache = torch.zeros(4, 1, 8, 64)
    ints = torch.zeros(2, dtype=torch.int32)
    pages = torch.zeros(1, 4, dtype=torch.int32)
    calls = [
        lambda: glsa.rotary(q, k, pos, table, head_dim=64),
        lambda: glsa.qk_norm_rotary(q, k, None, None, pos, table, head_dim=64),
        lambda: glsa.rope_table(8, 64, device="cpu"),
        lambda: glsa.build_tree(None, ints, ints[:1], max_nodes=2, n_tokens=2),
        lambda: glsa.tree_attention(q, cache, cache, pages, ints[:1], ints, max_nodes=2),
        lambda: glsa.keep_path(cache, cache, pages, ints[:1], pages, ints[:1]),
    ]
    for call in calls:
        with pytest.raises(glsa.LoraError) as e:
            call()
        assert e.value.status == BAD
