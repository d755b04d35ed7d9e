"""CPU tests of include/lora_cache.h and its binding: the library exports what
the header declares, sizes of workspaces, and bad arguments are rejected on the
host before anything reaches the GPU."""

import os
import random
import re

import pytest
import torch

import gemm_lora_shrink_amd as glsa
from gemm_lora_shrink_amd import cache as C

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BAD, NOT, OK = glsa.LORA_ERR_INVALID_ARG, glsa.LORA_ERR_UNSUPPORTED, glsa.LORA_OK
FAKE = 0x10000  # an aligned, never dereferenced address
FIELDS = ("k", "v", "k_exp", "v_exp", "k_page", "k_head", "k_row", "v_page", "v_head", "v_row", "k_exp_page", "k_exp_head",
          "v_exp_page", "v_exp_head", "n_pages", "page_size", "block", "format")


def test_library_exports_every_declared_symbol():
    src = open(os.path.join(ROOT, "include", "lora_cache.h")).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    names = sorted(set(re.findall(r"\b(lora_[a-z_0-9]+)\s*\(", src)))
    assert {"lora_store_quantized", "lora_tree_attention_quantized", "lora_keep_path_quantized", "lora_reserve_pages",
            "lora_fork_sequences", "lora_release_pages", "lora_compact_pages", "lora_copy_pages"} <= set(names)
    for n in names:
        assert hasattr(C._lib(), n), f"{n} is declared but not exported"
    for n in ("alloc_quantized_cache", "store_quantized", "tree_attention_quantized", "keep_path_quantized", "reserve_pages",
              "fork_sequences", "release_pages", "compact_pages", "copy_pages", "PagedTensors"):
        assert callable(getattr(glsa, n))


def _cache(**kw):
    a = dict(k=FAKE, v=FAKE, k_exp=FAKE, v_exp=FAKE, k_page=1024, k_head=512, k_row=64, v_page=1024, v_head=512, v_row=64,
             k_exp_page=4, k_exp_head=2, v_exp_page=4, v_exp_head=2, n_pages=4, page_size=8, block=4, format=0)
    assert set(kw) <= set(FIELDS)
    a.update(kw)
    return C._CACHE_FIELDS.pack(*(a[f] or 0 for f in FIELDS))


BAD_CACHES = [(dict(format=2), BAD), (dict(format=-1), BAD), (dict(page_size=0), BAD), (dict(block=0), BAD),
              (dict(block=3), BAD), (dict(block=16), BAD), (dict(n_pages=-1), BAD), (dict(k_row=-16), BAD),
              (dict(v_head=8), NOT), (dict(k_page=1000), NOT), (dict(k_exp_head=-1), BAD)]
BAD_POINTERS = [(dict(k=None), BAD), (dict(v=None), BAD), (dict(k_exp=None), BAD), (dict(v_exp=None), BAD),
                (dict(k=FAKE + 8), NOT), (dict(v=FAKE + 4), NOT)]


def _store(cache=None, **kw):
    a = dict(dt=2, k=FAKE, ldk=128, v=FAKE, ldv=128, T=4, hk=2, d=64, rows=FAKE)
    a.update(kw)
    return C._lib().lora_store_quantized(a["dt"], a["k"], a["ldk"], a["v"], a["ldv"], a["T"], a["hk"], a["d"],
                                         _cache() if cache is None else cache, a["rows"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(dt=3), BAD), (dict(dt=-1), BAD), (dict(T=-1), BAD), (dict(hk=0), BAD), (dict(hk=1025), NOT), (dict(d=0), BAD),
    (dict(d=72), NOT), (dict(d=272), NOT), (dict(k=None), BAD), (dict(v=None), BAD), (dict(k=FAKE + 2), NOT),
    (dict(ldk=127), BAD), (dict(ldv=132), NOT), (dict(rows=None), BAD), (dict(T=2 ** 31 - 1), NOT), (dict(cache=b""), BAD)])
def test_store_refused(kw, status):
    if kw.get("cache") == b"":
        assert C._lib().lora_store_quantized(2, FAKE, 128, FAKE, 128, 4, 2, 64, None, FAKE, None) == BAD
        return
    assert _store(**kw) == status and glsa.lib().lora_last_error()


@pytest.mark.parametrize("kw,status", BAD_CACHES + BAD_POINTERS + [(dict(n_pages=1 << 30), NOT)])
def test_store_refuses_caches(kw, status):
    assert _store(_cache(**kw)) == status


def test_store_of_nothing():
    assert _store(T=0, k=None, v=None, rows=None) == OK


def _attend(cache=None, **kw):
    a = dict(dt=2, q=FAKE, ldq=256, T=4, B=2, hq=4, hk=2, d=64, table=FAKE, ld=8, n_table=8, context=FAKE, q_start=FAKE,
             nodes=2, ctx=32, mask=None, words=0, scale=0.125, out=FAKE, ldo=256, lse=None, ws=FAKE, ws_bytes=1 << 40)
    a.update(kw)
    return C._lib().lora_tree_attention_quantized(
        a["dt"], a["q"], a["ldq"], a["T"], a["B"], a["hq"], a["hk"], a["d"], _cache() if cache is None else cache, a["table"],
        a["ld"], a["n_table"], a["context"], a["q_start"], a["nodes"], a["ctx"], a["mask"], a["words"], a["scale"], a["out"],
        a["ldo"], a["lse"], a["ws"], a["ws_bytes"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(dt=7), BAD), (dict(T=-1), BAD), (dict(B=-1), BAD), (dict(B=65536), NOT), (dict(hq=3), BAD), (dict(hq=0), BAD),
    (dict(hk=0), BAD), (dict(hq=2048, hk=1024), NOT), (dict(d=0), BAD), (dict(d=40), NOT), (dict(d=264), NOT),
    (dict(nodes=0), BAD), (dict(ctx=-1), BAD), (dict(ctx=2 ** 31 - 2), NOT), (dict(nodes=1 << 26), NOT),
    (dict(scale=float("inf")), BAD), (dict(scale=float("nan")), BAD), (dict(mask=FAKE, nodes=65, words=1), BAD),
    (dict(mask=FAKE, nodes=1025, words=17), NOT), (dict(mask=FAKE + 4, words=1), NOT), (dict(n_table=-1), BAD),
    (dict(table=None), BAD), (dict(ld=7), BAD), (dict(context=None), BAD), (dict(q_start=None), BAD), (dict(q=None), BAD),
    (dict(out=None), BAD), (dict(ldq=255), BAD), (dict(ldo=260), NOT), (dict(q=FAKE + 8), NOT), (dict(out=FAKE, ldo=512), BAD)])
def test_attention_refused(kw, status):
    assert _attend(**kw) == status and glsa.lib().lora_last_error()


@pytest.mark.parametrize("kw,status", BAD_CACHES + BAD_POINTERS + [(dict(k_page=1 << 33), NOT), (dict(v_row=1 << 32), NOT),
                                                                   (dict(k_exp_page=1 << 33), NOT)])
def test_attention_refuses_caches(kw, status):
    assert _attend(_cache(**kw)) == status


def test_attention_of_nothing():
    assert _attend(T=0, q=None, out=None, context=None, q_start=None) == OK
    assert _attend(B=0, q=None, out=None) == OK


def test_attention_refuses_workspaces():
    sizes = dict(B=1, T=1, hq=32, hk=8, d=128, nodes=1, ctx=100000, ldq=4096, ldo=4096, n_table=12501, ld=12501)
    most = glsa.quantized_workspace_bytes(1, 1, 1, 100000, 32, 8, 128)
    assert most > 0
    cache = _cache(k_head=1024, k_row=128, v_head=1024, v_row=128, k_page=8192, v_page=8192)
    assert _attend(cache, **sizes, ws=None) == BAD
    assert _attend(cache, **sizes, ws=FAKE + 128) == BAD
    assert _attend(cache, **sizes, ws_bytes=256) == BAD


def test_workspace_bytes_grow_with_their_sizes():
    """One for the largest call suffices for every smaller one: what any smaller call asks for is no more."""
    for hq, hk, d in ((32, 8, 128), (8, 8, 64), (16, 1, 256)):
        most = glsa.quantized_workspace_bytes(24, 400, 48, 20000, hq, hk, d)
        for B, T, nodes, ctx in ((1, 1, 1, 20000), (24, 24, 1, 20000), (3, 144, 48, 700), (1, 48, 48, 20000), (7, 100, 17, 9000),
                                 (24, 400, 48, 20000)):
            assert glsa.quantized_workspace_bytes(B, T, nodes, ctx, hq, hk, d) <= most
    assert glsa.quantized_workspace_bytes(-1, 1, 1, 1, 8, 8, 64) == 0


def _keep(cache=None, **kw):
    ptrs = C.struct.Struct("@2P").pack(FAKE, FAKE)
    a = dict(k=ptrs, v=ptrs, ke=ptrs, ve=ptrs, layers=2, hk=2, d=64, B=1, table=FAKE, ld=4, n_table=4, context=FAKE, path=FAKE,
             ld_path=4, n_path=4, kept=FAKE)
    a.update(kw)
    return C._lib().lora_keep_path_quantized(_cache() if cache is None else cache, a["k"], a["v"], a["ke"], a["ve"],
                                             a["layers"], a["hk"], a["d"], a["B"], a["table"], a["ld"], a["n_table"],
                                             a["context"], a["path"], a["ld_path"], a["n_path"], a["kept"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(layers=-1), BAD), (dict(layers=129), NOT), (dict(hk=0), BAD), (dict(d=24), NOT), (dict(B=-1), BAD),
    (dict(B=65536), NOT), (dict(n_path=-1), BAD), (dict(n_path=1025, ld_path=1025), NOT), (dict(ld_path=3), BAD),
    (dict(ld=3), BAD), (dict(table=None), BAD), (dict(k=None), BAD), (dict(ve=None), BAD), (dict(context=None), BAD),
    (dict(path=None), BAD), (dict(kept=None), BAD), (dict(k=C.struct.Struct("@2P").pack(FAKE, 0)), BAD),
    (dict(v=C.struct.Struct("@2P").pack(FAKE, FAKE + 8)), NOT)])
def test_keep_refused(kw, status):
    assert _keep(**kw) == status and glsa.lib().lora_last_error()


@pytest.mark.parametrize("kw,status", BAD_CACHES)
def test_keep_refuses_caches(kw, status):
    assert _keep(_cache(**kw)) == status


def test_keep_of_nothing():
    for kw in (dict(B=0), dict(layers=0), dict(n_path=0)):
        assert _keep(**kw, k=None, v=None, path=None, kept=None) == OK


# ---- pages -------------------------------------------------------------------

POOL = dict(refs=FAKE, n=10, table=FAKE, ld=4, n_table=4, B=3)


def _pool(a):
    return a["refs"], a["n"], a["table"], a["ld"], a["n_table"], a["B"]


def _reserve(**kw):
    a = dict(POOL, lengths=FAKE, page=16, missing=None, ws=FAKE, ws_bytes=1 << 30)
    a.update(kw)
    return C._lib().lora_reserve_pages(*_pool(a), a["lengths"], a["page"], a["missing"], a["ws"], a["ws_bytes"], None)


def _fork(**kw):
    a = dict(POOL, from_=FAKE, ld_from=4, B_from=3, parents=FAKE, children=FAKE, lengths=FAKE, m=2, page=16, source=FAKE,
             target=FAKE, missing=None, tensors=None, n_tensors=0, ws=FAKE, ws_bytes=1 << 30)
    a.update(kw)
    return C._lib().lora_fork_sequences(a["refs"], a["n"], a["from_"], a["ld_from"], a["B_from"], a["table"], a["ld"], a["B"],
                                        a["n_table"], a["parents"], a["children"], a["lengths"], a["m"], a["page"],
                                        a["source"], a["target"], a["missing"], a["tensors"], a["n_tensors"], a["ws"],
                                        a["ws_bytes"], None)


def _release(**kw):
    a = dict(POOL, rows=FAKE, keep=None, m=2, page=16)
    a.update(kw)
    return C._lib().lora_release_pages(*_pool(a), a["rows"], a["keep"], a["m"], a["page"], None)


def _compact(**kw):
    a = dict(POOL, source=FAKE, target=FAKE, live=FAKE, moves=FAKE, tensors=None, n_tensors=0, ws=FAKE, ws_bytes=1 << 30)
    a.update(kw)
    return C._lib().lora_compact_pages(*_pool(a), a["source"], a["target"], a["live"], a["moves"], a["tensors"],
                                       a["n_tensors"], a["ws"], a["ws_bytes"], None)


@pytest.mark.parametrize("call", [_reserve, _fork, _release, _compact])
@pytest.mark.parametrize("kw,status", [(dict(refs=None), BAD), (dict(n=-1), BAD), (dict(n=(1 << 28) + 1), NOT),
                                       (dict(table=None), BAD), (dict(ld=3), BAD), (dict(n_table=-1), BAD), (dict(B=-1), BAD),
                                       (dict(B=65536), NOT)])
def test_pools_refused(call, kw, status):
    assert call(**kw) == status and glsa.lib().lora_last_error()


@pytest.mark.parametrize("call", [_reserve, _fork, _compact])
def test_pool_workspaces_refused(call):
    need = int(C._lib().lora_pages_workspace_bytes(10, 0))
    assert call(ws=None) == BAD and call(ws=FAKE + 2) == BAD and call(ws_bytes=need - 1) == BAD


@pytest.mark.parametrize("call,kw,status", [
    (_reserve, dict(lengths=None), BAD), (_reserve, dict(page=0), BAD), (_reserve, dict(n_table=1 << 30, ld=1 << 30), NOT),
    (_fork, dict(from_=None), BAD), (_fork, dict(ld_from=3), BAD), (_fork, dict(B_from=-1), BAD), (_fork, dict(m=-1), BAD),
    (_fork, dict(m=65536), NOT), (_fork, dict(parents=None), BAD), (_fork, dict(children=None), BAD),
    (_fork, dict(lengths=None), BAD), (_fork, dict(source=None), BAD), (_fork, dict(target=None), BAD), (_fork, dict(page=0), BAD),
    (_release, dict(page=0), BAD), (_release, dict(m=-1), BAD), (_release, dict(m=65536), NOT),
    (_release, dict(rows=None, m=2), BAD), (_compact, dict(live=None), BAD), (_compact, dict(moves=None), BAD),
    (_compact, dict(source=None), BAD), (_compact, dict(target=None), BAD), (_fork, dict(n_tensors=-1), BAD),
    (_fork, dict(n_tensors=1), BAD), (_compact, dict(n_tensors=1), BAD),
    (_compact, dict(n_tensors=1, tensors=C._TENSOR_FIELDS.pack(0, 16, 0, 0, 1, 1, 16)), BAD),
    (_fork, dict(n_tensors=1, tensors=C._TENSOR_FIELDS.pack(FAKE, 16, 0, 0, 1, 0, 16)), BAD)])
def test_pool_calls_refused(call, kw, status):
    assert call(**kw) == status


def test_pool_calls_of_nothing():
    assert _reserve(B=0, table=None, lengths=None, ws=None) == OK
    assert _fork(m=0, parents=None, children=None, lengths=None, source=None, target=None, ws=None) == OK
    assert _release(m=0) == OK and _release(n_table=0, table=None) == OK
    assert int(C._lib().lora_pages_workspace_bytes(-1, 3)) == 0 == int(C._lib().lora_pages_workspace_bytes((1 << 28) + 1, 0))


def _copy(tensors=None, **kw):
    t = dict(data=FAKE, page=1024, outer=0, inner=0, n_outer=1, n_inner=1, run=1024)
    a = dict(n_tensors=1, n_pages=8, source=FAKE, target=FAKE, n=3, count=None)
    a.update({k: v for k, v in kw.items() if k in a})
    t.update({k: v for k, v in kw.items() if k in t})
    packed = C._TENSOR_FIELDS.pack(*(t[k] or 0 for k in ("data", "page", "outer", "inner", "n_outer", "n_inner", "run")))
    return C._lib().lora_copy_pages(packed if tensors is None else tensors, a["n_tensors"], a["n_pages"], a["source"],
                                    a["target"], a["n"], a["count"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(n_tensors=-1), BAD), (dict(n=-1), BAD), (dict(n_pages=-1), BAD), (dict(n_pages=(1 << 28) + 1), BAD),
    (dict(data=None), BAD), (dict(n_outer=0), BAD), (dict(n_inner=0), BAD), (dict(run=0), BAD), (dict(page=-1), BAD),
    (dict(outer=-16), BAD), (dict(inner=-16), BAD), (dict(source=None), BAD), (dict(target=None), BAD),
    (dict(n_outer=2 ** 31 - 1, n_inner=2 ** 31 - 1, run=2 ** 31 - 1), NOT), (dict(n_outer=1 << 11, n_inner=1 << 10, run=1024), NOT)])
def test_copy_refused(kw, status):
    assert _copy(**kw) == status and glsa.lib().lora_last_error()


def test_copy_of_nothing():
    assert _copy(n=0, source=None) == OK and _copy(n_tensors=0) == OK and _copy(n_pages=0, data=None) == OK


# ---- the binding (host tensors are refused; shapes and types before that where it can tell) ----

def _host_cache(**kw):
    return glsa.alloc_quantized_cache(4, 2, 16, 32, "cpu", **kw)


def test_alloc_quantized_cache():
    c = _host_cache(block=8)
    assert c.k.shape == (4, 2, 16, 32) and c.k.dtype == torch.float8_e4m3fn and c.v_exp.shape == (4, 2, 2)
    assert _host_cache(dtype=torch.int8).k_exp.shape == (4, 2, 1)
    for kw in (dict(block=5), dict(block=0), dict(block=32), dict(dtype=torch.uint8), dict(dtype=torch.float16)):
        with pytest.raises(glsa.LoraError):
            _host_cache(**kw)
    for d in (0, 24, 272):
        with pytest.raises(glsa.LoraError):
            glsa.alloc_quantized_cache(4, 2, 16, d, "cpu")


def test_host_tensors_are_refused():
    c, i = _host_cache(), torch.zeros(4, dtype=torch.int32)
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    table = torch.zeros(4, 2, dtype=torch.int32)
    for call in (lambda: glsa.store_quantized(x, x, c, i), lambda: glsa.keep_path_quantized([c], table, i, table, i),
                 lambda: glsa.tree_attention_quantized(x, c, table, i, i, max_nodes=1),
                 lambda: glsa.reserve_pages(i, table, i, page_size=16),
                 lambda: glsa.fork_sequences(i, table, i, i, i, page_size=16), lambda: glsa.release_pages(i, table),
                 lambda: glsa.compact_pages(i, table), lambda: glsa.copy_pages([x], i, i), lambda: glsa.PagedTensors([])):
        with pytest.raises(glsa.LoraError):
            call()


def test_cache_views():
    """_cache's own checks, on host tensors (device index -1)."""
    c = _host_cache(block=4)
    packed, shape = C._cache(c, -1)
    got = dict(zip(FIELDS, C._CACHE_FIELDS.unpack(packed)))
    assert tuple(shape) == (4, 2, 16, 32) and (got["n_pages"], got["page_size"], got["block"], got["format"]) == (4, 16, 4, 0)
    assert (got["k_page"], got["k_head"], got["k_row"], got["k_exp_page"], got["v_exp_head"]) == (1024, 512, 32, 8, 4)
    turned = [t.transpose(1, 2).contiguous().transpose(1, 2) for t in c[:2]]
    got = dict(zip(FIELDS, C._CACHE_FIELDS.unpack(C._cache([*turned, *c[2:]], -1)[0])))
    assert (got["k_head"], got["v_row"]) == (32, 64)
    k, v, ke, ve = c
    for bad in ([k, v[:3], ke, ve], [k[0], v[0], ke, ve], [k, v.view(torch.int8), ke, ve], [k.float(), v.float(), ke, ve],
                [k, v, ke.int(), ve.int()], [k, v, ke[:, :1], ve[:, :1]], [k, v, ke[..., :3], ve[..., :3]],
                [k, v, ke[..., ::2], ve[..., ::2]], [k[..., ::2], v[..., ::2], ke, ve], [k, v, ke, ve[..., :0]],
                [k[:, :, :0], v[:, :, :0], ke, ve]):
        with pytest.raises(glsa.LoraError):
            C._cache(bad, -1)


def test_runs_of_a_page():
    """A page's pieces, for the layouts that caches have."""
    t = torch.zeros(3, 4, 16, 32, dtype=torch.bfloat16)
    assert C._runs(t) == ((1, 0), (1, 0), 4 * 16 * 32)
    assert C._runs(t.transpose(1, 2).contiguous().transpose(1, 2)) == ((1, 0), (1, 0), 2048)
    assert C._runs(t[:, 1:3]) == ((1, 0), (1, 0), 1024) and C._runs(t[:, :, :8]) == ((1, 0), (4, 512), 256)
    assert C._runs(t[:, 1:3, :8, :16]) == ((2, 512), (8, 32), 16)
    assert C._runs(torch.zeros(7)) == ((1, 0), (1, 0), 1) and C._runs(torch.zeros(7, 1, 1)) == ((1, 0), (1, 0), 1)
    assert C._runs(torch.zeros(3, 8)[:, ::2]) == ((1, 0), (4, 2), 1)
    for bad in (torch.zeros(2, 2, 4, 4, 8)[:, :, :3, :3, :4], torch.zeros(2, 1, 4).expand(2, 3, 4)):
        with pytest.raises(glsa.LoraError):
            C._runs(bad)


@pytest.mark.skipif(os.path.exists("/dev/kfd"), reason="the calls pass the checks and would reach the GPU")
def test_a_workspace_suffices_for_every_smaller_call():
    """No call within the sizes asked for is refused for its workspace, whatever its type and number of chunks."""
    rng = random.Random(0)
    for hq, hk, d, B, T, nodes, ctx in ((32, 8, 128, 70, 400, 48, 20000), (8, 8, 64, 5, 9, 9, 100000), (16, 1, 256, 24, 24, 70, 3000),
                                        (4, 2, 80, 300, 900, 33, 9000), (2, 1, 16, 600, 600, 1, 700000)):
        most = glsa.quantized_workspace_bytes(B, T, nodes, ctx, hq, hk, d)
        cache = _cache(k_head=16 * d, k_row=d, v_head=16 * d, v_row=d, k_page=16 * hk * d, v_page=16 * hk * d, page_size=16,
                       block=16, k_exp_page=hk, k_exp_head=1, v_exp_page=hk, v_exp_head=1)
        n_table = -(-(ctx + nodes) // 16)
        for _ in range(200):
            b, n, c, t = rng.randint(1, B), rng.randint(1, nodes), rng.choice([ctx, rng.randint(0, ctx)]), rng.randint(1, T)
            status = _attend(cache, dt=rng.randint(0, 2), T=t, B=b, hq=hq, hk=hk, d=d, ldq=hq * d, ldo=hq * d, ld=n_table,
                             n_table=n_table, nodes=n, ctx=c, ws_bytes=most)
            assert status not in (BAD, NOT), (b, n, c, t, C._lib().lora_last_error())
