"""Python binding of include/lora_cache.h: a paged key/value cache held in 8
bits, and the pages of a cache of any type.

    alloc_quantized_cache(n_pages, kv_heads, page_size, head_dim, device, ...)
                                              a layer's cache (k, v, k_exp, v_exp)
    store_quantized(k, v, cache, cache_rows)  a step's keys and values into it
    tree_attention_quantized(q, cache, page_table, context, q_start, ...)
                                              attention of drafted tokens over it
    keep_path_quantized(caches, page_table, context, path, n_kept)
                                              move the accepted rows behind the context

    reserve_pages(refs, page_table, lengths, page_size=)   pages for sequences to grow into
    fork_sequences(refs, page_table, parents, children, lengths, page_size=, tensors=)
                                              sequences that share the pages of others
    release_pages(refs, page_table, rows)     give pages back
    compact_pages(refs, page_table, tensors=) the pages in use become the lowest ones
    copy_pages(tensors, source, target)       what pages hold

A cache's value is its byte's number times 2 ** exponent, one exponent for each
block of rows of a page and head: k, v [n_pages, kv_heads, page_size, head_dim]
of float8_e4m3fn or int8 with unit inner stride, exponents int8 [n_pages,
kv_heads, blocks of a page].  The page calls go by refs (int32 [n_pages], how
many table entries name a page; 0: free) and a page table (int32 [B, pages], -1
where a sequence holds none), both on the GPU, so that a step can be captured
with them.  The GPU of the tensors has to be the current one.
"""

import ctypes
import struct
from typing import NamedTuple

import torch

from . import _DTYPES, _check, _load
from .attention import _I32, _I64, _F32, _U8, MAX_HEAD_DIM, _bad, _gpu, _i32, _int_rows, _made, _matrix, _vector

CACHE_FORMATS = {torch.float8_e4m3fn: 0, torch.int8: 1}
MAX_KEEP_LAYERS = 128
_I8 = torch.int8


def _stream_of(stream, dev):
    """The stream's handle: `stream`, or the current one.  The default stream has the same handle on every GPU, so a
    call for another GPU than the current one would run on the wrong card."""
    if torch._C._cuda_getDevice() != dev:
        raise _bad(f"the tensors are on GPU {dev}, which is not the current one")
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream


class QuantizedCache(NamedTuple):
    """One layer's cache.  The functions here take any four tensors in this order."""
    k: torch.Tensor
    v: torch.Tensor
    k_exp: torch.Tensor
    v_exp: torch.Tensor


_bound = None


def _lib():
    """The library with this header's functions declared."""
    global _bound
    if _bound is None:
        lib = _load()
        vp, i32, i64, f32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
        lib.lora_store_quantized.argtypes = [i32, vp, i64, vp, i64, i32, i32, i32, vp, vp, vp]
        lib.lora_quantized_workspace_bytes.argtypes = [i32] * 7
        lib.lora_quantized_workspace_bytes.restype = sz
        lib.lora_tree_attention_quantized.argtypes = [i32, vp, i64, i32, i32, i32, i32, i32, vp, vp, i64, i32, vp, vp, i32,
                                                      i32, vp, i32, f32, vp, i64, vp, vp, sz, vp]
        lib.lora_keep_path_quantized.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, i32, vp, i64, i32, vp, vp, i64, i32, vp,
                                                 vp]
        lib.lora_pages_workspace_bytes.argtypes = [i64, i32]
        lib.lora_pages_workspace_bytes.restype = sz
        table = [vp, i64, i32, i32]
        lib.lora_reserve_pages.argtypes = [vp, i64, *table, vp, i32, vp, vp, sz, vp]
        lib.lora_fork_sequences.argtypes = [vp, i64, vp, i64, i32, vp, i64, i32, i32, vp, vp, vp, i32, i32, vp, vp, vp, vp, i32,
                                            vp, sz, vp]
        lib.lora_release_pages.argtypes = [vp, i64, *table, vp, vp, i32, i32, vp]
        lib.lora_compact_pages.argtypes = [vp, i64, *table, vp, vp, vp, vp, vp, i32, vp, sz, vp]
        lib.lora_copy_pages.argtypes = [vp, i32, i64, vp, vp, i32, vp, vp]
        for name in ("store_quantized", "tree_attention_quantized", "keep_path_quantized", "reserve_pages",
                     "fork_sequences", "release_pages", "compact_pages", "copy_pages"):
            getattr(lib, "lora_" + name).restype = ctypes.c_int
        _bound = lib
    return _bound


_CACHE_FIELDS = struct.Struct("@PPPP11q3i4x")  # lora_quantized_cache


def _cache(cache, dev):
    """(the C view of a quantized cache, the shape of k)."""
    k, v, k_exp, v_exp = cache
    shape = k.shape
    if len(shape) != 4 or v.shape != shape:
        raise _bad("a quantized cache's k and v must be [n_pages, kv_heads, page_size, head_dim] of one shape")
    code = CACHE_FORMATS.get(k.dtype)
    if code is None or v.dtype is not k.dtype:
        raise _bad(f"a quantized cache's k and v must be float8_e4m3fn or int8 (they are {k.dtype} and {v.dtype})")
    of = k_exp.shape
    if len(of) != 3 or v_exp.shape != of or of[0] != shape[0] or of[1] != shape[1] or k_exp.dtype is not _I8 \
            or v_exp.dtype is not _I8:
        raise _bad("a quantized cache's exponents must be int8 [n_pages, kv_heads, blocks of a page]")
    if k.get_device() != dev or v.get_device() != dev or k_exp.get_device() != dev or v_exp.get_device() != dev:
        raise _bad(f"the cache must be on GPU {dev}")
    n_pages, heads, page, d = shape
    blocks = of[2]
    if not 0 < page <= 0x7fffffff or heads > 0x7fffffff or d > 0x7fffffff:
        raise _bad("the cache's pages hold no rows, or more rows or heads than 32 bits count")
    if blocks < 1 or page % blocks:
        raise _bad(f"{blocks} exponents a page do not divide its {page} rows into blocks")
    k_page, k_head, k_row, k_one = k.stride()
    v_page, v_head, v_row, v_one = v.stride()
    ke_page, ke_head, ke_one = k_exp.stride()
    ve_page, ve_head, ve_one = v_exp.stride()
    if k_one != 1 or v_one != 1 or (blocks > 1 and (ke_one != 1 or ve_one != 1)):
        raise _bad("the cache's heads, and the exponents of a page, must be contiguous")
    return _CACHE_FIELDS.pack(k.data_ptr(), v.data_ptr(), k_exp.data_ptr(), v_exp.data_ptr(), k_page, k_head, k_row,
                              v_page, v_head, v_row, ke_page, ke_head, ve_page, ve_head, n_pages, page, page // blocks,
                              code), shape


# ---- a cache in 8 bits -------------------------------------------------------

def alloc_quantized_cache(n_pages, kv_heads, page_size, head_dim, device, *, dtype=torch.float8_e4m3fn, block=None):
    """A layer's cache of zeros: dtype float8_e4m3fn or int8, an exponent for
    each `block` rows of a page (a divisor of page_size; default: the page)."""
    block = page_size if block is None else block
    if dtype not in CACHE_FORMATS:
        raise _bad(f"a quantized cache is float8_e4m3fn or int8, not {dtype}")
    if page_size < 1 or block < 1 or page_size % block:
        raise _bad(f"block = {block} must divide page_size = {page_size}")
    if head_dim < 16 or head_dim % 16 or head_dim > MAX_HEAD_DIM:
        raise _bad(f"head_dim = {head_dim} of a quantized cache must be a multiple of 16 up to {MAX_HEAD_DIM}")
    rows, exps = (n_pages, kv_heads, page_size, head_dim), (n_pages, kv_heads, page_size // block)
    held = [torch.zeros(rows, dtype=_U8, device=device).view(dtype) for _ in range(2)]
    return QuantizedCache(*held, *(torch.zeros(exps, dtype=_I8, device=device) for _ in range(2)))


def store_quantized(k, v, cache, cache_rows, *, stream=None):
    """Put a step's k and v ([T, kv_heads * head_dim], rows of any stride, such
    as slices of one fused q/k/v row) into a quantized cache: token t at
    cache_rows[t] = page * page_size + row (from build_tree; one outside the
    cache is not placed).  The tokens of one block must be neighbours in
    ascending, consecutive rows, as a sequence's are.

    A block's exponent becomes the least that its new rows fit under, or stays
    where rows before them (of the same sequence) need more; it grows for the
    new rows where they need more, and the earlier ones are rounded again."""
    dev, dtype = _gpu(k, "k"), k.dtype
    code = _DTYPES.get(dtype)
    if code is None:
        raise _bad(f"unsupported dtype {dtype}")
    held, (_, heads, _, d) = _cache(cache, dev)
    T, width, ldk = _matrix(k, "k", dtype, dev)
    Tv, wv, ldv = _matrix(v, "v", dtype, dev)
    if width != heads * d or wv != width or Tv != T:
        raise _bad(f"k and v must be rows of the cache's {heads} heads of {d}, one row a token")
    lib = _bound or _lib()
    _check(lib.lora_store_quantized(code, k.data_ptr(), ldk, v.data_ptr(), ldv, T, heads, d, held,
                                    _vector(cache_rows, "cache_rows", _I32, dev, T), _stream_of(stream, dev)))


def quantized_workspace_bytes(n_seqs, n_tokens, max_nodes, max_context, q_heads, kv_heads, head_dim):
    """Bytes that suffice for every tree_attention_quantized call of these heads,
    of any type, with at most n_seqs sequences, n_tokens rows, max_nodes and
    max_context."""
    sizes = (n_seqs, n_tokens, max_nodes, max_context, q_heads, kv_heads, head_dim)
    return int(_lib().lora_quantized_workspace_bytes(*(_i32(n, "a size") for n in sizes)))


def alloc_quantized_workspace(n_seqs, n_tokens, max_nodes, max_context, q_heads, kv_heads, head_dim, device):
    """A workspace for tree_attention_quantized calls of these sizes or smaller
    ones of the same heads (uint8, maybe empty)."""
    n = quantized_workspace_bytes(n_seqs, n_tokens, max_nodes, max_context, q_heads, kv_heads, head_dim)
    ws = torch.empty(n, dtype=_U8, device=device)
    if ws.data_ptr() % 256:
        raise _bad("allocator returned a workspace not aligned to 256 bytes")
    return ws


def tree_attention_quantized(q, cache, page_table, context, q_start, *, max_nodes, max_context=None, mask=None, scale=None,
                             out=None, lse=None, workspace=None, stream=None):
    """tree_attention over a quantized cache: the same arguments with `cache` in
    place of k_cache and v_cache, and a workspace from
    alloc_quantized_workspace.  Returns out.  Keys and values enter the products
    as they are held; out has q's type."""
    dev, dtype = _gpu(q, "q"), q.dtype
    code = _DTYPES.get(dtype)
    if code is None:
        raise _bad(f"unsupported dtype {dtype}")
    T, width, ldq = _matrix(q, "q", dtype, dev)
    held, (_, kv_heads, page, d) = _cache(cache, dev)
    if d < 1 or width % d:
        raise _bad(f"q must be rows of whole heads of {d}")
    q_heads = width // d
    if out is None:
        out = _made(stream, torch.empty, (T, width), dtype=dtype, device=q.device)
    To, wo, ldo = _matrix(out, "out", dtype, dev)
    if To != T or wo != width:
        raise _bad("out must have q's shape")
    B = _i32(context.numel(), "the number of sequences")
    table, ld_table, n_table = _int_rows(page_table, "page_table", dev, B)
    _i32(max_nodes, "max_nodes")
    if max_context is None:  # of what positions and their nodes go up to
        max_context = max(0, min(n_table * page, 0x7fffffff - max_nodes))
    else:
        _i32(max_context, "max_context")
    mask_at = lse_at = ws = None
    words = ws_bytes = 0
    if mask is not None:
        shape = mask.shape
        if len(shape) != 2 or shape[0] != T:
            raise _bad(f"mask must have {T} rows")
        words = shape[1]
        mask_at = _vector(mask, "mask", _I64, dev, T * words)
    if lse is not None:
        lse_at = _vector(lse, "lse", _F32, dev, T * q_heads)
    if workspace is not None:
        ws_bytes = workspace.numel()
        ws = _vector(workspace, "workspace", _U8, dev, ws_bytes)
    lib = _bound or _lib()
    _check(lib.lora_tree_attention_quantized(
        code, q.data_ptr(), ldq, T, B, q_heads, kv_heads, d, held, table, ld_table, n_table,
        _vector(context, "context", _I32, dev, B), _vector(q_start, "q_start", _I32, dev, B + 1), max_nodes,
        max_context, mask_at, words, d ** -0.5 if scale is None else scale, out.data_ptr(), ldo, lse_at, ws, ws_bytes,
        _stream_of(stream, dev)))
    return out


def keep_path_quantized(caches, page_table, context, path, n_kept, *, stream=None):
    """keep_path over the layers' quantized caches, alike in shapes, strides and
    type (a list of them, any number; no tensor twice, exponents neither).  A row that
    moves into a block of a larger exponent is rounded again."""
    n = len(caches)
    if n < 1:
        raise _bad("need one cache at least")
    first = caches[0]
    dev = _gpu(first[0], "the cache")
    held, shape = _cache(first, dev)
    if any(len(c) != 4 for c in caches):
        raise _bad("a quantized cache is k, v, k_exp and v_exp")
    at = []
    for t, like in zip(zip(*caches), first):
        shape_, dtype, stride = like.shape, like.dtype, like.stride()
        dense = like.is_contiguous()
        for x in t:
            if x.shape != shape_ or x.dtype is not dtype or x.get_device() != dev or (
                    not x.is_contiguous() if dense else x.stride() != stride):
                raise _bad("the layers' caches must be alike in shape, strides, type and GPU")
        at.append([x.data_ptr() for x in t])
    if shape[0] and len(set().union(*at)) != 4 * n:
        raise _bad("a cache, or exponents, are listed twice")  # rows would move, or be rounded, twice at once
    B = _i32(context.numel(), "the number of sequences")
    table = _int_rows(page_table, "page_table", dev, B)
    steps = _int_rows(path, "path", dev, B)
    kept, ctx = _vector(n_kept, "n_kept", _I32, dev, B), _vector(context, "context", _I32, dev, B)
    for i in range(0, n, MAX_KEEP_LAYERS):
        m = min(n - i, MAX_KEEP_LAYERS)
        layers = struct.Struct(f"@{m}P")
        _check(_lib().lora_keep_path_quantized(held, *(layers.pack(*x[i:i + m]) for x in at), m, shape[1], shape[3], B,
                                               *table, ctx, *steps, kept, _stream_of(stream, dev)))


# ---- pages -------------------------------------------------------------------

_TENSOR_FIELDS = struct.Struct("@P3q3i4x")  # lora_paged_tensor


def _runs(t):
    """(outer, inner, run) of a page of t as (number, stride) pairs in elements:
    its dimensions by falling stride, joined where they follow one another."""
    dims = sorted(((s, n) for n, s in zip(t.shape[1:], t.stride()[1:]) if n > 1), reverse=True)
    joined = []
    for s, n in dims:
        if joined and joined[-1][1] == s * n:
            joined[-1] = (joined[-1][0] * n, s)
        else:
            joined.append((n, s))
    run = 1
    if joined and joined[-1][1] == 1:
        run = joined.pop()[0]
    if len(joined) > 2 or any(s < 1 for _, s in joined):
        raise _bad(f"a page of shape {tuple(t.shape[1:])} and strides {t.stride()[1:]} is in too many pieces to be copied")
    joined = [(1, 0)] * (2 - len(joined)) + joined
    return joined[0], joined[1], run


def _listed(tensors):
    """A tuple of tensors, or of the one that is given."""
    return (tensors,) if isinstance(tensors, torch.Tensor) else tuple(tensors)


class PagedTensors:
    """Tensors whose first dimension is the pages of one pool (the layers' k, v and
    exponents), laid out once for copy_pages, fork_sequences and compact_pages."""

    def __init__(self, tensors):
        self.tensors = _listed(tensors)
        if not self.tensors:
            raise _bad("need one tensor at least")
        self.dev = _gpu(self.tensors[0], "a paged tensor")
        self.n_pages = self.tensors[0].size(0) if self.tensors[0].dim() else 0
        packed = []
        for t in self.tensors:
            if t.dim() < 1 or t.size(0) != self.n_pages or t.get_device() != self.dev:
                raise _bad(f"paged tensors must have {self.n_pages} pages each, on one GPU")
            if t.numel() == 0:
                if self.n_pages:
                    raise _bad("the pages of a tensor hold nothing")
                continue
            (n_outer, outer), (n_inner, inner), run = _runs(t)
            e = t.element_size()
            if max(n_outer, n_inner, run * e) > 0x7fffffff:
                raise _bad("a page is larger than 32 bits count")
            if self.n_pages > 1 and t.stride(0) < 1:
                raise _bad("the pages of a tensor lie on each other")
            packed.append(_TENSOR_FIELDS.pack(t.data_ptr(), t.stride(0) * e, outer * e, inner * e, n_outer, n_inner, run * e))
        self.n, self.packed = len(packed), b"".join(packed)


def _paged(tensors):
    return tensors if isinstance(tensors, PagedTensors) else PagedTensors(tensors)


def _of_pool(tensors, n_pages, dev):
    """(the C view, the number) of a pool's tensors, of which there may be none."""
    if not isinstance(tensors, PagedTensors):
        tensors = _listed(tensors)
        if not tensors:
            return None, 0
        tensors = PagedTensors(tensors)
    if tensors.n_pages != n_pages or tensors.dev != dev:
        raise _bad(f"the tensors must have the pool's {n_pages} pages and be on its GPU")
    return tensors.packed, tensors.n


def copy_pages(tensors, source, target, *, count=None, stream=None):
    """Copy page source[i] to page target[i] (int32 [n]) in every tensor: a list of
    tensors with the pages of one pool as their first dimension, or a
    PagedTensors of it, which saves laying them out again.  No target may be in
    another pair.  Numbers outside the pool are passed over; count (int32, one
    entry, optional) bounds the pairs from the GPU."""
    tensors = _paged(tensors)
    dev, n = tensors.dev, _i32(source.numel(), "the number of pairs")
    _check(_lib().lora_copy_pages(tensors.packed, tensors.n, tensors.n_pages, _vector(source, "source", _I32, dev, n),
                                  _vector(target, "target", _I32, dev, n), n,
                                  None if count is None else _vector(count, "count", _I32, dev, 1),
                                  _stream_of(stream, dev)))


def _moves(n_pages, n_seqs):
    """Pairs of pages that a call may have to copy."""
    return max(n_pages // 2, n_seqs, 1)


def pages_workspace_bytes(n_pages, n_seqs):
    """Bytes for reserve_pages, fork_sequences and compact_pages on a pool of
    n_pages with at most n_seqs sequences or forks a call."""
    need = int(_lib().lora_pages_workspace_bytes(n_pages, _i32(n_seqs, "n_seqs")))
    if need == 0:
        raise _bad(f"no pool has {n_pages} pages and {n_seqs} sequences")
    return 4 * (2 * _moves(n_pages, n_seqs) + 1) + need


def alloc_pages_workspace(n_pages, n_seqs, device):
    """A workspace (uint8) for reserve_pages, fork_sequences and compact_pages; calls
    that may overlap need distinct ones."""
    return torch.empty(pages_workspace_bytes(n_pages, n_seqs), dtype=_U8, device=device)


def _space(workspace, n_pages, n_seqs, refs, dev, stream):
    """Addresses in a workspace: (sources, targets, number of moves, the library's own, its bytes, the tensor)."""
    if workspace is None:
        workspace = _made(stream, alloc_pages_workspace, n_pages, n_seqs, refs.device)
    size, n = workspace.numel(), _moves(n_pages, n_seqs)
    at = _vector(workspace, "workspace", _U8, dev, size)
    if at % 4:
        raise _bad("the workspace must be 4-byte aligned")
    used = 4 * (2 * n + 1)
    if size < used:
        raise _bad(f"the workspace has {size} bytes, the call needs {pages_workspace_bytes(n_pages, n_seqs)}")
    return at, at + 4 * n, at + 8 * n, at + used, size - used, workspace


def _pool(refs):
    """(GPU index, address, pages) of a pool's reference counts."""
    dev, n = _gpu(refs, "refs"), refs.numel()
    return dev, _vector(refs, "refs", _I32, dev, n), n


def _table(page_table, name, dev):
    """(address, row stride, columns, rows) of a page table."""
    if page_table.dim() != 2:
        raise _bad(f"{name} must be a matrix")
    B = page_table.size(0)
    if B == 0:
        return None, page_table.size(1), page_table.size(1), 0
    return (*_int_rows(page_table, name, dev, B), _i32(B, "the number of sequences"))


def reserve_pages(refs, page_table, lengths, *, page_size, missing=None, workspace=None, stream=None):
    """Give every sequence the pages that lengths[b] (int32 [B]) tokens need and it
    lacks, free ones from the lowest number on, in the order of sequences.
    missing (int32, one entry, optional) receives how many there were not: their
    entries stay -1."""
    dev, at, n = _pool(refs)
    table = _table(page_table, "page_table", dev)
    *_, ws, ws_bytes, kept = _space(workspace, n, table[3], refs, dev, stream)
    _check(_lib().lora_reserve_pages(at, n, *table, _vector(lengths, "lengths", _I32, dev, table[3]),
                                     _i32(page_size, "page_size"),
                                     None if missing is None else _vector(missing, "missing", _I32, dev, 1), ws, ws_bytes,
                                     _stream_of(stream, dev)))


def fork_sequences(refs, page_table, parents, children, lengths, *, page_size, tensors=(), out_table=None, missing=None,
                   workspace=None, stream=None):
    """Fork f makes row children[f] of out_table (default: page_table itself) a
    sequence with the first lengths[f] tokens of row parents[f] of page_table
    (int32 [n] each): full pages are shared, one that is filled in part becomes
    a copy on a free page, in every tensor (a list or a PagedTensors; none: only
    the tables).  Returns out_table.

    Children must differ, and in one table none may be a parent; what a child's
    row held before is overwritten, not released.  A step of beams forks into
    another table and releases the old one.  missing (int32, one entry,
    optional) receives the number of forks whose copy found no free page."""
    dev, at, n = _pool(refs)
    source = _table(page_table, "page_table", dev)
    if out_table is None:
        out_table = page_table
    to = _table(out_table, "out_table", dev)
    if to[2] != source[2]:
        raise _bad(f"out_table must have {source[2]} columns (it has {to[2]})")
    m = _i32(parents.numel(), "the number of forks")
    packed, n_tensors = _of_pool(tensors, n, dev)
    of, dest, _, ws, ws_bytes, kept = _space(workspace, n, m, refs, dev, stream)
    _check(_lib().lora_fork_sequences(
        at, n, source[0], source[1], source[3], to[0], to[1], to[3], to[2], _vector(parents, "parents", _I32, dev, m),
        _vector(children, "children", _I32, dev, m), _vector(lengths, "lengths", _I32, dev, m), m,
        _i32(page_size, "page_size"), of, dest, None if missing is None else _vector(missing, "missing", _I32, dev, 1),
        packed, n_tensors, ws, ws_bytes, _stream_of(stream, dev)))
    return out_table


def release_pages(refs, page_table, rows=None, *, keep=None, page_size=None, stream=None):
    """Give back the pages of the sequences `rows` (int32 [n]; None: all), or, with
    keep (int32 [n], tokens that stay) and page_size, those behind keep's.  Their
    entries become -1.  A row listed twice is released once."""
    dev, at, n = _pool(refs)
    table = _table(page_table, "page_table", dev)
    m = table[3] if rows is None else _i32(rows.numel(), "the number of rows")
    if keep is not None and page_size is None:
        raise _bad("keep needs a page_size")
    _check(_lib().lora_release_pages(at, n, *table, None if rows is None else _vector(rows, "rows", _I32, dev, m),
                                     None if keep is None else _vector(keep, "keep", _I32, dev, m), m,
                                     1 if page_size is None else _i32(page_size, "page_size"), _stream_of(stream, dev)))


def compact_pages(refs, page_table, *, tensors=(), n_live=None, workspace=None, stream=None):
    """Move what lies on the highest pages in use to free ones below, in every tensor
    (a list or a PagedTensors), so that the n pages in use are the first n; refs and
    page_table follow.  Returns n_live, an int32 tensor of one entry: n.  Every
    table that names pages of the pool has to be in page_table."""
    dev, at, n = _pool(refs)
    table = _table(page_table, "page_table", dev)
    packed, n_tensors = _of_pool(tensors, n, dev)
    if n_live is None:
        n_live = _made(stream, torch.empty, (), dtype=_I32, device=refs.device)
    of, dest, moved, ws, ws_bytes, kept = _space(workspace, n, 0, refs, dev, stream)
    _check(_lib().lora_compact_pages(at, n, *table, of, dest, _vector(n_live, "n_live", _I32, dev, 1), moved, packed,
                                     n_tensors, ws, ws_bytes, _stream_of(stream, dev)))
    return n_live
