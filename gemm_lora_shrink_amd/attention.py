"""Python binding of include/lora_attention.h: the operators that follow the
adapters' q/k/v projection in a serving step.

    rope_frequencies(rot_dim, base, scaling)  -> the rotation's frequencies (host)
    rope_table(n, rot_dim, base=, scaling=)   -> cos | sin of n positions, fp32
    rotary(q, k, positions, table, ...)       positions on q and k, k and v into a paged cache
    qk_norm_rotary(q, k, q_weight, k_weight, positions, table, ...)
                                              the same after a norm of each head
    build_tree(parents, q_start, context, ...) -> masks, positions, cache rows of a step
    tree_attention(q, k_cache, v_cache, page_table, context, q_start, ...)
                                              attention of drafted tokens over the cache
    keep_path(k_caches, v_caches, page_table, context, path, n_kept)
                                              move the accepted rows behind the context

Caches are tensors [n_pages, kv_heads, page_size, head_dim] with unit inner
stride; a cache kept as [n_pages, page_size, kv_heads, head_dim] is passed as
its transpose(1, 2).  As in the rest of the package, argument checks raise
LoraError and every computation runs in the library's HIP kernels.
"""

import ctypes

import torch

from . import (LORA_ERR_INVALID_ARG, LORA_ERR_UNSUPPORTED, LoraError, _check, _check_tensor, _dtype_code, _load, _on_device,
               _rows, _stream)

ROPE_LAYOUTS = {"half": 0, "interleaved": 1}
ROPE_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "llama3": 3, "yarn": 4}
MAX_TREE_NODES = 1024
MAX_KEEP_LAYERS = 128


class _RopeConfig(ctypes.Structure):
    _fields_ = [("scaling", ctypes.c_int32), ("factor", ctypes.c_double), ("original_context", ctypes.c_double),
                ("low", ctypes.c_double), ("high", ctypes.c_double), ("magnitude", ctypes.c_double)]


class _KVCache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_page", ctypes.c_int64), ("k_head", ctypes.c_int64),
                ("k_row", ctypes.c_int64), ("v_page", ctypes.c_int64), ("v_head", ctypes.c_int64),
                ("v_row", ctypes.c_int64), ("n_pages", ctypes.c_int64), ("page_size", ctypes.c_int32)]


_bound = None


def _lib():
    """The library with this header's functions declared."""
    global _bound
    if _bound is None:
        lib = _load()
        vp, i32, i64, f32, f64, sz = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float,
                                      ctypes.c_double, ctypes.c_size_t)
        lib.lora_rope_frequencies.argtypes = [i32, f64, vp, vp, vp]
        lib.lora_rope_table.argtypes = [vp, i32, f64, i64, i64, vp, vp]
        rows = [i32, vp, i64, vp, i64, vp, i64, i32, i32, i32, i32, i32, i32]
        rest = [vp, i64, vp, vp, i64, vp, i64, vp, vp, vp]
        lib.lora_rotary.argtypes = rows + rest
        lib.lora_qk_norm_rotary.argtypes = rows + [vp, vp, f32] + rest
        lib.lora_build_tree.argtypes = [vp, i32, i32, vp, vp, i32, vp, i64, i32, i64, i32, vp, i32, vp, vp, vp]
        lib.lora_tree_attention_workspace_bytes.argtypes = [i32] * 7
        lib.lora_tree_attention_workspace_bytes.restype = sz
        lib.lora_tree_attention.argtypes = [i32, vp, i64, i32, i32, i32, i32, i32, vp, vp, i64, i32, vp, vp, i32, i32, vp,
                                            i32, f32, vp, i64, vp, vp, sz, vp]
        lib.lora_keep_path.argtypes = [i32, vp, i32, i32, i32, i32, vp, i64, i32, vp, vp, i64, i32, vp, vp]
        for name in ("rope_frequencies", "rope_table", "rotary", "qk_norm_rotary", "build_tree", "tree_attention",
                     "keep_path"):
            getattr(lib, "lora_" + name).restype = ctypes.c_int
        _bound = lib
    return _bound


def _bad(message):
    return LoraError(LORA_ERR_INVALID_ARG, message)


def _choice(table, name, what):
    try:
        return table[name]
    except (KeyError, TypeError):
        raise _bad(f"unknown {what} {name!r}") from None


def _ints(t, name, dev, numel):
    """A contiguous int32 vector of `numel` entries on the call's GPU."""
    if t.dtype != torch.int32 or t.numel() != numel or not t.is_contiguous() or not _on_device(t, dev):
        raise _bad(f"{name} must be a contiguous int32 tensor of {numel} entries on {dev}")
    return t.data_ptr()


def _int_rows(t, name, dev, rows):
    """(pointer, row stride, columns) of an int32 matrix with contiguous rows."""
    if t.dtype != torch.int32 or t.dim() != 2 or t.size(0) != rows or not _on_device(t, dev) \
            or (t.size(1) > 1 and t.stride(1) != 1):
        raise _bad(f"{name} must be an int32 tensor of {rows} contiguous rows on {dev}")
    cols = t.size(1)
    return t.data_ptr(), max(t.stride(0), cols) if rows > 1 else cols, cols


def _cache(k, v, dtype, dev, heads, d):
    """The C view of a cache; heads and d None: any."""
    if k.dim() != 4 or v.shape != k.shape:
        raise _bad("k_cache and v_cache must be [n_pages, kv_heads, page_size, head_dim] of one shape")
    n_pages, h, page, width = k.shape
    if (heads is not None and h != heads) or (d is not None and width != d):
        raise _bad(f"the cache holds {h} heads of {width}, the call has {heads} of {d}")
    ks, vs = k.stride(), v.stride()
    if ks[3] != 1 or vs[3] != 1:
        raise _bad("the cache's heads must be contiguous")
    if k.dtype != dtype or v.dtype != dtype:
        raise _bad(f"the cache must be {dtype}")
    if not (_on_device(k, dev) and _on_device(v, dev)):
        raise _bad(f"the cache must be on {dev}")
    if page < 1:
        raise _bad("the cache's pages hold no rows")
    return _KVCache(k.data_ptr(), v.data_ptr(), ks[0], ks[1], ks[2], vs[0], vs[1], vs[2], n_pages, page)


# ---- rotary positions --------------------------------------------------------

def rope_frequencies(rot_dim, base=10000.0, scaling=None):
    """(frequencies, magnitude) of a rotation of rot_dim elements: a list of
    rot_dim / 2 angles per position, and the factor of cosine and sine.

    scaling: None or a dict with "type" ("none", "linear", "ntk", "llama3",
    "yarn") and the type's numbers: "factor", "original_max_position",
    "low" and "high" (turns of the original context; defaults 1 and 4 for
    llama3, 1 and 32 for yarn), "magnitude" (yarn: 0.1 ln(factor) + 1)."""
    config = _RopeConfig()
    if scaling is not None:
        known = {"type", "factor", "original_max_position", "low", "high", "magnitude"}
        if "type" not in scaling or set(scaling) - known:
            raise _bad(f"a scaling has a type and of {sorted(known - {'type'})}: got {sorted(scaling)}")
        config = _RopeConfig(_choice(ROPE_SCALINGS, scaling["type"], "rotary scaling"), scaling.get("factor", 1.0),
                             scaling.get("original_max_position", 0.0), scaling.get("low", 0.0),
                             scaling.get("high", 0.0), scaling.get("magnitude", 0.0))
    freq = (ctypes.c_double * max(1, int(rot_dim) // 2))()
    magnitude = ctypes.c_double()
    _check(_lib().lora_rope_frequencies(rot_dim, base, ctypes.byref(config), freq, ctypes.byref(magnitude)))
    return list(freq), magnitude.value


def rope_table(n, rot_dim, *, base=10000.0, scaling=None, frequencies=None, magnitude=1.0, first=0, out=None,
               device="cuda", stream=None):
    """cos | sin of the positions first .. first + n - 1 ([n, rot_dim] fp32).

    frequencies (optional, rot_dim / 2 numbers, with magnitude): a rotation of
    the caller's own in place of base and scaling."""
    if frequencies is None:
        frequencies, magnitude = rope_frequencies(rot_dim, base, scaling)
    elif len(frequencies) != rot_dim // 2:
        raise _bad("one frequency for each pair")
    if out is None:
        out = torch.empty((n, rot_dim), dtype=torch.float32, device=device)
    if tuple(out.shape) != (n, rot_dim):
        raise _bad(f"out must be [{n}, {rot_dim}]")
    if out.device.type != "cuda":
        raise _bad(f"the table must be on a GPU (it is on {out.device})")
    _check_tensor(out, "out", out.device, dtype=torch.float32)
    freq = (ctypes.c_double * (rot_dim // 2))(*frequencies)
    _check(_lib().lora_rope_table(freq, rot_dim, magnitude, first, n, out.data_ptr(), _stream(stream, out.device)))
    return out


def _rotate(norm, q, k, positions, table, head_dim, layout, q_out, k_out, v, k_cache, v_cache, cache_rows, stream):
    dev, dtype = q.device, q.dtype
    if dev.type != "cuda":
        raise _bad(f"q must be on a GPU (it is on {dev})")
    if head_dim < 1:
        raise _bad(f"head_dim = {head_dim} must be >= 1")
    T, qw, ldq = _rows(q, "q")
    if q_out is None:
        q_out = q
    _, qow, ldqo = _rows(q_out, "q_out")
    Tk, kw, ldk = _rows(k, "k")
    if qw % head_dim or kw % head_dim or q_out.shape != q.shape or Tk != T:
        raise _bad("q, q_out and k must be rows of whole heads, one row a token")
    hk = kw // head_dim
    cached = k_cache is not None
    if k_out is None and not cached:
        k_out = k
    ldko = ldk
    if k_out is not None:
        if k_out.shape != k.shape:
            raise _bad("k_out must have k's shape")
        ldko = _rows(k_out, "k_out")[2]
    if table.dim() != 2 or table.dtype != torch.float32 or not table.is_contiguous() or not _on_device(table, dev):
        raise _bad(f"table must be a contiguous float32 [positions, rot_dim] on {dev}")
    for t, name in ((q_out, "q_out"), (k, "k"), (k_out, "k_out")):
        if t is not None and (t.dtype != dtype or t.device != dev):
            raise _bad(f"{name} must be {dtype} on {dev}, as q is")
    cache = rows = None
    ldv = 0
    if cached:
        if v is None or v_cache is None or cache_rows is None:
            raise _bad("a cache takes v, k_cache, v_cache and cache_rows")
        if v.shape != k.shape or v.dtype != dtype or v.device != dev:
            raise _bad(f"v must have k's shape and be {dtype} on {dev}")
        ldv = _rows(v, "v")[2]
        cache = _cache(k_cache, v_cache, dtype, dev, hk, head_dim)
        rows = _ints(cache_rows, "cache_rows", dev, T)
    elif v is not None or v_cache is not None or cache_rows is not None:
        raise _bad("v, v_cache and cache_rows belong to a k_cache")
    head = (_dtype_code(q), q.data_ptr(), ldq, k.data_ptr(), ldk, v.data_ptr() if cached else None, ldv, T,
            qw // head_dim, hk, head_dim, _choice(ROPE_LAYOUTS, layout, "rotary layout"), table.size(1))
    tail = (table.data_ptr(), table.size(0), _ints(positions, "positions", dev, T), q_out.data_ptr(), ldqo,
            k_out.data_ptr() if k_out is not None else None, ldko, ctypes.byref(cache) if cached else None, rows,
            _stream(stream, dev))
    if norm is None:
        _check(_lib().lora_rotary(*head, *tail))
    else:
        weights = []
        for w, name in zip(norm[:2], ("q_weight", "k_weight")):
            if w is not None and (w.dtype != dtype or w.numel() != head_dim or not w.is_contiguous()
                                  or not _on_device(w, dev)):
                raise _bad(f"{name} must be {head_dim} contiguous elements of {dtype} on {dev}")
            weights.append(w.data_ptr() if w is not None else None)
        _check(_lib().lora_qk_norm_rotary(*head, *weights, norm[2], *tail))
    return q_out, k_out


def rotary(q, k, positions, table, *, head_dim, layout="half", q_out=None, k_out=None, v=None, k_cache=None,
           v_cache=None, cache_rows=None, stream=None):
    """Turn the first table.size(1) elements of every head of q and k by the
    token's row of `table` (from rope_table).  Returns (q_out, k_out).

    q, k (and v): [T, heads * head_dim] with contiguous rows of any stride, such
    as slices of one fused q/k/v row.  q_out and k_out default to in place.
    With k_cache, v_cache and cache_rows (int32 [T], page * page_size + row)
    the rotated k and the v rows go into the cache in the same pass; k_out is
    then written only where given (None is returned for it otherwise).
    A token with a position outside the table is padding: nothing of it is
    written.  A cache row outside the cache is not written."""
    return _rotate(None, q, k, positions, table, head_dim, layout, q_out, k_out, v, k_cache, v_cache, cache_rows,
                   stream)


def qk_norm_rotary(q, k, q_weight, k_weight, positions, table, *, head_dim, eps=1e-6, layout="half", q_out=None,
                   k_out=None, v=None, k_cache=None, v_cache=None, cache_rows=None, stream=None):
    """rotary after x * weight / sqrt(mean(x^2) + eps) over every head of q and
    k, in one pass.  Weights: [head_dim] of q's dtype, or None (= 1)."""
    return _rotate((q_weight, k_weight, eps), q, k, positions, table, head_dim, layout, q_out, k_out, v, k_cache,
                   v_cache, cache_rows, stream)


# ---- trees of drafted tokens -------------------------------------------------

def build_tree(parents, q_start, context, *, max_nodes, n_tokens=None, page_table=None, n_pages=0, page_size=1,
               mask=None, positions=None, cache_rows=None, stream=None):
    """What a step's layers share, from the trees of its sequences:
    (mask, positions, cache_rows), computed once.

    parents: int32 [T], the node of the same sequence a token follows (smaller
    than its own) or -1 where it follows the context; None: chains of
    n_tokens tokens in all, whose mask is None.  q_start: int32 [B + 1], rows
    of each sequence; context: int32 [B], its tokens in the cache.  page_table:
    int32 [B, pages]; without it cache_rows is None.  mask: int64
    [T, ceil(max_nodes / 64)], bit j = sees node j."""
    dev = context.device
    if dev.type != "cuda":
        raise _bad(f"context must be on a GPU (it is on {dev})")
    B = context.numel()
    T = parents.numel() if parents is not None else n_tokens
    if T is None:
        raise _bad("n_tokens is needed where parents is None")
    words = -(-max_nodes // 64)
    if parents is not None and mask is None:
        mask = torch.zeros((T, max(words, 1)), dtype=torch.int64, device=dev)
    if mask is not None and (mask.dim() != 2 or mask.size(0) != T or mask.dtype != torch.int64
                             or not mask.is_contiguous() or not _on_device(mask, dev)):
        raise _bad(f"mask must be a contiguous int64 tensor of {T} rows on {dev}")
    if positions is None:
        positions = torch.full((T,), -1, dtype=torch.int32, device=dev)
    table = (None, 0, 0)
    if page_table is not None:
        table = _int_rows(page_table, "page_table", dev, B)
        if cache_rows is None:
            cache_rows = torch.full((T,), -1, dtype=torch.int32, device=dev)
    elif cache_rows is not None:
        raise _bad("cache_rows needs a page_table")
    _check(_lib().lora_build_tree(
        _ints(parents, "parents", dev, T) if parents is not None else None, T, B, _ints(q_start, "q_start", dev, B + 1),
        _ints(context, "context", dev, B), max_nodes, *table, n_pages, page_size,
        mask.data_ptr() if mask is not None else None, mask.size(1) if mask is not None else 0,
        _ints(positions, "positions", dev, T), _ints(cache_rows, "cache_rows", dev, T) if cache_rows is not None else None,
        _stream(stream, dev)))
    return mask, positions, cache_rows


def attention_workspace_bytes(n_seqs, n_tokens, max_nodes, max_context, q_heads, kv_heads, head_dim):
    return int(_lib().lora_tree_attention_workspace_bytes(n_seqs, n_tokens, max_nodes, max_context, q_heads, kv_heads,
                                                          head_dim))


def alloc_attention_workspace(n_seqs, n_tokens, max_nodes, max_context, q_heads, kv_heads, head_dim, device):
    """A workspace for tree_attention calls of these sizes (uint8, maybe empty)."""
    n = attention_workspace_bytes(n_seqs, n_tokens, max_nodes, max_context, q_heads, kv_heads, head_dim)
    ws = torch.empty(n, dtype=torch.uint8, device=device)
    if ws.data_ptr() % 256:
        raise _bad("allocator returned a workspace not aligned to 256 bytes")
    return ws


def tree_attention(q, k_cache, v_cache, page_table, context, q_start, *, max_nodes, max_context=None, mask=None,
                   scale=None, out=None, lse=None, workspace=None, stream=None):
    """Attention of the step's tokens over the context and the drafted tokens of
    their own sequence.  Returns out ([T, q_heads * head_dim]).

    q: [T, q_heads * head_dim], any row stride.  The tokens' own k and v are in
    the cache already (rotary puts them there).  page_table: int32 [B, pages];
    context: int32 [B]; q_start: int32 [B + 1]; mask: from build_tree, None for
    chains (one token a sequence, or tokens that each see those before them).
    max_nodes and max_context bound the sequences' new tokens and contexts (max_context
    defaults to what the page table holds).  scale defaults to
    head_dim ** -0.5.  lse (optional, float32 [T, q_heads]) receives the
    logarithm of the softmax sums.  workspace: from alloc_attention_workspace
    for these sizes or larger ones of the same heads; None where it is empty."""
    dev, dtype = q.device, q.dtype
    if dev.type != "cuda":
        raise _bad(f"q must be on a GPU (it is on {dev})")
    T, width, ldq = _rows(q, "q")
    if k_cache.dim() != 4:
        raise _bad("k_cache and v_cache must be [n_pages, kv_heads, page_size, head_dim] of one shape")
    cache = _cache(k_cache, v_cache, dtype, dev, None, None)
    hk, page, d = k_cache.size(1), k_cache.size(2), k_cache.size(3)
    if d < 1 or width % d:
        raise _bad(f"q must be rows of whole heads of {d}")
    if out is None:
        out = torch.empty((T, width), dtype=dtype, device=dev)
    if out.shape != q.shape or out.dtype != dtype or out.device != dev:
        raise _bad(f"out must have q's shape and be {dtype} on {dev}")
    ldo = _rows(out, "out")[2]
    B = context.numel()
    table, ld_table, n_table = _int_rows(page_table, "page_table", dev, B)
    if max_context is None:
        max_context = max(0, n_table * page)
    words = 0
    if mask is not None:
        if mask.dtype != torch.int64 or mask.dim() != 2 or mask.size(0) != T or not mask.is_contiguous() \
                or not _on_device(mask, dev):
            raise _bad(f"mask must be a contiguous int64 tensor of {T} rows on {dev}")
        words = mask.size(1)
    if lse is not None:
        _check_tensor(lse, "lse", dev, dtype=torch.float32, min_numel=T * (width // d))
    ws, ws_bytes = None, 0
    if workspace is not None:
        if workspace.dtype != torch.uint8 or not workspace.is_contiguous() or not _on_device(workspace, dev):
            raise _bad(f"workspace must be a contiguous uint8 tensor on {dev}")
        ws, ws_bytes = workspace.data_ptr(), workspace.numel()
    _check(_lib().lora_tree_attention(
        _dtype_code(q), q.data_ptr(), ldq, T, B, width // d, hk, d, ctypes.byref(cache), table, ld_table, n_table,
        _ints(context, "context", dev, B), _ints(q_start, "q_start", dev, B + 1), max_nodes, max_context,
        mask.data_ptr() if mask is not None else None, words, d ** -0.5 if scale is None else scale, out.data_ptr(),
        ldo, lse.data_ptr() if lse is not None else None, ws, ws_bytes, _stream(stream, dev)))
    return out


def keep_path(k_caches, v_caches, page_table, context, path, n_kept, *, stream=None):
    """For every layer's cache and every sequence b, move the rows of the nodes
    path[b, :n_kept[b]] (ascending, int32) behind the context: node path[b, j]
    to position context[b] + j.  k_caches, v_caches: the layers' caches, alike
    in shape and strides, any number of them."""
    if isinstance(k_caches, torch.Tensor):
        k_caches, v_caches = [k_caches], [v_caches]
    k_caches, v_caches = list(k_caches), list(v_caches)
    if not k_caches or len(k_caches) != len(v_caches):
        raise _bad("need as many k_caches as v_caches, one at least")
    dev, dtype = k_caches[0].device, k_caches[0].dtype
    if dev.type != "cuda":
        raise _bad(f"the caches must be on a GPU (they are on {dev})")
    if dtype not in (torch.float32, torch.float16, torch.bfloat16):
        raise LoraError(LORA_ERR_UNSUPPORTED, f"unsupported dtype {dtype}")
    caches = [_cache(k, v, dtype, dev, None, None) for k, v in zip(k_caches, v_caches)]
    shape = k_caches[0].shape
    if any(k.shape != shape for k in k_caches):
        raise _bad("the layers' caches must share one shape")
    B = context.numel()
    table = _int_rows(page_table, "page_table", dev, B)
    steps, ld_path, n_path = _int_rows(path, "path", dev, B)
    kept, at = _ints(n_kept, "n_kept", dev, B), _ints(context, "context", dev, B)
    for i in range(0, len(caches), MAX_KEEP_LAYERS):
        some = caches[i:i + MAX_KEEP_LAYERS]
        _check(_lib().lora_keep_path(_dtype_code(k_caches[0]), (_KVCache * len(some))(*some), len(some), shape[1],
                                     shape[3], B, *table, at, steps, ld_path, n_path, kept, _stream(stream, dev)))
