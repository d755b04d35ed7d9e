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
LoraError and every computation runs in the library's HIP kernels.  With
stream= another stream than torch's current one, the tensors that a call
returns are made on that stream.
"""

import ctypes
import struct

import torch

from . import LORA_ERR_INVALID_ARG, LORA_ERR_UNSUPPORTED, LoraError, _check, _DTYPES, _load

ROPE_LAYOUTS = {"half": 0, "interleaved": 1}
ROPE_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "llama3": 3, "yarn": 4}
MAX_HEAD_DIM = 256
MAX_TREE_NODES = 1024
MAX_KEEP_LAYERS = 128


class _RopeConfig(ctypes.Structure):
    _fields_ = [("scaling", ctypes.c_int32), ("factor", ctypes.c_double), ("original_context", ctypes.c_double),
                ("low", ctypes.c_double), ("high", ctypes.c_double), ("magnitude", ctypes.c_double)]


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
        lib.lora_keep_path.argtypes = [i32, vp, vp, vp, i32, i32, i32, i32, vp, i64, i32, vp, vp, i64, i32, vp, vp]
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


# The checks below run on every call of a decode step, where the host's time
# counts: they ask each tensor once for its shape, strides, type and device
# index (-1 on the host) and build no message unless they refuse.

_I32, _I64, _F32, _U8 = torch.int32, torch.int64, torch.float32, torch.uint8


def _gpu(t, name):
    """The GPU index of the tensor that says where the call runs."""
    dev = t.get_device()
    if dev < 0:
        raise _bad(f"{name} must be on a GPU (it is on {t.device})")
    return dev


def _stream_of(stream, dev):
    """The stream's handle: `stream`, or the current one of GPU `dev`."""
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream


def _i32(value, name):
    """A number that the C ABI takes in 32 bits (ctypes would cut it to them)."""
    if -0x80000000 <= value <= 0x7fffffff:
        return value
    raise _bad(f"{name} = {value} is beyond 32 bits")


def _made(stream, make, *args, **kw):
    """make(*args, **kw), a new tensor, on the stream of the call that it is for:
    a fill on the current stream would not be ordered with the call on another,
    and a block that was freed there may still be in use."""
    if stream is None:
        return make(*args, **kw)
    with torch.cuda.stream(stream):
        return make(*args, **kw)


def _matrix(t, name, dtype, dev):
    """(rows, width, row stride) of a matrix with contiguous rows."""
    shape = t.shape
    if len(shape) != 2 or t.dtype is not dtype or t.get_device() != dev:
        raise _bad(f"{name} must be a matrix of {dtype} on GPU {dev} (it is {t.dtype} of {tuple(shape)} on {t.device})")
    rows, width = shape
    if rows > 0x7fffffff or width > 0x7fffffff:
        raise _bad(f"{name} has more rows or columns than 32 bits count")
    ld, inner = t.stride()
    if rows < 2 or width < 1:  # the stride of a single row is no one's
        ld = max(ld, width, 1)
    if inner != 1 and width > 1:
        raise _bad(f"{name} must have contiguous rows")
    return rows, width, ld


def _vector(t, name, dtype, dev, numel):
    """The address of a contiguous tensor of numel entries."""
    if t.dtype is not dtype or t.numel() != numel or t.get_device() != dev or not t.is_contiguous():
        raise _bad(f"{name} must be contiguous, {numel} entries of {dtype} on GPU {dev}")
    return t.data_ptr()


def _int_rows(t, name, dev, rows):
    """(address, row stride, columns) of an int32 matrix of `rows` rows."""
    n, cols, ld = _matrix(t, name, _I32, dev)
    if n != rows:
        raise _bad(f"{name} must have {rows} rows (it has {n})")
    if ld < cols:
        raise _bad(f"the rows of {name} overlap: {cols} columns, row stride {ld} (an expanded row, say)")
    return t.data_ptr(), ld, cols


_CACHE_FIELDS = struct.Struct("@PP7qi")  # lora_kv_cache


def _cache(k, v, dtype, dev):
    """(the C view of a cache, its shape)."""
    shape = k.shape
    if len(shape) != 4 or v.shape != shape:
        raise _bad("k_cache and v_cache must be [n_pages, kv_heads, page_size, head_dim] of one shape")
    if k.dtype is not dtype or v.dtype is not dtype or k.get_device() != dev or v.get_device() != dev:
        raise _bad(f"the cache must be {dtype} on GPU {dev}")
    k_page, k_head, k_row, k_one = k.stride()
    v_page, v_head, v_row, v_one = v.stride()
    if k_one != 1 or v_one != 1:
        raise _bad("the cache's heads must be contiguous")
    if not 0 < shape[2] <= 0x7fffffff or shape[1] > 0x7fffffff:
        raise _bad("the cache's pages hold no rows, or more rows or heads than 32 bits count")
    return _CACHE_FIELDS.pack(k.data_ptr(), v.data_ptr(), k_page, k_head, k_row, v_page, v_head, v_row, shape[0],
                              shape[2]), shape


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
    if not 0 <= _i32(rot_dim, "rot_dim") <= MAX_HEAD_DIM:
        raise _bad(f"rot_dim = {rot_dim} must be even, from 2 to {MAX_HEAD_DIM}")
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
    elif len(frequencies) != _i32(rot_dim, "rot_dim") // 2:
        raise _bad("one frequency for each pair")
    if not -(1 << 63) <= first < 1 << 63:
        raise _bad(f"first = {first} is no position")
    if out is None:
        out = _made(stream, torch.empty, (n, rot_dim), dtype=_F32, device=device)
    if tuple(out.shape) != (n, rot_dim):
        raise _bad(f"out must be [{n}, {rot_dim}]")
    dev = _gpu(out, "the table")
    to = _vector(out, "out", _F32, dev, n * rot_dim)
    freq = (ctypes.c_double * (rot_dim // 2))(*frequencies)
    _check(_lib().lora_rope_table(freq, rot_dim, magnitude, first, n, to, _stream_of(stream, dev)))
    return out


def _rotate(norm, q, k, positions, table, head_dim, layout, q_out, k_out, v, k_cache, v_cache, cache_rows, stream):
    dev, dtype = _gpu(q, "q"), q.dtype
    code = _DTYPES.get(dtype)
    if code is None:
        raise _bad(f"unsupported dtype {dtype}")
    if _i32(head_dim, "head_dim") < 1:
        raise _bad(f"head_dim = {head_dim} must be >= 1")
    T, qw, ldq = _matrix(q, "q", dtype, dev)
    Tk, kw, ldk = _matrix(k, "k", dtype, dev)
    q_heads, kv_heads = qw // head_dim, kw // head_dim
    if q_heads * head_dim != qw or kv_heads * head_dim != kw or Tk != T:
        raise _bad("q and k must be rows of whole heads, one row a token")
    if q_out is None:
        q_out, ldqo = q, ldq
    else:
        To, wo, ldqo = _matrix(q_out, "q_out", dtype, dev)
        if To != T or wo != qw:
            raise _bad("q_out must have q's shape")
    cache = rows = v_at = k_to = None
    ldv, ldko = 0, ldk
    if k_cache is not None:
        if v is None or v_cache is None or cache_rows is None:
            raise _bad("a cache takes v, k_cache, v_cache and cache_rows")
        Tv, vw, ldv = _matrix(v, "v", dtype, dev)
        if Tv != T or vw != kw:
            raise _bad("v must have k's shape")
        cache, shape = _cache(k_cache, v_cache, dtype, dev)
        if shape[1] != kv_heads or shape[3] != head_dim:
            raise _bad(f"the cache holds {shape[1]} heads of {shape[3]}, the call has {kv_heads} of {head_dim}")
        rows, v_at = _vector(cache_rows, "cache_rows", _I32, dev, T), v.data_ptr()
    elif v is not None or v_cache is not None or cache_rows is not None:
        raise _bad("v, v_cache and cache_rows belong to a k_cache")
    elif k_out is None:
        k_out = k
    if k_out is k:
        k_to = k.data_ptr()
    elif k_out is not None:
        To, wo, ldko = _matrix(k_out, "k_out", dtype, dev)
        if To != T or wo != kw:
            raise _bad("k_out must have k's shape")
        k_to = k_out.data_ptr()
    n_positions, rot, ld = _matrix(table, "table", _F32, dev)
    if ld != rot and n_positions > 1:
        raise _bad("table must be contiguous")
    lib = _bound or _lib()
    if norm is None:
        call, extra = lib.lora_rotary, ()
    else:
        call = lib.lora_qk_norm_rotary
        extra = (None if norm[0] is None else _vector(norm[0], "q_weight", dtype, dev, head_dim),
                 None if norm[1] is None else _vector(norm[1], "k_weight", dtype, dev, head_dim), norm[2])
    _check(call(code, q.data_ptr(), ldq, k.data_ptr(), ldk, v_at, ldv, T, q_heads, kv_heads, head_dim,
                _choice(ROPE_LAYOUTS, layout, "rotary layout"), rot, *extra, table.data_ptr(), n_positions,
                _vector(positions, "positions", _I32, dev, T), q_out.data_ptr(), ldqo, k_to, ldko, cache, rows,
                _stream_of(stream, dev)))
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

def build_tree(parents, q_start, context, *, max_nodes, n_tokens=None, page_table=None, n_pages=None, page_size=None,
               mask=None, positions=None, cache_rows=None, stream=None):
    """What a step's layers share, from the trees of its sequences:
    (mask, positions, cache_rows), computed once.

    parents: int32 [T], the node of the same sequence a token follows (smaller
    than its own) or -1 where it follows the context; None: chains of
    n_tokens tokens in all, whose mask is None.  q_start: int32 [B + 1], rows
    of each sequence; context: int32 [B], its tokens in the cache.  page_table:
    int32 [B, pages], with the n_pages and page_size of the cache; without it
    cache_rows is None.  mask: int64 [T, ceil(max_nodes / 64)], bit j = sees
    node j."""
    dev = _gpu(context, "context")
    device = context.device
    B = _i32(context.numel(), "the number of sequences")
    T = parents.numel() if parents is not None else n_tokens
    if T is None:
        raise _bad("n_tokens is needed where parents is None")
    _i32(T, "the number of tokens")
    _i32(max_nodes, "max_nodes")
    words = 0
    if parents is not None and mask is None:
        mask = _made(stream, torch.zeros, (T, max(-(-max_nodes // 64), 1)), dtype=_I64, device=device)
    if mask is not None:
        if mask.dim() != 2 or mask.size(0) != T:
            raise _bad(f"mask must have {T} rows")
        _vector(mask, "mask", _I64, dev, mask.numel())
        words = mask.size(1)
    if positions is None:
        positions = _made(stream, torch.full, (T,), -1, dtype=_I32, device=device)
    table = (None, 0, 0)
    if page_table is not None:
        if n_pages is None or page_size is None:
            raise _bad("a page_table takes the cache's n_pages and page_size")
        _i32(page_size, "page_size")
        table = _int_rows(page_table, "page_table", dev, B)
        if cache_rows is None:
            cache_rows = _made(stream, torch.full, (T,), -1, dtype=_I32, device=device)
    else:
        if cache_rows is not None:
            raise _bad("cache_rows needs a page_table")
        n_pages, page_size = 0, 1
    _check(_lib().lora_build_tree(
        None if parents is None else _vector(parents, "parents", _I32, dev, T), T, B,
        _vector(q_start, "q_start", _I32, dev, B + 1), _vector(context, "context", _I32, dev, B), max_nodes, *table,
        n_pages, page_size, None if mask is None else mask.data_ptr(), words,
        _vector(positions, "positions", _I32, dev, T),
        None if cache_rows is None else _vector(cache_rows, "cache_rows", _I32, dev, T), _stream_of(stream, dev)))
    return mask, positions, cache_rows


def attention_workspace_bytes(n_seqs, n_tokens, max_nodes, max_context, q_heads, kv_heads, head_dim):
    """Bytes that suffice for every tree_attention call of these heads, of any
    type, with at most n_seqs sequences, n_tokens rows, max_nodes and max_context."""
    sizes = (n_seqs, n_tokens, max_nodes, max_context, q_heads, kv_heads, head_dim)
    return int(_lib().lora_tree_attention_workspace_bytes(*(_i32(n, "a size") for n in sizes)))


def alloc_attention_workspace(n_seqs, n_tokens, max_nodes, max_context, q_heads, kv_heads, head_dim, device):
    """A workspace for tree_attention calls of these sizes or smaller ones of the
    same heads (uint8, maybe empty)."""
    n = attention_workspace_bytes(n_seqs, n_tokens, max_nodes, max_context, q_heads, kv_heads, head_dim)
    ws = torch.empty(n, dtype=torch.uint8, device=device)
    if ws.data_ptr() % 256:
        raise _bad("allocator returned a workspace not aligned to 256 bytes")
    return ws


def tree_attention(q, k_cache, v_cache, page_table, context, q_start, *, max_nodes, max_context=None, mask=None,
                   scale=None, out=None, lse=None, workspace=None, stream=None):
    """Attention of the step's tokens over the context and the drafted tokens of
    their own sequence.  Returns out ([T, q_heads * head_dim]); rows of no sequence
    are not written, so in an out of the call's own making they hold anything.

    q: [T, q_heads * head_dim], any row stride.  The tokens' own k and v are in
    the cache already (rotary puts them there).  page_table: int32 [B, pages];
    context: int32 [B]; q_start: int32 [B + 1]; mask: from build_tree, None for
    chains (one token a sequence, or tokens that each see those before them).
    max_nodes and max_context bound the sequences' new tokens and contexts (max_context
    defaults to what the page table holds).  scale defaults to
    head_dim ** -0.5.  lse (optional, float32 [T, q_heads]) receives the
    logarithm of the softmax sums.  workspace: from alloc_attention_workspace
    for these sizes or larger ones of the same heads, so one for the largest batch
    serves all; None where it is empty."""
    dev, dtype = _gpu(q, "q"), q.dtype
    code = _DTYPES.get(dtype)
    if code is None:
        raise _bad(f"unsupported dtype {dtype}")
    T, width, ldq = _matrix(q, "q", dtype, dev)
    cache, (n_pages, kv_heads, page, d) = _cache(k_cache, v_cache, dtype, dev)
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
    _check(lib.lora_tree_attention(
        code, q.data_ptr(), ldq, T, B, q_heads, kv_heads, d, cache, table, ld_table, n_table,
        _vector(context, "context", _I32, dev, B), _vector(q_start, "q_start", _I32, dev, B + 1), max_nodes,
        max_context, mask_at, words, d ** -0.5 if scale is None else scale, out.data_ptr(), ldo, lse_at, ws, ws_bytes,
        _stream_of(stream, dev)))
    return out


def keep_path(k_caches, v_caches, page_table, context, path, n_kept, *, stream=None):
    """For every layer's cache and every sequence b, move the rows of the nodes
    path[b, :n_kept[b]] (ascending, int32) behind the context: node path[b, j]
    to position context[b] + j.  k_caches, v_caches: the layers' caches, alike
    in shape and strides, any number of them."""
    if isinstance(k_caches, torch.Tensor):
        k_caches, v_caches = (k_caches,), (v_caches,)
    n = len(k_caches)
    if n < 1 or len(v_caches) != n:
        raise _bad("need as many k_caches as v_caches, one at least")
    k, v = k_caches[0], v_caches[0]
    dev, dtype = _gpu(k, "the cache"), k.dtype
    code = _DTYPES.get(dtype)
    if code is None:
        raise LoraError(LORA_ERR_UNSUPPORTED, f"unsupported dtype {dtype}")
    cache, shape = _cache(k, v, dtype, dev)
    if n > 1:
        ks, vs = k.stride(), v.stride()
        for caches, strides in ((k_caches, ks), (v_caches, vs)):
            for c in caches:
                if c.shape != shape or c.stride() != strides or c.dtype is not dtype or c.get_device() != dev:
                    raise _bad("the layers' caches must be alike in shape, strides, type and GPU")
    B = _i32(context.numel(), "the number of sequences")
    table = _int_rows(page_table, "page_table", dev, B)
    steps = _int_rows(path, "path", dev, B)
    kept, at = _vector(n_kept, "n_kept", _I32, dev, B), _vector(context, "context", _I32, dev, B)
    k_at, v_at = [c.data_ptr() for c in k_caches], [c.data_ptr() for c in v_caches]
    for i in range(0, n, MAX_KEEP_LAYERS):
        m = min(n - i, MAX_KEEP_LAYERS)
        layers = struct.Struct(f"@{m}P")
        _check(_lib().lora_keep_path(code, cache, layers.pack(*k_at[i:i + m]), layers.pack(*v_at[i:i + m]), m, shape[1],
                                     shape[3], B, *table, at, *steps, kept, _stream_of(stream, dev)))
