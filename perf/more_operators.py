"""What is timed of a paged cache held in 8 bits and of the pages of a cache.

Keys and values of a step's tokens are put into a cache of bytes with an exponent for each block of tokens and head, a
tree of drafted tokens attends over it, and the accepted path is kept.  Sequences are forked (the beams of a request
share the pages of what they have in common), finished ones give their pages back, and the pool is compacted.  Head
shapes are those of the workloads of this repository (32 query and 8 key/value heads of 128, 256 and 8192 tokens) or
generic.

The cache: k, v [n_pages, kv_heads, page, d] of float8_e4m3fn or int8 and exponents int8 [n_pages, kv_heads,
page / block]; a value is its byte's number times 2 ** exponent.  The bytes and the exponents are compared as they are
held, which is stricter than comparing the values that they stand for: every rounding is to a power of two's grid.

`own` false: the operators in elementary torch operations.  `own` true: the library's entry points.
"""

import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}
FORMATS = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}
LARGEST = {"e4m3": 448.0, "int8": 127.0}  # the largest number of a byte
TOP = {"e4m3": 119, "int8": 121}          # the largest exponent whose values are finite in fp32
LOW = -126                                # the smallest


# ---- cases ------------------------------------------------------------------

def listed():
    return [
        # one decode step of 256 requests: a token each, into blocks that are partly filled
        dict(name="store_decode_256", op="store", B=256, n=1, ragged=False, ctx=60, hk=8, d=128, dtype="bf16", fmt="e4m3",
             page=16, block=16),
        # prompts of up to 512 tokens behind contexts of odd lengths
        dict(name="store_prompt_16", op="store", B=16, n=512, ragged=True, ctx=100, hk=8, d=128, dtype="bf16", fmt="int8",
             page=32, block=8),
        # the smallest call: one request, one token, a short context
        dict(name="attend_one_100", op="attend", B=1, nodes=1, ctx=100, ragged=False, tree=False, hq=32, hk=8, d=128,
             dtype="bf16", fmt="e4m3", page=16, block=16),
        # a full decode batch, contexts of all lengths
        dict(name="attend_decode_256", op="attend", B=256, nodes=1, ctx=4096, ragged=True, tree=False, hq=32, hk=8,
             d=128, dtype="bf16", fmt="e4m3", page=16, block=16),
        # one request with a long context and a wide tree
        dict(name="attend_tree64_32768", op="attend", B=1, nodes=64, ctx=32768, ragged=False, tree=True, hq=32, hk=8,
             d=128, dtype="bf16", fmt="e4m3", page=64, block=32),
        # 16 requests, trees and contexts of different sizes, pages that are no power of two
        dict(name="attend_ragged_16", op="attend", B=16, nodes=45, ctx=8192, ragged=True, tree=True, hq=32, hk=8, d=128,
             dtype="f16", fmt="int8", page=24, block=8),
        # the accepted path of one request, four layers
        dict(name="keep_1", op="keep", B=1, layers=4, path=4, nodes=16, ctx=500, hk=8, d=128, fmt="e4m3", page=16,
             block=16),
        # the accepted paths of a batch, eight layers at once
        dict(name="keep_64", op="keep", B=64, layers=8, path=8, nodes=64, ctx=300, hk=8, d=128, fmt="int8", page=16,
             block=4),
        # a step of one request's beams
        dict(name="fork_4", op="fork", B=4, ctx=500, layers=4, hk=8, d=128, fmt="e4m3", page=16, block=16),
        # a step of the beams of 64 requests, four each
        dict(name="fork_256", op="fork", B=256, ctx=1000, layers=8, hk=8, d=128, fmt="e4m3", page=16, block=16),
        # a small pool, a few requests done
        dict(name="compact_100", op="compact", B=10, ctx=150, layers=2, hk=8, d=64, fmt="e4m3", page=16, block=16),
        # a pool of 2 GB (all layers) from which half of the requests are gone
        dict(name="compact_8192", op="compact", B=64, ctx=2100, layers=8, hk=8, d=128, fmt="e4m3", page=16, block=16),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["store", "store", "store", "attend", "attend", "attend", "attend", "keep", "keep", "fork", "fork",
                     "compact"])
    page = rng.choice([8, 16, 24, 32, 64, 128])
    block = rng.choice([b for b in (1, 2, 4, 8, 16, 24, 32, 64, 128) if page % b == 0])
    hk = rng.choice([1, 2, 4, 8, 16])
    d = rng.choice([64, 80, 128, 128, 256])
    held = dict(hk=hk, d=d, fmt=rng.choice(["e4m3", "e4m3", "int8"]), page=page, block=block)
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op == "store":
        B = _log(rng, 1, 256)
        n = min(_log(rng, 1, 2048), max(1, 8192 * 8 * 128 // (B * hk * d)))
        return dict(op=op, B=B, n=n, ragged=rng.random() < 0.6, ctx=_log(rng, 1, 100), dtype=dtype, **held)
    if op == "attend":
        hq = hk * rng.choice([g for g in (1, 2, 4, 8) if hk * g <= 32])
        B = _log(rng, 1, 256)
        nodes = _log(rng, 1, 128)
        ctx = _log(rng, 16, 32768)
        # no more keys in all, and no more products, than the largest listed cases have
        ctx = max(1, min(ctx, (1 << 29) // (B * hk * d), (1 << 33) // (B * nodes * hq * d)))
        return dict(op=op, B=B, nodes=nodes, ctx=ctx, ragged=rng.random() < 0.6, tree=rng.random() < 0.6, hq=hq,
                    dtype=dtype, **held)
    held.update(hk=min(hk, 8), d=min(d, 128))
    layers = rng.choice([1, 2, 5, 8])
    if op == "keep":
        nodes = _log(rng, 1, 64)
        return dict(op=op, B=_log(rng, 1, 64), layers=layers, path=_log(rng, 1, min(nodes, 12)), nodes=nodes,
                    ctx=_log(rng, 1, 300), **held)
    if op == "fork":
        held.update(page=min(page, 32), block=min(block, 8))
        return dict(op=op, B=_log(rng, 1, 200), ctx=_log(rng, 1, 1000), layers=layers, **held)
    held.update(page=min(page, 32), block=min(block, 8))
    return dict(op=op, B=_log(rng, 2, 60), ctx=_log(rng, 16, 2000), layers=layers, **held)


# ---- inputs -----------------------------------------------------------------

def _spread(B, lo, hi, g, dev):
    """B whole numbers from hi down towards lo in even steps, in shuffled order."""
    steps = hi - torch.arange(B, device=dev) * (hi - lo) // max(B - 1, 1)
    return steps[torch.randperm(B, generator=g, device=dev)].to(torch.int32)


def _cache(case, n_pages, g, dev):
    """A filled cache: (k, v, k_exp, v_exp), values of about unit size."""
    fmt, shape = case["fmt"], (n_pages, case["hk"], case["page"], case["d"])
    held = []
    for _ in range(2):
        x = torch.empty(shape, dtype=torch.float16, device=dev).normal_(0, 100.0 if fmt == "e4m3" else 32.0, generator=g)
        x = x.clamp_(-LARGEST[fmt], LARGEST[fmt])
        held.append((x if fmt == "e4m3" else x.round_()).to(FORMATS[fmt]))
        del x
    mid = -7 if fmt == "e4m3" else -5
    for _ in range(2):
        held.append(torch.randint(mid - 1, mid + 2, (n_pages, case["hk"], case["page"] // case["block"]), generator=g,
                                  device=dev).to(torch.int8))
    return held


def _trees(count, nodes, g, dev):
    """Packed mask rows: node j of each request hangs from one of the nodes before it or from the context."""
    B = count.numel()
    pick = torch.rand(B, nodes, generator=g, device=dev).cpu()
    bits = torch.zeros(B, nodes, nodes, dtype=torch.bool)
    for j in range(nodes):
        parent = (pick[:, j] * (j + 1)).long() - 1
        bits[:, j] = torch.where((parent >= 0)[:, None], bits[torch.arange(B), parent.clamp(min=0)], False)
        bits[:, j, j] = True
    words = -(-nodes // 64)
    wide = torch.zeros(B, nodes, words * 64, dtype=torch.bool)
    wide[:, :, :nodes] = bits
    packed = (wide.view(B, nodes, words, 64).long() << torch.arange(64, dtype=torch.int64)).sum(-1).to(dev)
    return packed[torch.arange(nodes, device=dev)[None] < count[:, None]].contiguous()


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    s = {"case": case}
    op, B, ctx, page = case["op"], case["B"], case["ctx"], case["page"]
    if op in ("store", "attend", "keep"):
        new = {"store": case.get("n"), "attend": case.get("nodes"), "keep": case.get("nodes")}[op]
        per = -(-(ctx + new) // page)
        table = torch.randperm(B * per, generator=g, device=dev).to(torch.int32).view(B, per)
        if op == "keep":
            s["caches"] = [_cache(case, B * per, g, dev) for _ in range(case["layers"])]
            s["page_table"] = table
            s["context"] = torch.randint(0, ctx + 1, (B,), dtype=torch.int32, device=dev, generator=g)
            s["kept"] = torch.randint(0, case["path"] + 1, (B,), dtype=torch.int32, device=dev, generator=g)
            order = torch.rand(B, new, device=dev, generator=g).argsort(1)[:, :case["path"]]
            s["path"] = order.sort(1).values.to(torch.int32).contiguous()
            return s
        s["cache"] = _cache(case, B * per, g, dev)
        dt = DTYPES[case["dtype"]]
        if op == "store":
            context = torch.randint(0, ctx + 1, (B,), dtype=torch.int32, device=dev, generator=g)
            count = _spread(B, (new + 1) // 2, new, g, dev) if case["ragged"] else torch.full_like(context, new)
            end = count.cumsum(0)
            T = int(end[-1])
            seq = torch.repeat_interleave(torch.arange(B, device=dev), count.long())
            at = context[seq].long() + torch.arange(T, device=dev) - (end - count)[seq]
            s["cache_rows"] = (table[seq, at // page].long() * page + at % page).to(torch.int32)
            # keys and values as slices of fused rows; tokens and channels of different sizes
            hk, d = case["hk"], case["d"]
            size = torch.exp(torch.empty(T, 1, device=dev).normal_(0, 0.5, generator=g))
            size = size * torch.exp(torch.empty(1, 3 * hk * d, device=dev).normal_(0, 0.5, generator=g))
            s["rows"] = (torch.empty(T, 3 * hk * d, device=dev).normal_(0, 1, generator=g) * size).to(dt)
            return s
        hq, d = case["hq"], case["d"]
        if case["ragged"]:
            s["context"], count = _spread(B, ctx // 32, ctx, g, dev), _spread(B, (new + 1) // 2, new, g, dev)
        else:
            s["context"] = torch.full((B,), ctx, dtype=torch.int32, device=dev)
            count = torch.full((B,), new, dtype=torch.int32, device=dev)
        s["page_table"] = table
        s["q_start"] = torch.cat([count.new_zeros(1), count.cumsum(0).to(torch.int32)])
        T = int(s["q_start"][-1])
        s["q"] = torch.empty(T, hq * d, dtype=dt, device=dev).normal_(0.0, 1.5, generator=g)  # some keys stand out
        s["out"] = torch.empty(T, hq * d, dtype=dt, device=dev)
        s["mask"] = _trees(count, new, g, dev) if case["tree"] else None
        return s
    # fork, compact: B sequences of different lengths and a pool with room
    lengths = _spread(B, ctx // 2, ctx, g, dev) if op == "fork" else torch.randint(
        1, ctx + 1, (B,), dtype=torch.int32, device=dev, generator=g)
    per = -(-ctx // page)
    held = -(-lengths.long() // page)
    n_pages = B * per + B
    order = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32)[:B * per].view(B, per)
    table = torch.where(torch.arange(per, device=dev)[None] < held[:, None], order, -1)
    refs = torch.zeros(n_pages, dtype=torch.int32, device=dev)
    refs[table[table >= 0].long()] = 1
    s.update(table_at_start=table, refs_at_start=refs, table=table.clone(), refs=refs.clone(), lengths=lengths)
    s["caches"] = [_cache(case, n_pages, g, dev) for _ in range(case["layers"])]
    if op == "fork":
        # four beams a request: each goes on from one of the request's beams
        beams = min(4, B)
        s["parents"] = (torch.arange(B, device=dev) // beams * beams + torch.randint(
            0, beams, (B,), device=dev, generator=g)).clamp(max=B - 1).to(torch.int32)
        s["rows"] = torch.arange(B, dtype=torch.int32, device=dev)
        s["fork_lengths"] = lengths[s["parents"].long()].contiguous()
        s["new_table"] = torch.empty_like(table)
    else:
        s["done"] = torch.randperm(B, generator=g, device=dev)[:B // 2].to(torch.int32)
    return s


# ---- one pass ---------------------------------------------------------------

def _scaled(x, e):
    """x 2^e, exactly, for whole numbers e (below LOW: of LOW, where a byte's numbers are 0)."""
    return x * ((e.int().clamp(min=LOW) + 127) << 23).view(torch.float32)


def _rounded(x, fmt):
    """fp32 numbers to bytes: ties to even, the largest beyond it."""
    x = x.clamp(-LARGEST[fmt], LARGEST[fmt])
    return (x if fmt == "e4m3" else x.round()).to(FORMATS[fmt])


def _exponent(most, fmt):
    """The least e from LOW to TOP with most <= LARGEST 2^e."""
    part, e = torch.frexp(most)                      # most = part 2^e, part in [0.5, 1)
    top, up = math.frexp(LARGEST[fmt])
    e = torch.where(part <= top, e - up, e - up + 1)
    return torch.where(most > 0, e, LOW).clamp(LOW, TOP[fmt])


def _place(held, exp, x, need, row, case):
    """Rows x [n, hk, d] (fp32) into the flat rows `row` of one of the cache's tensors, in whose blocks the exponents
    become no smaller than need [n, hk]; rows before the first new one of a block live on."""
    fmt, page, block, hk = case["fmt"], case["page"], case["block"], case["hk"]
    blocks = held.shape[0] * (page // block)
    of = row // block
    old = exp.permute(0, 2, 1).reshape(blocks, hk).int().clamp(LOW, TOP[fmt])
    got = torch.full_like(old, LOW - 1).scatter_reduce_(0, of[:, None].expand(-1, hk), need.int(), "amax")
    first = torch.full((blocks,), block, device=row.device).scatter_reduce_(0, of, row % block, "amin")
    touched = first < block
    e = torch.where((first > 0)[:, None], torch.maximum(got, old), got)
    e = torch.where(touched[:, None], e, old)
    lives = torch.arange(block, device=row.device)[None] < torch.where(touched, first, 0)[:, None]      # [blocks, block]
    lower = torch.where(lives[:, None], (old - e)[..., None], 0)                                        # [blocks, hk, block]
    lower = lower.view(-1, page // block, hk, block).permute(0, 2, 1, 3).reshape(-1, hk, page, 1)
    held.copy_(_rounded(_scaled(held.float(), lower), fmt))
    exp.copy_(torch.where(touched[:, None], e, exp.permute(0, 2, 1).reshape(blocks, hk).int())
              .view(-1, page // block, hk).permute(0, 2, 1))
    new = _rounded(_scaled(x, -e[of][..., None]), fmt)
    held.view(torch.uint8)[row // page, :, row % page] = new.view(torch.uint8)


def _plain_store(s, case):
    hk, d = case["hk"], case["d"]
    row = s["cache_rows"].long()
    rows = s["rows"].float().view(-1, 3, hk, d)
    for i in (0, 1):
        x = rows[:, 1 + i]
        _place(s["cache"][i], s["cache"][2 + i], x, _exponent(x.abs().amax(-1), case["fmt"]), row, case)
    return s["cache"]


def _values(held, exp, pages, place, case):
    """fp32 rows [.., hk, d] of flat positions (pages, place)."""
    e = exp[pages, :, place // case["block"]].int()
    return _scaled(held.view(torch.uint8)[pages, :, place].view(held.dtype).float(), e[..., None])


def _plain_attend(s, case):
    B, n, hq, hk, d, page = (case[k] for k in ("B", "nodes", "hq", "hk", "d", "page"))
    dev, start, context = s["q"].device, s["q_start"].long(), s["context"].long()
    count = start[1:] - start[:-1]
    there = torch.arange(n, device=dev)[None] < count[:, None]                       # [B, n]
    row = (start[:-1, None] + torch.arange(n, device=dev)[None]).clamp(max=max(s["q"].shape[0] - 1, 0))
    q = s["q"].float()[row].view(B, n, hk, hq // hk, d).permute(0, 2, 1, 3, 4).reshape(B, hk, n * (hq // hk), d)
    at = torch.arange(case["ctx"] + n, device=dev)                                   # every position a request may have
    pages, place = s["page_table"].long()[:, at // page], (at % page).expand(B, -1)
    held_k, held_v, k_exp, v_exp = s["cache"]
    k = _values(held_k, k_exp, pages, place, case).permute(0, 2, 3, 1).contiguous()  # [B, hk, d, L]
    scores = torch.matmul(q, k).view(B, hk, n, hq // hk, -1) * d ** -0.5
    del k
    node = at[None] - context[:, None]                                               # [B, L]
    drafted = (node >= 0) & (node < count[:, None])
    if s["mask"] is None:
        sees = node[:, None] <= torch.arange(n, device=dev)[None, :, None]
    else:
        bits = s["mask"][row]                                                        # [B, n, words]
        word = (node.clamp(min=0) // 64).clamp(max=bits.shape[2] - 1)
        picked = bits.gather(2, word[:, None].expand(B, n, -1))
        sees = (picked >> (node.clamp(min=0) % 64)[:, None] & 1).bool()
    sees = (node < 0)[:, None] | (drafted[:, None] & sees)
    scores.masked_fill_(~sees[:, None, :, None], -math.inf)
    weight = torch.exp(scores - scores.amax(-1, keepdim=True).clamp(min=-1e30))
    del scores
    total = weight.sum(-1, keepdim=True)
    v = _values(held_v, v_exp, pages, place, case).permute(0, 2, 1, 3).contiguous()  # [B, hk, L, d]
    o = torch.matmul(weight.view(B, hk, n * (hq // hk), -1), v).view(B, hk, n, hq // hk, d) / total.clamp(min=1e-30)
    o = o.permute(0, 2, 1, 3, 4).reshape(B, n, hq * d)
    s["out"].copy_(o[there])
    return s["out"]


def _plain_keep(s, case):
    B, page = case["B"], case["page"]
    step = torch.arange(case["path"], device=s["path"].device)
    kept = (step[None] < s["kept"][:, None]).flatten()
    to = (s["context"].long()[:, None] + step).flatten()[kept]
    of = (s["context"].long()[:, None] + s["path"].long()).flatten()[kept]
    seq = torch.arange(B, device=to.device)[:, None].expand(B, case["path"]).flatten()[kept]
    table = s["page_table"].long()
    to_row, of_page, of_place = table[seq, to // page] * page + to % page, table[seq, of // page], of % page
    for layer in s["caches"]:
        for held, exp in ((layer[0], layer[2]), (layer[1], layer[3])):
            x = _values(held, exp, of_page, of_place, case)
            _place(held, exp, x, exp[of_page, :, of_place // case["block"]], to_row, case)
    return s["caches"]


def _plain_fork(s, case):
    page, refs, table = case["page"], s["refs"].copy_(s["refs_at_start"]), s["table"].copy_(s["table_at_start"])
    n = s["fork_lengths"].long()
    full, column = n // page, torch.arange(table.shape[1], device=n.device)[None]
    row = table[s["parents"].long()]
    shared = column < full[:, None]
    refs.index_add_(0, row.clamp(min=0).flatten().long(), shared.flatten().int())
    # the i-th fork with a partly filled page takes the i-th free page
    part = n % page > 0
    free = torch.argsort((refs > 0).to(torch.int8), stable=True)
    page_of = free[(part.cumsum(0) - 1).clamp(min=0)]
    new = torch.where(shared, row, torch.where((column == full[:, None]) & part[:, None], page_of[:, None].int(), -1))
    s["new_table"].copy_(new)
    refs.index_add_(0, page_of, part.int())
    source = row.gather(1, full.clamp(max=table.shape[1] - 1)[:, None])[:, 0].long()
    source, target = source[part], page_of[part]
    for layer in s["caches"]:
        for t in layer:
            t.view(torch.uint8)[target] = t.view(torch.uint8)[source]
    # the beams that the step went on from are done
    refs.index_add_(0, table.clamp(min=0).flatten().long(), -(table >= 0).flatten().int())
    table.fill_(-1)
    return s["new_table"], refs, table, s["caches"]


def _plain_compact(s, case):
    refs, table = s["refs"].copy_(s["refs_at_start"]), s["table"].copy_(s["table_at_start"])
    done = s["done"].long()
    gone = table[done]
    refs.index_add_(0, gone.clamp(min=0).flatten().long(), -(gone >= 0).flatten().int())
    table[done] = -1
    live = refs > 0
    n_live = live.sum()
    number = torch.arange(refs.numel(), device=refs.device)
    of, to = (live & (number >= n_live)).nonzero()[:, 0], (~live & (number < n_live)).nonzero()[:, 0]
    number[of] = to
    table.copy_(torch.where(table >= 0, number[table.clamp(min=0).long()].int(), table))
    refs[to] = refs[of]
    refs[of] = 0
    for layer in s["caches"]:
        for t in layer:
            t.view(torch.uint8)[to] = t.view(torch.uint8)[of]
    return n_live.to(torch.int32), refs, table, s["caches"]


def _own(s, case):
    import gemm_lora_shrink_amd as glsa
    op = case["op"]
    if op == "store":
        hk, d, rows = case["hk"], case["d"], s["rows"]
        glsa.store_quantized(rows[:, hk * d:2 * hk * d], rows[:, 2 * hk * d:], s["cache"], s["cache_rows"])
        return s["cache"]
    if op == "keep":
        glsa.keep_path_quantized(s["caches"], s["page_table"], s["context"], s["path"], s["kept"])
        return s["caches"]
    if op == "attend":
        if "workspace" not in s:  # a server keeps it
            s["workspace"] = glsa.alloc_quantized_workspace(
                case["B"], s["q"].shape[0], case["nodes"], case["ctx"], case["hq"], case["hk"], case["d"], s["q"].device)
        return glsa.tree_attention_quantized(s["q"], s["cache"], s["page_table"], s["context"], s["q_start"],
                                             max_nodes=case["nodes"], max_context=case["ctx"], mask=s["mask"],
                                             out=s["out"], workspace=s["workspace"])
    refs, table, page = s["refs"].copy_(s["refs_at_start"]), s["table"].copy_(s["table_at_start"]), case["page"]
    if "tensors" not in s:  # a server keeps both
        s["tensors"] = glsa.PagedTensors(t for layer in s["caches"] for t in layer)
        s["workspace"] = glsa.alloc_pages_workspace(refs.numel(), case["B"], refs.device)
    if op == "fork":
        glsa.fork_sequences(refs, table, s["parents"], s["rows"], s["fork_lengths"], page_size=page, tensors=s["tensors"],
                            out_table=s["new_table"], workspace=s["workspace"])
        glsa.release_pages(refs, table)
        return s["new_table"], refs, table, s["caches"]
    glsa.release_pages(refs, table, s["done"])
    n_live = glsa.compact_pages(refs, table, tensors=s["tensors"], workspace=s["workspace"])
    return n_live, refs, table, s["caches"]


def run(state):
    case = state["case"]
    if own:
        return _own(state, case)
    return {"store": _plain_store, "attend": _plain_attend, "keep": _plain_keep, "fork": _plain_fork,
            "compact": _plain_compact}[case["op"]](state, case)


# ---- what a pass cannot do without ------------------------------------------

def _mean_lengths(case):
    """Means over the requests of prepare(): tokens before the nodes, and nodes."""
    if not case["ragged"] or case["B"] == 1:
        return case["ctx"], case["nodes"]
    return (case["ctx"] // 32 + case["ctx"]) / 2, ((case["nodes"] + 1) // 2 + case["nodes"]) / 2


def work(case):
    op, B, hk, d, page = (case[k] for k in ("op", "B", "hk", "d", "page"))
    row = 2 * hk * d                    # bytes of a token's keys and values
    of_block = 2 * hk / case["block"]   # bytes of exponents a token
    if op == "store":
        T = B * (((case["n"] + 1) // 2 + case["n"]) / 2 if case["ragged"] and B > 1 else case["n"])
        return {"bytes": T * (row * BYTES[case["dtype"]] + row + 4 + of_block), "flops": 3 * T * row}
    if op == "keep":
        return {"bytes": case["layers"] * B * (case["path"] / 2) * 2 * (row + of_block) + 4 * B * (case["path"] + 2),
                "flops": 0}
    if op == "attend":
        ctx, n = _mean_lengths(case)
        hq, e = case["hq"], BYTES[case["dtype"]]
        return {"bytes": B * ((ctx + n) * (row + of_block) + 2 * n * hq * d * e + 4 * (ctx + n) / page
                              + (8 * n * -(-case["nodes"] // 64) if case["tree"] else 0)),
                "flops": 4 * B * n * hq * d * (ctx + n / 2)}
    of_page, per = case["layers"] * page * (row + of_block), -(-case["ctx"] // page)
    if op == "fork":
        return {"bytes": B * (2 * of_page + 2 * 4 * per * 2 + 2 * 4 * per), "flops": 0}
    # half of the pages are live at most, spread over the pool: about half of those lie past the number of live ones
    live = B / 2 * (case["ctx"] / 2 / page + 0.5)
    pool = B * per + B
    return {"bytes": 2 * of_page * live * max(0.0, 1 - live / pool) + 2 * 4 * pool + 2 * 4 * B * per, "flops": 0}


# ---- the same from the definition, in 64 bits --------------------------------

def _nearest(x, fmt):
    """64-bit numbers to the nearest that a byte holds, ties to even."""
    if fmt == "int8":
        return torch.round(x).clamp(-127, 127)
    power = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6)))
    power = power - (torch.pow(2.0, power) > x.abs().clamp(min=2.0 ** -6)).double()  # where log2 rounded up
    step = torch.pow(2.0, power - 3)
    return (torch.round(x / step) * step).clamp(-448, 448)


def _least(most, fmt):
    if most == 0:
        return LOW
    e = LOW
    guess = math.ceil(math.log2(most / LARGEST[fmt])) - 1
    e = max(e, guess)
    while e < TOP[fmt] and most > math.ldexp(LARGEST[fmt], e):
        e += 1
    return min(e, TOP[fmt])


def _exact_store(s, case):
    fmt, page, block, hk, d = (case[k] for k in ("fmt", "page", "block", "hk", "d"))
    rows = s["rows"].double().view(-1, 3, hk, d).cpu()
    blocks = {}
    for t, r in enumerate(s["cache_rows"].tolist()):
        blocks.setdefault(r // block, []).append((r % block, t))
    held = [t.double().cpu() for t in s["cache"][:2]]
    for i in (0, 1):
        exps = s["cache"][2 + i].cpu()
        for of, tokens in blocks.items():
            p, j = divmod(of, page // block)
            first = min(r for r, _ in tokens)
            x = rows[[t for _, t in tokens], 1 + i]                                   # [m, hk, d]
            old = exps[p, :, j].tolist()
            e = [_least(v, fmt) for v in x.abs().amax((0, 2)).tolist()]
            if first:
                e = [max(a, b) for a, b in zip(e, old)]
                down = torch.tensor([2.0 ** (b - a) for a, b in zip(e, old)], dtype=torch.float64)[:, None, None]
                part = held[i][p, :, j * block:j * block + first]
                part.copy_(_nearest(part * down, fmt))
            grid = torch.tensor([2.0 ** -a for a in e], dtype=torch.float64)[:, None]
            for (r, _), row in zip(tokens, _nearest(x * grid, fmt)):
                held[i][p, :, j * block + r] = row
    return held + [None, None] if fmt == "e4m3" else None


def exact(case, seed):
    if case["op"] not in ("store", "attend"):
        return None  # bytes that are moved
    s = prepare(case, seed)
    hk, d, page, block = (case[k] for k in ("hk", "d", "page", "block"))
    if case["op"] == "store":
        return _exact_store(s, case) if s["cache_rows"].numel() <= 10000 else None
    hq, group = case["hq"], case["hq"] // case["hk"]
    start, context = s["q_start"].tolist(), s["context"].tolist()
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    for b in range(case["B"]):
        n, c = start[b + 1] - start[b], context[b]
        pages = s["page_table"][b, :-(-(c + n) // page)].long()
        scale = [torch.pow(2.0, t[pages].double()).repeat_interleave(block, 2)[..., None] for t in s["cache"][2:]]
        held = [t.view(torch.uint8)[pages].view(t.dtype).double() for t in s["cache"][:2]]
        k, v = ((x * e).transpose(0, 1).reshape(hk, -1, d)[:, :c + n] for x, e in zip(held, scale))
        q = s["q"][start[b]:start[b + 1]].double().view(n, hk, group, d).permute(1, 2, 0, 3).reshape(hk, group * n, d)
        score = torch.bmm(q, k.transpose(1, 2).contiguous()).view(hk, group, n, c + n) / math.sqrt(d)
        if s["mask"] is None:
            seen = torch.ones(n, n, dtype=torch.bool, device=q.device).tril()
        else:
            words = s["mask"][start[b]:start[b + 1]]
            seen = (words[:, :, None] >> torch.arange(64, device=q.device) & 1).bool().flatten(1)[:, :n]
        score[..., c:].masked_fill_(~seen, -math.inf)
        o = torch.bmm(torch.softmax(score, -1).view(hk, group * n, c + n), v.contiguous())
        out[start[b]:start[b + 1]] = o.view(hk, group, n, d).permute(2, 0, 1, 3).reshape(n, hq * d)
    return out
