"""What is timed of the operators that follow the adapters' q/k/v projection.

A batch's rows [q | k | v] leave the LoRA update, are given their positions (with or without a norm of each head) and
put into a paged cache, a tree of drafted tokens attends over that cache, and the accepted path is kept.  Head shapes are
those of the workloads of this repository (32 query and 8 key/value heads of 128, 256 and 8192 tokens) or generic.

`own` false: the operators in elementary torch operations.  `own` true: the library's entry points.
"""

import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}


# ---- cases ------------------------------------------------------------------

def listed():
    return [
        # the table of a model of 131072 positions, made when a server starts
        dict(name="table_131072", op="table", n=131072, rot=128, base=500000.0, scaling="llama3", factor=8.0,
             original=8192),
        # one decode step of 64 requests, 32 + 8 heads of 128
        dict(name="rotary_decode_64", op="rotary", T=64, hq=32, hk=8, d=128, rot=128, layout="half", dtype="bf16",
             page=16),
        # a prompt through a model with 16 heads of 256 of which 64 elements are rotated, pairs side by side; odd length
        dict(name="rotary_part_4097", op="rotary", T=4097, hq=16, hk=16, d=256, rot=64, layout="interleaved",
             dtype="f16", page=32),
        # one decode step of 256 requests with normed heads
        dict(name="norm_decode_256", op="norm", T=256, hq=32, hk=8, d=128, rot=128, layout="half", dtype="f16",
             page=16),
        # 16 prompts of 512 tokens with normed heads
        dict(name="norm_prompt_8192", op="norm", T=8192, hq=32, hk=8, d=128, rot=128, layout="half", dtype="bf16",
             page=16),
        # the smallest call: one request, one token, a short context
        dict(name="attend_one_100", op="attend", B=1, nodes=1, ctx=100, ragged=False, tree=False, hq=32, hk=8, d=128,
             dtype="bf16", page=16),
        # a full decode batch, contexts of all lengths
        dict(name="attend_decode_256", op="attend", B=256, nodes=1, ctx=4096, ragged=True, tree=False, hq=32, hk=8,
             d=128, dtype="bf16", page=16),
        # one request with a long context and a wide tree
        dict(name="attend_tree64_32768", op="attend", B=1, nodes=64, ctx=32768, ragged=False, tree=True, hq=32, hk=8,
             d=128, dtype="bf16", page=64),
        # 16 requests, trees and contexts of different sizes, pages that are no power of two
        dict(name="attend_ragged_16", op="attend", B=16, nodes=45, ctx=8192, ragged=True, tree=True, hq=32, hk=8,
             d=128, dtype="f16", page=24),
        # fp32, a head for each query head, chains of drafted tokens
        dict(name="attend_chain_f32", op="attend", B=8, nodes=7, ctx=1500, ragged=True, tree=False, hq=16, hk=16, d=64,
             dtype="f32", page=16),
        # the accepted path of one request, four layers
        dict(name="keep_1", op="keep", B=1, layers=4, path=4, nodes=16, ctx=500, hk=8, d=128, dtype="bf16", page=16),
        # the accepted paths of a batch, 16 layers at once
        dict(name="keep_64", op="keep", B=64, layers=16, path=8, nodes=64, ctx=300, hk=8, d=128, dtype="bf16", page=16),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["table", "rotary", "rotary", "norm", "norm", "attend", "attend", "attend", "attend", "keep"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op == "table":
        return dict(op=op, n=_log(rng, 1000, 131072), rot=rng.choice([20, 32, 64, 80, 128]),
                    base=rng.choice([10000.0, 500000.0]), scaling=rng.choice(["none", "linear", "ntk", "llama3", "yarn"]),
                    factor=rng.choice([2.0, 4.0, 8.0]), original=rng.choice([4096, 8192]))
    hk = rng.choice([1, 2, 4, 8, 16])
    hq = hk * rng.choice([g for g in (1, 2, 4, 8) if hk * g <= 32])
    d = rng.choice([64, 80, 128, 128, 256])
    page = rng.choice([8, 16, 24, 32, 64, 128])
    if op in ("rotary", "norm"):
        return dict(op=op, T=_log(rng, 1, 8192), hq=hq, hk=hk, d=d, rot=rng.choice([d, d, d // 2, d // 4]),
                    layout=rng.choice(["half", "interleaved"]), dtype=dtype, page=page)
    if op == "attend":
        B = _log(rng, 1, 256)
        nodes = _log(rng, 1, 128)
        ctx = _log(rng, 16, 32768)
        # no more keys in all, and no more products, than the largest listed cases have
        ctx = max(1, min(ctx, (1 << 29) // (B * hk * d), (1 << 33) // (B * nodes * hq * d)))
        return dict(op=op, B=B, nodes=nodes, ctx=ctx, ragged=rng.random() < 0.6, tree=rng.random() < 0.6, hq=hq, hk=hk,
                    d=d, dtype=dtype, page=page)
    nodes = _log(rng, 1, 64)
    return dict(op=op, B=_log(rng, 1, 64), layers=rng.choice([1, 2, 5, 16]), path=_log(rng, 1, min(nodes, 12)),
                nodes=nodes, ctx=_log(rng, 1, 300), hk=min(hk, 8), d=min(d, 128), dtype=dtype, page=page)


# ---- inputs -----------------------------------------------------------------

def _pages(case, B, length, g, dev):
    """A page table of B requests of up to `length` tokens over pages in shuffled order."""
    per = -(-length // case["page"])
    table = torch.randperm(B * per, generator=g, device=dev).to(torch.int32).view(B, per)
    return table, B * per


def _spread(B, lo, hi, g, dev):
    """B whole numbers from hi down towards lo in even steps, in shuffled order."""
    steps = hi - torch.arange(B, device=dev) * (hi - lo) // max(B - 1, 1)
    return steps[torch.randperm(B, generator=g, device=dev)].to(torch.int32)


def _frequencies(case):
    """The rotation's frequencies by the formulas of the scalings, as Python floats, and the factor of cos and sin."""
    rot, base, kind, f, orig = (case[k] for k in ("rot", "base", "scaling", "factor", "original"))
    plain = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    if kind == "linear":
        return [v / f for v in plain], 1.0
    if kind == "ntk":
        grown = base * f ** (rot / (rot - 2.0))
        return [grown ** (-2.0 * i / rot) for i in range(rot // 2)], 1.0
    if kind == "llama3":
        got = []
        for v in plain:
            turns = orig * v / (2 * math.pi)  # in the original context; slow below 1, fast above 4
            smooth = min(1.0, max(0.0, (turns - 1.0) / (4.0 - 1.0)))
            got.append((1 - smooth) * v / f + smooth * v)
        return got, 1.0
    if kind == "yarn":
        def place(turns):
            return rot * math.log(orig / (turns * 2 * math.pi)) / (2 * math.log(base))
        lo, hi = max(math.floor(place(32.0)), 0), min(math.ceil(place(1.0)), rot - 1)
        keep = [1 - min(1.0, max(0.0, (i - lo) / max(hi - lo, 1e-3))) for i in range(rot // 2)]
        return [v / f * (1 - k) + v * k for v, k in zip(plain, keep)], 0.1 * math.log(f) + 1.0
    return plain, 1.0


def _positions_table(n, rot, dev):
    """cos | sin of the unscaled rotation, which a server keeps from its start."""
    freq = 10000.0 ** (torch.arange(rot // 2, dtype=torch.float64, device=dev) * (-2.0 / rot))
    angle = torch.arange(n, dtype=torch.float64, device=dev)[:, None] * freq
    return torch.cat([torch.cos(angle), torch.sin(angle)], 1).float()


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    s = {"case": case}
    op = case["op"]
    if op == "table":
        # a model's base is its own: another seed is another model
        s["case"] = dict(case, base=case["base"] * (1.0 + (seed % 1009) / 1009.0))
        s["out"] = torch.empty(case["n"], case["rot"], device=dev)
        return s
    dt = DTYPES[case["dtype"]]

    def normal(*shape, scale=1.0):
        return torch.empty(shape, dtype=dt, device=dev).normal_(0.0, scale, generator=g)

    hk, d = case["hk"], case["d"]
    if op in ("rotary", "norm"):
        T, hq = case["T"], case["hq"]
        s["rows"] = normal(T, (hq + 2 * hk) * d)
        n_pos = 8192
        s["table"] = _positions_table(n_pos, case["rot"], dev)
        s["positions"] = torch.randint(0, n_pos, (T,), dtype=torch.int32, device=dev, generator=g)
        pages = -(-(T + 2 * case["page"]) // case["page"])
        s["k_cache"], s["v_cache"] = normal(pages, hk, case["page"], d), normal(pages, hk, case["page"], d)
        s["cache_rows"] = torch.randperm(pages * case["page"], generator=g, device=dev)[:T].to(torch.int32)
        s["q_out"] = torch.empty(T, hq * d, dtype=dt, device=dev)
        if op == "norm":
            s["q_weight"], s["k_weight"] = normal(d, scale=0.2) + 1, normal(d, scale=0.2) + 1
        return s
    B, nodes, ctx = case["B"], case["nodes"], case["ctx"]
    s["page_table"], n_pages = _pages(case, B, ctx + nodes, g, dev)
    if op == "keep":
        s["caches"] = [(normal(n_pages, hk, case["page"], d), normal(n_pages, hk, case["page"], d))
                       for _ in range(case["layers"])]
        s["context"] = torch.randint(0, ctx + 1, (B,), dtype=torch.int32, device=dev, generator=g)
        s["kept"] = torch.randint(0, case["path"] + 1, (B,), dtype=torch.int32, device=dev, generator=g)
        order = torch.rand(B, nodes, device=dev, generator=g).argsort(1)[:, :case["path"]]
        s["path"] = order.sort(1).values.to(torch.int32).contiguous()
        return s
    hq = case["hq"]
    s["k_cache"], s["v_cache"] = normal(n_pages, hk, case["page"], d), normal(n_pages, hk, case["page"], d)
    if case["ragged"]:
        context = _spread(B, ctx // 32, ctx, g, dev)
        count = _spread(B, (nodes + 1) // 2, nodes, g, dev)
    else:
        context = torch.full((B,), ctx, dtype=torch.int32, device=dev)
        count = torch.full((B,), nodes, dtype=torch.int32, device=dev)
    s["context"] = context
    s["q_start"] = torch.cat([count.new_zeros(1), count.cumsum(0).to(torch.int32)])
    T = int(s["q_start"][-1])
    s["q"] = normal(T, hq * d, scale=1.5)  # scores of unit scale and more: some keys stand out
    s["out"] = torch.empty(T, hq * d, dtype=dt, device=dev)
    s["mask"] = None
    if case["tree"]:
        # node j hangs from one of the nodes before it or from the context; a row of bits holds a node's ancestors
        draw_ = torch.rand(B, nodes, generator=g, device=dev).cpu()
        bits = torch.zeros(B, nodes, nodes, dtype=torch.bool)
        for j in range(nodes):
            parent = (draw_[:, j] * (j + 1)).long() - 1
            bits[:, j] = torch.where((parent >= 0)[:, None], bits[torch.arange(B), parent.clamp(min=0)], False)
            bits[:, j, j] = True
        words = -(-nodes // 64)
        wide = torch.zeros(B, nodes, words * 64, dtype=torch.bool)
        wide[:, :, :nodes] = bits
        shifts = torch.arange(64, dtype=torch.int64)
        packed = (wide.view(B, nodes, words, 64).long() << shifts).sum(-1).to(dev)
        there = torch.arange(nodes, device=dev)[None] < count[:, None]
        s["mask"] = packed[there].contiguous()
    return s


# ---- one pass ---------------------------------------------------------------

def _rotated(x, cos, sin, layout):
    """x [T, h, d] in fp32 with its first 2 * cos.size(1) elements rotated."""
    half = cos.shape[1]
    cos, sin, part = cos[:, None], sin[:, None], x[..., :2 * half]
    if layout == "half":
        a, b = part[..., :half], part[..., half:]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = part[..., 0::2], part[..., 1::2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([turned, x[..., 2 * half:]], -1)


def _plain_rows(s, case):
    T, hq, hk, d, half = case["T"], case["hq"], case["hk"], case["d"], case["rot"] // 2
    rows = s["rows"].float().view(T, hq + 2 * hk, d)
    qk, v = rows[:, :hq + hk], rows[:, hq + hk:]
    if case["op"] == "norm":
        weight = torch.cat([s["q_weight"].float().expand(hq, d), s["k_weight"].float().expand(hk, d)])
        qk = qk * torch.rsqrt(qk.square().mean(-1, keepdim=True) + 1e-6) * weight
    at = s["table"][s["positions"].long()]
    turned = _rotated(qk, at[:, :half], at[:, half:], case["layout"])
    s["q_out"].copy_(turned[:, :hq].reshape(T, hq * d))
    row = s["cache_rows"].long()
    page, place = row // case["page"], row % case["page"]
    s["k_cache"][page, :, place] = turned[:, hq:].to(s["k_cache"].dtype)
    s["v_cache"][page, :, place] = v.to(s["v_cache"].dtype)
    return s["q_out"], s["k_cache"], s["v_cache"]


def _plain_attend(s, case):
    B, n, hq, hk, d, page = (case[k] for k in ("B", "nodes", "hq", "hk", "d", "page"))
    dev, start, context = s["q"].device, s["q_start"].long(), s["context"].long()
    count = start[1:] - start[:-1]
    there = torch.arange(n, device=dev)[None] < count[:, None]                       # [B, n]
    row = (start[:-1, None] + torch.arange(n, device=dev)[None]).clamp(max=max(s["q"].shape[0] - 1, 0))
    q = s["q"].float()[row].view(B, n, hk, hq // hk, d).permute(0, 2, 1, 3, 4).reshape(B, hk, n * (hq // hk), d)
    at = torch.arange(case["ctx"] + n, device=dev)                                   # every position a request may have
    pages, place = s["page_table"].long()[:, at // page], at % page
    k = s["k_cache"][pages, :, place].float().permute(0, 2, 3, 1).contiguous()       # [B, hk, d, L]
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
    v = s["v_cache"][pages, :, place].float().permute(0, 2, 1, 3).contiguous()       # [B, hk, L, d]
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
    to_page, of_page = table[seq, to // page], table[seq, of // page]
    for pair in s["caches"]:  # the layers
        for c in pair:
            c[to_page, :, to % page] = c[of_page, :, of % page]
    return s["caches"]


def _plain_table(case, out):
    freq, magnitude = _frequencies(case)
    angle = torch.arange(case["n"], dtype=torch.float64, device=out.device)[:, None] * torch.tensor(
        freq, dtype=torch.float64, device=out.device)
    return out.copy_(torch.cat([torch.cos(angle), torch.sin(angle)], 1) * magnitude)


def _own(s, case):
    import gemm_lora_shrink_amd as glsa
    op = case["op"]
    if op == "table":
        scaling = None if case["scaling"] == "none" else dict(type=case["scaling"], factor=case["factor"],
                                                              original_max_position=case["original"])
        return glsa.rope_table(case["n"], case["rot"], base=case["base"], scaling=scaling, out=s["out"])
    if op in ("rotary", "norm"):
        hq, hk, d, rows = case["hq"], case["hk"], case["d"], s["rows"]
        q, k, v = rows[:, :hq * d], rows[:, hq * d:(hq + hk) * d], rows[:, (hq + hk) * d:]
        more = dict(head_dim=d, layout=case["layout"], q_out=s["q_out"], v=v, k_cache=s["k_cache"],
                    v_cache=s["v_cache"], cache_rows=s["cache_rows"])
        if op == "rotary":
            glsa.rotary(q, k, s["positions"], s["table"], **more)
        else:
            glsa.qk_norm_rotary(q, k, s["q_weight"], s["k_weight"], s["positions"], s["table"], eps=1e-6, **more)
        return s["q_out"], s["k_cache"], s["v_cache"]
    if op == "keep":
        glsa.keep_path([k for k, _ in s["caches"]], [v for _, v in s["caches"]], s["page_table"], s["context"],
                       s["path"], s["kept"])
        return s["caches"]
    if "workspace" not in s:  # a server keeps it
        s["workspace"] = glsa.alloc_attention_workspace(
            case["B"], s["q"].shape[0], case["nodes"], case["ctx"], case["hq"], case["hk"], case["d"], s["q"].device)
    return glsa.tree_attention(s["q"], s["k_cache"], s["v_cache"], s["page_table"], s["context"], s["q_start"],
                               max_nodes=case["nodes"], max_context=case["ctx"], mask=s["mask"], out=s["out"],
                               workspace=s["workspace"])


def run(state):
    case = state["case"]
    if own:
        return _own(state, case)
    if case["op"] == "table":
        return _plain_table(case, state["out"])
    if case["op"] == "attend":
        return _plain_attend(state, case)
    return (_plain_keep if case["op"] == "keep" else _plain_rows)(state, case)


# ---- what a pass cannot do without ------------------------------------------

def _mean_lengths(case):
    """Means over the requests of prepare(): tokens before the nodes, and nodes."""
    if not case["ragged"] or case["B"] == 1:
        return case["ctx"], case["nodes"]
    return (case["ctx"] // 32 + case["ctx"]) / 2, ((case["nodes"] + 1) // 2 + case["nodes"]) / 2


def work(case):
    op = case["op"]
    if op == "table":
        return {"bytes": 4 * case["n"] * case["rot"], "flops": 20 * case["n"] * case["rot"]}
    e, hk, d = BYTES[case["dtype"]], case["hk"], case["d"]
    if op in ("rotary", "norm"):
        T, hq = case["T"], case["hq"]
        per = 2 * (hq + 2 * hk) * d * e + 4 * case["rot"] + 8
        return {"bytes": T * per, "flops": T * (hq + hk) * (3 * case["rot"] + (4 * d if op == "norm" else 0))}
    if op == "keep":
        return {"bytes": case["layers"] * case["B"] * (case["path"] / 2) * 4 * hk * d * e
                + 4 * case["B"] * (case["path"] + 2), "flops": 0}
    ctx, n = _mean_lengths(case)
    B, hq = case["B"], case["hq"]
    return {"bytes": B * (2 * (ctx + n) * hk * d * e + 2 * n * hq * d * e + 4 * (ctx + n) / case["page"]
                          + (8 * n * -(-case["nodes"] // 64) if case["tree"] else 0)),
            "flops": 4 * B * n * hq * d * (ctx + n / 2)}


# ---- the same from the definition, in 64 bits --------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    case, op = s["case"], case["op"]
    if op == "table":
        freq, magnitude = _frequencies(case)
        freq = torch.tensor(freq, dtype=torch.float64, device="cuda")
        turn = torch.polar(torch.full((), magnitude, dtype=torch.float64, device="cuda"),
                           torch.arange(case["n"], device="cuda").double().outer(freq))
        return torch.cat([turn.real, turn.imag], 1)
    if op == "keep":
        return None
    hk, d, page = case["hk"], case["d"], case["page"]
    if op in ("rotary", "norm"):
        T, hq, rot = case["T"], case["hq"], case["rot"]
        x = s["rows"].double().view(T, hq + 2 * hk, d)
        heads = x[:, :hq + hk]
        if op == "norm":
            heads = heads / (heads.pow(2).sum(-1, keepdim=True) / d + 1e-6).sqrt()
            heads = torch.cat([heads[:, :hq] * s["q_weight"].double(), heads[:, hq:] * s["k_weight"].double()], 1)
        pairs = torch.arange(rot, device=x.device)
        pairs = pairs.view(2, -1).t() if case["layout"] == "half" else pairs.view(-1, 2)  # [rot / 2, 2]
        at = s["table"].double()[s["positions"].long()]
        turn = torch.complex(at[:, :rot // 2], at[:, rot // 2:])[:, None]
        z = torch.complex(heads[..., pairs[:, 0]], heads[..., pairs[:, 1]]) * turn
        heads = heads.clone()
        heads[..., pairs[:, 0]], heads[..., pairs[:, 1]] = z.real, z.imag
        k, v = s["k_cache"].double(), s["v_cache"].double()
        for cache, new in ((k, heads[:, hq:]), (v, x[:, hq + hk:])):
            flat = cache.transpose(1, 2).reshape(-1, hk, d)
            flat[s["cache_rows"].long()] = new
            cache.copy_(flat.view(-1, page, hk, d).transpose(1, 2))
        return heads[:, :hq].reshape(T, hq * d), k, v
    hq, group = case["hq"], case["hq"] // case["hk"]
    start, context = s["q_start"].tolist(), s["context"].tolist()
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    for b in range(case["B"]):
        n, c = start[b + 1] - start[b], context[b]
        pages = s["page_table"][b, :-(-(c + n) // page)].long()
        k, v = (t[pages].transpose(0, 1).reshape(hk, -1, d)[:, :c + n].double() for t in (s["k_cache"], s["v_cache"]))
        q = s["q"][start[b]:start[b + 1]].double().view(n, hk, group, d).permute(1, 2, 0, 3).reshape(hk, group * n, d)
        score = torch.bmm(q, k.transpose(1, 2).contiguous()).view(hk, group, n, c + n) / math.sqrt(d)
        if s["mask"] is None:
            seen = torch.ones(n, n, dtype=torch.bool, device=q.device).tril()
        else:
            words = s["mask"][start[b]:start[b + 1]]
            seen = (words[:, :, None] >> torch.arange(64, device=q.device) & 1).bool().flatten(1)[:, :n]
        score[..., c:].masked_fill_(~seen, -math.inf)
        o = torch.bmm(torch.softmax(score, -1).view(hk, group * n, c + n), v)
        out[start[b]:start[b + 1]] = o.view(hk, group, n, d).permute(2, 0, 1, 3).reshape(n, hq * d)
    return out
