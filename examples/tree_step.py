"""A speculative decoding step of a batch with LoRA adapters, from the fused
q/k/v rows to the accepted tokens' place in the cache.

For each layer: the base projection, the adapters' part of it (shrink_expand),
rotary positions with the keys and values into the paged cache (rotary, or
qk_norm_rotary for a model with normed heads), attention of the drafted trees
(tree_attention) and the output projection.  The trees' masks, positions and
cache rows are made once for all layers (build_tree); when the draft is
verified the accepted path's rows move up to follow the context (keep_path).
The prompt goes through the same calls as a chain, and so does a plain decode
step, as a chain of one token.

    python examples/tree_step.py [--dtype bf16] [--norm]

prints how far the tree's accepted rows are from the same tokens decoded one by
one."""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gemm_lora_shrink_amd as glsa  # noqa: E402

HIDDEN, HQ, HK, D, RANK, SLOTS, LAYERS, PAGE = 256, 8, 2, 64, 16, 3, 2, 16
WIDTH = (HQ + 2 * HK) * D


class Layers:
    """Random weights and an empty paged cache for `B` sequences of `tokens`."""

    def __init__(self, B, tokens, dtype, norm, seed=0):
        g = torch.Generator("cuda").manual_seed(seed)

        def rand(*shape, scale):
            return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)

        outs = (HQ * D, HK * D, HK * D)
        self.norm = [(rand(D, scale=0.1) + 1, rand(D, scale=0.1) + 1) if norm else None for _ in range(LAYERS)]
        self.w = [rand(WIDTH, HIDDEN, scale=HIDDEN ** -0.5) for _ in range(LAYERS)]
        self.wo = [rand(HIDDEN, HQ * D, scale=(HQ * D) ** -0.5) for _ in range(LAYERS)]
        self.a = [[rand(SLOTS, RANK, HIDDEN, scale=HIDDEN ** -0.5) for _ in outs] for _ in range(LAYERS)]
        self.b = [[rand(SLOTS, n, RANK, scale=RANK ** -0.5) for n in outs] for _ in range(LAYERS)]
        self.scale = torch.full((SLOTS,), 0.5, device="cuda")
        self.table = glsa.rope_table(tokens, D, base=10000.0)
        pages = -(-tokens // PAGE)
        self.page_table = torch.randperm(B * pages, generator=g, device="cuda").to(torch.int32).view(B, pages)
        self.k = [torch.zeros(B * pages, HK, PAGE, D, dtype=dtype, device="cuda") for _ in range(LAYERS)]
        self.v = [torch.zeros_like(k) for k in self.k]
        self.max_context = pages * PAGE
        self.offsets = [0, HQ * D, (HQ + HK) * D]

    def step(self, h, slot, parents, counts, context):
        """Hidden rows of the step's tokens: h [T, HIDDEN], slot int32 [T] (-1: no
        adapter), counts new tokens of each sequence, parents as build_tree takes them."""
        T, most = h.size(0), max(counts)
        q_start = torch.tensor([0] + counts, dtype=torch.int32).cumsum(0).to(torch.int32).cuda()
        mask, pos, rows = glsa.build_tree(parents, q_start, context, max_nodes=most, n_tokens=T,
                                          page_table=self.page_table, n_pages=self.k[0].size(0), page_size=PAGE)
        seg = glsa.alloc_segments(T, SLOTS, "cuda")
        lora_ws = glsa.alloc_workspace(T, SLOTS, 3, RANK, "cuda")
        ws = glsa.alloc_attention_workspace(len(counts), T, most, self.max_context, HQ, HK, D, "cuda")
        for i in range(LAYERS):
            y = h @ self.w[i].t()
            glsa.shrink_expand(h, self.a[i], self.b[i], y, seg, self.offsets, workspace=lora_ws, scale=self.scale,
                               idx=slot if i == 0 else None)
            q, k, v = y[:, :HQ * D], y[:, HQ * D:(HQ + HK) * D], y[:, (HQ + HK) * D:]
            cached = dict(head_dim=D, v=v, k_cache=self.k[i], v_cache=self.v[i], cache_rows=rows)
            if self.norm[i]:
                glsa.qk_norm_rotary(q, k, *self.norm[i], pos, self.table, **cached)
            else:
                glsa.rotary(q, k, pos, self.table, **cached)
            o = glsa.tree_attention(q, self.k[i], self.v[i], self.page_table, context, q_start, max_nodes=most,
                                    max_context=self.max_context, mask=mask, workspace=ws)
            h = h + o @ self.wo[i].t()
        return h


def run(dtype=torch.bfloat16, norm=False):
    """(tree, one_by_one): the rows of the accepted nodes and of one token after
    them, from a verified tree and from the same tokens decoded one by one."""
    B, prompt = 3, [21, 40, 5]
    m = Layers(B, 96, dtype, norm)
    g = torch.Generator("cuda").manual_seed(1)

    def rows(n):
        return torch.randn(n, HIDDEN, generator=g, device="cuda").to(dtype)

    adapter = [0, -1, 2]

    def slots(counts):
        return torch.tensor([s for s, n in zip(adapter, counts) for _ in range(n)], dtype=torch.int32, device="cuda")

    context = torch.zeros(B, dtype=torch.int32, device="cuda")
    m.step(rows(sum(prompt)), slots(prompt), None, prompt, context)
    context += torch.tensor(prompt, dtype=torch.int32, device="cuda")
    at_prompt = [(k.clone(), v.clone()) for k, v in zip(m.k, m.v)], context.clone()

    # a tree of seven nodes, a chain of three, a single token
    counts = [7, 3, 1]
    parents = torch.tensor([-1, 0, 0, 1, 2, 2, 5] + [-1, 0, 1] + [-1], dtype=torch.int32, device="cuda")
    kept = [[0, 2, 5], [0, 1], []]
    drafted, after = rows(sum(counts)), rows(B)
    out = m.step(drafted, slots(counts), parents, counts, context)
    path = torch.tensor([p + [0] * (3 - len(p)) for p in kept], dtype=torch.int32, device="cuda")
    n_kept = torch.tensor([len(p) for p in kept], dtype=torch.int32, device="cuda")
    glsa.keep_path(m.k, m.v, m.page_table, context, path, n_kept)
    context += n_kept
    start = [0, 7, 10]
    tree = [out[s + n] for s, p in zip(start, kept) for n in p]
    tree += list(m.step(after, slots([1] * B), None, [1] * B, context))

    caches, context = at_prompt
    for i, (k, v) in enumerate(caches):
        m.k[i].copy_(k)
        m.v[i].copy_(v)
    single = [[], [], []]
    for j in range(3):  # sequences whose path has ended take no token
        counts = [int(j < len(p)) for p in kept]
        now = [b for b in range(B) if counts[b]]
        h = torch.stack([drafted[start[b] + kept[b][j]] for b in now])
        out = m.step(h, slots(counts), None, counts, context)
        for row, b in enumerate(now):
            single[b].append(out[row])
        context += torch.tensor(counts, dtype=torch.int32, device="cuda")
    one_by_one = [r for s in single for r in s] + list(m.step(after, slots([1] * B), None, [1] * B, context))
    return torch.stack(tree), torch.stack(one_by_one)


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--dtype", choices=("f32", "f16", "bf16"), default="bf16")
    ap.add_argument("--norm", action="store_true")
    args = ap.parse_args()
    tree, single = run({"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[args.dtype], args.norm)
    off, most = float((tree - single).abs().max()), float(single.abs().max())
    print(f"{len(tree)} rows, largest difference {off:.3g} of {most:.3g}")
