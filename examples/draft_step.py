"""One speculative decoding step over a cache that is kept compressed.

A cache is coded against its predictor, and its pages come back into a page pool
(decode_chunks). A tree of drafted tokens is then verified in one pass: pages and
slots for it (PagePool), its K and V rows into the pages (append), attention of the
whole tree over context and ancestors (attend), and the accepted path written again in
order over the tree (append with rows), ready for the next step.

    python examples/draft_step.py
"""
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

from lossless_kv_cache_scalar_gb300 import Coder, Layout, PagedKV, PagePool, synth  # noqa: E402


def tree_mask(parents):
    """int64 [nodes][1]: bit j of node i iff j is i or an ancestor of i (parents come
    before their children; -1: a child of the context), for up to 64 nodes."""
    bits = []
    for i, p in enumerate(parents):
        bits.append((bits[p] if p >= 0 else 0) | (1 << i))
    return torch.tensor([[b - (1 << 64) if b >> 63 else b] for b in bits], dtype=torch.int64)


def step(tokens=1000, group=4):
    """The whole step; returns what it made and what it had."""
    heads, dim, page = 8, 128, 256
    # a one-layer cache of `tokens` tokens, compressed against its predictor
    cfg = synth.CONFIGS["tiny"].scaled(n_tokens=tokens)
    w = {k: v.cuda() for k, v in synth.generate(cfg).items()}
    kv = w["mu"]                                           # what the predictor says, for a cache without outliers
    lay = Layout("bf16", 1, 2, heads, dim, tokens, tokens_per_chunk=page)
    coder = Coder(lay)
    bits, offsets = coder.encode(kv, w["mu"], w["sigma"], w["counts"])

    # a pool with room for the tree; the prompt takes its pages
    pages = -(-tokens // page)
    pool = PagePool(1, pages + 2, page, pages + 2)
    ctx = torch.zeros(1, dtype=torch.int32, device="cuda")
    new = torch.full((1,), tokens, dtype=torch.int32, device="cuda")
    pool.step(ctx, new, tokens)
    # its pages, K then V, are decoded to where the block table says
    at = pool.block_table[0, :pages].long()
    kv_pages = torch.zeros(2, pages + 2, page, heads, dim, dtype=torch.int16, device="cuda")
    got = coder.decode_chunks(bits, offsets, w["mu"], w["sigma"], w["counts"],
                              torch.arange(2 * pages, dtype=torch.int32, device="cuda"))
    kv_pages[:, at] = got.view(2, pages, page, heads, dim)
    cache = PagedKV(kv_pages[0], kv_pages[1], pool.block_table, q_heads=heads * group)

    # the drafted tree
    parents = [-1, 0, 0, 1, 1, 2, 3, 6, 6, -1, 9]
    n = len(parents)
    g = torch.Generator("cuda")
    g.manual_seed(0)
    q = torch.randn(n, heads * group, dim, generator=g, device="cuda").to(torch.bfloat16)
    k, v = (torch.randn(n, heads, dim, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    ctx.fill_(tokens)
    new.fill_(n)
    cu, slots = pool.step(ctx, new, n)
    cache.append(k, v, slots)
    out = cache.attend(q, ctx, cu, mask=tree_mask(parents).cuda(), max_nodes=n)

    # say the path 0 - 1 - 3 - 6 - 8 is accepted: its rows move to the front of the tree's slots
    path = [0, 1, 3, 6, 8]
    rows = torch.zeros(n, dtype=torch.int32, device="cuda")
    rows[:len(path)] = torch.tensor(path, dtype=torch.int32, device="cuda")
    keep = torch.where(torch.arange(n, device="cuda") < len(path), slots, torch.full_like(slots, -1))
    cache.append(k, v, keep, rows=rows)

    # the last accepted token again, now as a single token over a longer context: the same attention
    ctx.fill_(tokens + len(path) - 1)
    cu1 = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    again = cache.attend(q[path[-1]:path[-1] + 1], ctx, cu1, max_nodes=1)
    return dict(out=out, again=again, path=path, cache=cache, pool=pool, slots=slots, q=q, k=k, v=v, parents=parents,
                bytes=bits.numel(), values=lay.n_elems)


def main(tokens=1000, group=4):
    s = step(tokens, group)
    out, again, path = s["out"], s["again"], s["path"]
    off = (again[0].float() - out[path[-1]].float()).abs().max().item()
    print(f"{tokens} tokens in {s['bytes']} bytes ({8.0 * s['bytes'] / s['values']:.2f} bits per value); "
          f"{len(s['parents'])} drafted, {len(path)} accepted; tree and single-token attention differ by {off:.4f} at most")
    return out, again, path


if __name__ == "__main__":
    main()
