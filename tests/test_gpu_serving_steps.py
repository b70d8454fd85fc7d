"""Many speculative serving steps with every operator of the paged cache: pages and
slots, rotated rows, tree attention, verification, the accepted path moved together, forks, ends and
compaction. After each step the cache holds, for every request, exactly the rows of the tokens it
stands for at their positions."""
import random

import pytest
import torch

from tests._servetest import verify
from lossless_kv_cache_scalar_gb300 import PagedKV, PagePool, Rotary, Verifier

pytestmark = pytest.mark.gpu

VOCAB, HEADS, GROUP, DIM = 48, 2, 4, 64


def i32(v):
    return torch.tensor(v, dtype=torch.int32).cuda()


class Model:
    """One layer with random weights: rows of a token, and probabilities from what attention gives."""

    def __init__(self, seed, dtype, axes):
        g = torch.Generator()
        g.manual_seed(seed)
        self.rows = torch.randn(VOCAB, HEADS * GROUP + 2 * HEADS, DIM, generator=g).to(torch.bfloat16).cuda()
        self.head = (0.04 * torch.randn(HEADS * GROUP * DIM, VOCAB, generator=g)).cuda()
        self.draft = torch.softmax(1.5 * torch.randn(VOCAB, VOCAB, generator=g), -1).cuda()
        w = 1 + 0.2 * torch.randn(2, DIM, generator=g)
        freq = [1e4 ** (-2.0 * i / DIM) for i in range(DIM // 2)]
        self.axes = axes
        self.rotary = Rotary(DIM, freq, w[0], w[1], axes=[j % axes for j in range(DIM // 2)] if axes > 1 else None)
        self.scales = (torch.full((HEADS,), 0.02).cuda(), torch.full((HEADS,), 0.01).cuda()) if dtype == "e4m3" else (None, None)
        self.kind = torch.bfloat16 if dtype == "bf16" else torch.uint8

    def cache(self, pages, page, table):
        shape = (pages, page, HEADS, DIM)
        k, v = (torch.zeros(shape, dtype=self.kind, device="cuda") for _ in range(2))
        return PagedKV(k, v, table, k_scale=self.scales[0], v_scale=self.scales[1], q_heads=HEADS * GROUP)

    def write(self, cache, tokens, positions, slots):
        """The tokens' rows into the cache; their queries."""
        x = self.rows[tokens.long()]
        q, k, v = x[:, :HEADS * GROUP], x[:, HEADS * GROUP:HEADS * GROUP + HEADS], x[:, HEADS * GROUP + HEADS:]
        pos = positions if self.axes == 1 else torch.stack([positions // (a + 1) for a in range(self.axes)])
        return cache.rotate_append(self.rotary, q, k, v, pos.contiguous(), slots)


@pytest.mark.parametrize("dtype,axes,tree,draft", [("bf16", 1, True, "drawn"), ("e4m3", 1, True, "distinct"), ("bf16", 3, False, "drawn"),
                                                   ("e4m3", 3, True, "best")])
def test_steps(dtype, axes, tree, draft):
    rng = random.Random(5)
    g = torch.Generator()
    g.manual_seed(11)
    n, width, page, pages = 6, 24, 8, 150
    m = Model(3, dtype, axes)
    pool = PagePool(n, width, page, pages)
    cache, verifier = m.cache(pages, page, pool.block_table), Verifier(n, VOCAB)
    history = [[rng.randrange(VOCAB) for _ in range(rng.randint(1, 30))] for _ in range(n - 2)] + [None, None]     # None: an idle row
    # the prompts: all but their last token, which is the first tree's root
    ctx = [0 if h else -1 for h in history]
    new = [len(h) - 1 if h else 0 for h in history]
    cu, slots = pool.step(i32(ctx), i32(new), sum(new))
    flat = [t for h in history if h for t in h[:-1]]
    at = [i for h in history if h for i in range(len(h) - 1)]
    m.write(cache, i32(flat), i32(at), slots)
    ctx = [len(h) - 1 if h else -1 for h in history]
    accepted_in_all = 0
    for step in range(14):
        if step in (4, 9):
            live = [r for r in range(n) if ctx[r] >= 0]
            parents = [r if ctx[r] >= 0 and rng.random() < 0.7 else rng.choice(live) for r in range(n)]
            lens, src, dst, tokens = pool.fork(i32(parents), i32(ctx))
            cache.copy(src, dst, tokens)
            history = [list(history[p]) for p in parents]
            ctx = [ctx[p] for p in parents]
            assert lens.tolist() == ctx
        if step == 7:
            ctx[1], history[1] = -1, None
        if step in (6, 11):
            cache.copy(*pool.compact())
        # trees below each request's last token
        counts = [rng.choice([1, 4, 9]) if c >= 0 else 0 for c in ctx]
        rows, parents, depth = sum(counts), [], []
        for c in counts:
            d = [0]
            par = [-1]
            for i in range(1, c):
                p = rng.randrange(i) if tree else i - 1
                par.append(p)
                d.append(d[p] + 1)
            parents += par[:c]
            depth += d[:c]
        starts = [sum(counts[:r]) for r in range(n + 1)]
        tokens, bits = [0] * rows, [0] * rows
        for r in range(n):
            if counts[r]:
                tokens[starts[r]] = history[r][-1]
            used = {}
            for i in range(counts[r]):
                j = starts[r] + i
                if i:
                    p = starts[r] + parents[j]
                    w = m.draft[tokens[p]].cpu().clone()
                    if draft != "drawn":
                        w[used.get(p, [])] = 0
                    tokens[j] = int(w.argmax()) if draft == "best" else int(torch.multinomial(w, 1, generator=g))
                    used.setdefault(p, []).append(tokens[j])
                    bits[j] = bits[p]
                bits[j] |= 1 << i
        cu, slots = pool.step(i32(ctx), i32(counts), rows)
        assert cu.tolist() == starts
        pos = [ctx[r] + depth[starts[r] + i] for r in range(n) for i in range(counts[r])]
        q = m.write(cache, i32(tokens), i32(pos), slots)
        lens = i32(ctx)
        out = cache.attend(q, lens, cu, mask=torch.tensor(bits, dtype=torch.int64)[:, None].cuda(), max_nodes=9)
        probs = torch.softmax(m.draft[i32(tokens).long()].log() + out.float().flatten(1) @ m.head, -1)       # a draft that comes near
        q_rows = None if draft == "best" else m.draft[i32(tokens).long()]
        uniform = torch.rand(rows, generator=g)
        par = i32(parents) if tree else None
        acc, path, nxt, kept, after = verifier.verify(probs, i32(tokens), cu, uniform.cuda(), parents=par, draft_probs=q_rows, distinct=draft == "distinct",
                                                      slots=slots, ctx_len=lens)
        want = verify(probs.cpu().numpy(), None if q_rows is None else q_rows.cpu().numpy(), tokens, parents if tree else None, uniform.numpy(), starts,
                      VOCAB, draft == "distinct")
        assert acc.tolist() == want[0] and nxt.tolist() == want[2]
        cache.move(cu, path, slots, kept)
        path, nxt, after = path.tolist(), nxt.tolist(), after.tolist()
        for r in range(n):
            if counts[r]:
                took = path[starts[r]:starts[r] + want[0][r]]
                assert took == want[1][r]
                history[r] += [tokens[j] for j in took[1:]] + [nxt[r]]
                ctx[r] = after[r]
                accepted_in_all += len(took) - 1
                assert ctx[r] == len(history[r]) - 1
        # the cache holds what the tokens' rows are, written from scratch
        live = [r for r in range(n) if ctx[r] > 0]
        flat = [t for r in live for t in history[r][:-1]]
        at = [i for r in live for i in range(ctx[r])]
        fresh = m.cache(-(-len(flat) // page), page, None)
        m.write(fresh, i32(flat), i32(at), torch.arange(len(flat), device="cuda"))
        table = pool.block_table.tolist()
        where = torch.tensor([table[r][i // page] * page + i % page for r in live for i in range(ctx[r])]).cuda()
        for mine, theirs in ((cache.k_pages, fresh.k_pages), (cache.v_pages, fresh.v_pages)):
            assert torch.equal(mine.flatten(0, 1)[where], theirs.flatten(0, 1)[:len(flat)])
    assert accepted_in_all >= 5
