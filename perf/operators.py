"""Measured cases of the paged-cache operators that serve a speculative decoder.

A serving step over a paged KV cache is three operators, each with its own
cases here:

  map     block tables and slot maps built on the GPU from request lengths
          (PageTable.map_into);
  append  the step's new K and V rows written into the cache's pages at those
          slots, copied (bf16) or quantised (e4m3) (PagedKV.append_into);
  attend  attention of a tree of drafted tokens over the pages, one token per
          request being the tree of one node (PagedKV.attend_into).

The shapes are the repository's own KV caches (8 KV heads of 128 channels, bf16
or e4m3, 256-token pages, contexts up to 131,072 tokens) and generic ones around
them (other page lengths, head sizes and query groups).

`own` False computes the plain form of each operator in elementary torch
operations; True calls the library.
"""
import math

import torch

own = False

KV_HEADS = 8


def listed():
    return [
        # one request, one token, a chat-sized context: pure latency
        dict(name="attend_decode_one", op="attend", requests=1, nodes=1, ctx=1000, group=4, page=256, dtype="bf16", dim=128),
        # four requests verifying small trees over short contexts, small pages
        dict(name="attend_tree_small", op="attend", requests=4, nodes=16, ctx=4096, group=2, page=16, dtype="bf16", dim=64),
        # a full serving batch of plain single-token decoding over an 8-bit cache
        dict(name="attend_decode_batch", op="attend", requests=64, nodes=1, ctx=8192, group=8, page=64, dtype="e4m3", dim=128),
        # mixed batch, odd tree size, odd query group, pages that end inside any power-of-two tile
        dict(name="attend_tree_ragged", op="attend", requests=24, nodes=27, ctx=6000, group=5, page=24, dtype="bf16", dim=128),
        # one long document, a wide tree, the format's 256-token pages
        dict(name="attend_tree_long", op="attend", requests=1, nodes=63, ctx=131072, group=5, page=256, dtype="bf16", dim=128),
        # a batch of wide trees over the 8-bit cache
        dict(name="attend_tree_fp8", op="attend", requests=16, nodes=60, ctx=16384, group=8, page=64, dtype="e4m3", dim=128),
        # the largest: 64-node trees, 64 query heads, 32,768-token contexts
        dict(name="attend_tree_large", op="attend", requests=16, nodes=64, ctx=32768, group=8, page=256, dtype="bf16", dim=128),
        # the map of one decoding step of a small batch
        dict(name="map_decode", op="map", requests=8, new=1, ctx=4000, page=256),
        # the map of a step that admits many prompts at once, while other requests end
        dict(name="map_prefill", op="map", requests=2000, new=2000, ctx=3000, page=16),
        # the new rows of one decoding step
        dict(name="append_decode", op="append", tokens=8, page=256, dtype="bf16", dim=128, accepted=False),
        # drafted rows of which the accepted ones are rewritten in order (row indices, holes), 8-bit cache
        dict(name="append_accept_fp8", op="append", tokens=1919, page=64, dtype="e4m3", dim=128, accepted=True),
        # the rows of a long prompt
        dict(name="append_prompt", op="append", tokens=65536, page=256, dtype="bf16", dim=128, accepted=False),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "map", "append"])
    if op == "map":
        return dict(op=op, requests=_log_int(rng, 1, 2000), new=_log_int(rng, 1, 2000), ctx=_log_int(rng, 1, 3000),
                    page=rng.choice([16, 24, 64, 256]))
    if op == "append":
        return dict(op=op, tokens=_log_int(rng, 1, 65536), page=rng.choice([16, 24, 64, 256]), dtype=rng.choice(["bf16", "e4m3"]),
                    dim=rng.choice([64, 96, 128]), accepted=rng.random() < 0.4)
    requests = _log_int(rng, 1, 64)
    nodes = 1 if rng.random() < 0.3 else rng.randint(2, 64)
    group = rng.choice([1, 2, 4, 5, 8])
    # tokens of context over the batch stay within the largest listed case's
    ctx = _log_int(rng, 1, min(131072, (16 * 32768) // requests))
    return dict(op=op, requests=requests, nodes=nodes, ctx=ctx, group=group, page=rng.choice([16, 24, 64, 256]),
                dtype=rng.choice(["bf16", "e4m3"]), dim=rng.choice([64, 96, 128]))


# ---------------------------------------------------------------- inputs

def _lengths(case, gen):
    """Context and new-token counts of an attend case: the first request has the full
    context and tree, the others are spread below (host lists, from the case's generator)."""
    b = case["requests"]
    r = torch.rand(b, generator=gen, dtype=torch.float64)
    u = torch.rand(b, generator=gen, dtype=torch.float64)
    ctx = [case["ctx"] if i == 0 else int(case["ctx"] * (0.25 + 0.75 * float(r[i]))) for i in range(b)]
    new = [case["nodes"] if i == 0 or float(u[i]) < 0.6 else 1 + int(float(u[i]) * (case["nodes"] - 1)) for i in range(b)]
    return ctx, new


def _host_gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def _trees(new, count, gen):
    """Parent-before-child trees: node i of a request hangs below a random earlier
    node, or below the context. Returns the ancestor-or-self bits, int64 [count, words]."""
    words = -(-max(new) // 64)
    rows = []
    for n in new:
        r = torch.rand(n, generator=gen, dtype=torch.float64).tolist()
        bits = []
        for i in range(n):
            p = int(r[i] * (i + 1)) - 1                 # -1: a child of the context
            bits.append((bits[p] if p >= 0 else 0) | (1 << i))
        rows += bits
    out = torch.zeros(count, words, dtype=torch.int64)
    for w in range(words):
        part = [(b >> (64 * w)) & ((1 << 64) - 1) for b in rows]
        out[:len(rows), w] = torch.tensor([p - (1 << 64) if p >> 63 else p for p in part], dtype=torch.int64)
    return out


def _channel_scale(dim, gen):
    """Per-channel magnitudes of keys: log-normal, as real key channels are uneven."""
    return torch.exp(0.5 * torch.randn(KV_HEADS, dim, generator=gen, device="cuda"))


def _pool(pages, case, gen, spread):
    shape = (pages, case["page"], KV_HEADS, case["dim"])
    x = torch.randn(shape, generator=gen, device="cuda")
    x *= spread
    if case["dtype"] == "bf16":
        return x.to(torch.bfloat16), None
    scale = x.abs().amax(dim=(0, 1, 3)) / 448.0          # per head
    return (x / scale[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8), scale


def _prepare_attend(case, seed):
    hg = _host_gen(seed)
    gen = torch.Generator("cuda")
    gen.manual_seed(seed)
    ctx, new = _lengths(case, hg)
    page, dim, b = case["page"], case["dim"], case["requests"]
    need = [-(-(c + n) // page) for c, n in zip(ctx, new)]
    width, total = max(need), sum(need)
    perm = torch.randperm(total, generator=hg, dtype=torch.int32)
    table = torch.full((b, width), -1, dtype=torch.int32)
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = perm[at:at + n]
        at += n
    spread = _channel_scale(dim, gen)
    k, ks = _pool(total, case, gen, spread)
    v, vs = _pool(total, case, gen, 1.0)
    # buffers of a fixed size, as a captured step keeps them: rows past the step's tokens stay 0
    rows, heads = b * case["nodes"], KV_HEADS * case["group"]
    # queries as they leave a fused projection: a slice of wider rows; scores spread by about 2
    wide = torch.randn(rows, heads + 2 * KV_HEADS, dim, generator=gen, device="cuda")
    wide *= 2.0 / float(spread.square().mean().sqrt())
    q = wide.to(torch.bfloat16)[:, :heads]
    cu = torch.zeros(b + 1, dtype=torch.int32)
    cu[1:] = torch.tensor(new, dtype=torch.int32).cumsum(0)
    s = dict(q=q, k=k, v=v, ks=ks, vs=vs, table=table.cuda(), ctx=torch.tensor(ctx, dtype=torch.int32).cuda(), cu=cu.cuda(),
             mask=None if case["nodes"] == 1 else _trees(new, rows, hg).cuda(), most=case["nodes"],
             out=torch.zeros(rows, heads, dim, dtype=torch.bfloat16, device="cuda"))
    if own:
        from lossless_kv_cache_scalar_gb300 import PagedKV
        s["cache"] = PagedKV(k, v, s["table"], k_scale=ks, v_scale=vs, q_heads=heads)
    return s


def _prepare_map(case, seed):
    hg = _host_gen(seed)
    b, page = case["requests"], case["page"]
    r = torch.rand(3, b, generator=hg, dtype=torch.float64)
    ctx = [case["ctx"] if i == 0 else 1 + int(case["ctx"] * float(r[0, i])) for i in range(b)]
    new = [case["new"] if i == 0 else 1 + int((case["new"] - 1) * float(r[1, i])) for i in range(b)]
    have = [-(-c // page) for c in ctx]
    ended = [i > 0 and float(r[2, i]) < 0.1 for i in range(b)]
    width = -(-(case["ctx"] + case["new"]) // page)
    pool = b * width
    perm = torch.randperm(pool, generator=hg, dtype=torch.int32)
    used = sum(have)
    table = torch.full((b, width), -1, dtype=torch.int32)
    at = 0
    for i, n in enumerate(have):
        table[i, :n] = perm[at:at + n]
        at += n
    free = torch.full((pool,), -1, dtype=torch.int32)
    # a ring of free pages that has gone round before
    head = int(float(torch.rand(1, generator=hg, dtype=torch.float64)) * pool)
    free[(head + torch.arange(pool - used)) % pool] = perm[used:]
    ctx = [-1 if e else c for c, e in zip(ctx, ended)]
    new = [0 if e else n for n, e in zip(new, ended)]

    def dev(v):
        return torch.tensor(v, dtype=torch.int32).cuda()

    s = dict(page=page, pool=pool, table=table.cuda(), free=free.cuda(), ctx=dev(ctx), new=dev(new), n_pages=dev(have),
             state=dev([head, pool - used]), n_pages_out=dev([0] * b), state_out=dev([0, 0]), cu=dev([0] * (b + 1)),
             # a fixed-size buffer, as a captured step keeps it: its tail past the step's tokens reads -1
             slots=torch.empty(b * case["new"] + 3, dtype=torch.int64, device="cuda"))
    if own:
        from lossless_kv_cache_scalar_gb300 import PageTable
        s["pages"] = PageTable(s["table"], page, pool)
    return s


def _prepare_append(case, seed):
    hg = _host_gen(seed)
    gen = torch.Generator("cuda")
    gen.manual_seed(seed)
    n, page, dim = case["tokens"], case["page"], case["dim"]
    pages = -(-n // page) + 8
    spread = _channel_scale(dim, gen)
    k, ks = _pool(pages, case, gen, spread)
    v, vs = _pool(pages, case, gen, 1.0)
    # rows of a fused projection: K and V are slices of the same wide rows (behind 8 query heads)
    wide = torch.randn(n, 3 * KV_HEADS, dim, generator=gen, device="cuda")
    wide[:, KV_HEADS:2 * KV_HEADS] *= spread
    wide = wide.to(torch.bfloat16)
    # tokens of one request fill its pages in order; the pages lie anywhere in the pool
    order = torch.randperm(pages, generator=hg)
    t = torch.arange(n)
    slots = order[t // page] * page + t % page
    rows = None
    if case["accepted"]:
        # of every 60 drafted rows an ascending few are accepted: they move to the front
        keep = torch.rand(n, generator=hg) < 0.3
        rows = torch.arange(n)
        for a in range(0, n, 60):
            z = min(n, a + 60)
            took = torch.arange(a, z)[keep[a:z]]
            rows[a:a + len(took)] = took
            rows[a + len(took):z] = 0
            slots[a + len(took):z] = -1
        rows = rows.to(torch.int32).cuda()
    s = dict(k_new=wide[:, KV_HEADS:2 * KV_HEADS], v_new=wide[:, 2 * KV_HEADS:], k=k, v=v, ks=ks, vs=vs, slots=slots.cuda(), rows=rows, page=page)
    if own:
        from lossless_kv_cache_scalar_gb300 import PagedKV
        s["cache"] = PagedKV(k, v, k_scale=ks, v_scale=vs)
    return s


def prepare(case, seed):
    s = {"attend": _prepare_attend, "map": _prepare_map, "append": _prepare_append}[case["op"]](case, seed)
    s["op"] = case["op"]
    return s


# ---------------------------------------------------------------- plain forms

def _values(pages, scale):
    x = pages.float() if scale is None else pages.view(torch.float8_e4m3fn).float()
    return x if scale is None else x * scale[:, None]


def _plain_attend(s):
    q, table, ctx, cu = s["q"], s["table"], s["ctx"].long(), s["cu"].long()
    b, heads, dim, n = table.shape[0], q.shape[1], q.shape[2], s["most"]
    group = heads // KV_HEADS
    tab = table.clamp(min=0).long()
    k = _values(s["k"], s["ks"])[tab].flatten(1, 2).permute(0, 2, 3, 1)          # [b, h, d, t]
    v = _values(s["v"], s["vs"])[tab].flatten(1, 2).permute(0, 2, 1, 3)          # [b, h, t, d]
    t = torch.arange(k.shape[3], device=q.device)
    count = cu[1:] - cu[:-1]
    node = torch.arange(n, device=q.device)
    row = (cu[:-1, None] + node).clamp(max=q.shape[0] - 1)                       # [b, n]
    at = t - ctx[:, None]                                                        # [b, t] drafted index of a position
    drafted = (at >= 0) & (at < count[:, None])
    if s["mask"] is None:
        sees = at[:, None, :] <= node[:, None]
    else:
        word = s["mask"][row].gather(2, (at.clamp(0, n - 1) // 64)[:, None, :].expand(-1, n, -1))
        sees = ((word >> (at.clamp(0, n - 1) % 64)[:, None, :]) & 1).bool()
    sees = (at < 0)[:, None, :] | (drafted[:, None, :] & sees)                   # [b, n, t]
    qq = q.float()[row].view(b, n, KV_HEADS, group, dim).permute(0, 2, 3, 1, 4).reshape(b, KV_HEADS, group * n, dim)
    score = (qq @ k * (1.0 / math.sqrt(dim))).view(b, KV_HEADS, group, n, -1)
    score = score.masked_fill(~sees[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    w = torch.exp(score - torch.where(torch.isinf(top), torch.zeros_like(top), top))
    den = w.sum(-1, keepdim=True)
    o = (w.flatten(2, 3) @ v).view(b, KV_HEADS, group, n, dim) / torch.where(den == 0, torch.ones_like(den), den)
    o = o.permute(0, 3, 1, 2, 4).reshape(b, n, heads, dim)
    i = torch.arange(q.shape[0], device=q.device)
    of = torch.searchsorted(cu[1:], i, right=True)
    live = of < b
    of = of.clamp(max=b - 1)
    o = o[of, (i - cu[of]).clamp(max=n - 1)]
    return torch.where(live[:, None, None], o, torch.zeros_like(o)).to(torch.bfloat16)


def _plain_map(s):
    page, table, free, slots = s["page"], s["table"], s["free"], s["slots"]
    ctx, new, have, state = s["ctx"].long(), s["new"].long(), s["n_pages"].long(), s["state"].long()
    gone = ctx < 0
    head, count, size = state[0], state[1], free.numel()
    want = torch.where(gone, torch.zeros_like(ctx), -(-(ctx + new) // page))
    need = torch.where(gone, torch.zeros_like(ctx), (want - have).clamp(min=0))
    back = torch.where(gone, have, torch.zeros_like(have))
    j = torch.arange(table.shape[1], device=table.device)
    # new pages come off the front of the ring, in order of request and page
    take = (j >= have[:, None]) & (j < want[:, None]) & ~gone[:, None]
    rank = (need.cumsum(0) - need)[:, None] + j - have[:, None]
    page_of = free[(head + rank.clamp(min=0)) % size]
    # pages of ended requests go behind its end, in the same order
    put = gone[:, None] & (j < have[:, None])
    to = (head + count + (back.cumsum(0) - back)[:, None] + j) % size
    longer = torch.cat([free, free.new_zeros(1)])
    longer[torch.where(put, to, size).flatten()] = table.flatten()
    free.copy_(longer[:-1])
    table.copy_(torch.where(take, page_of, table))
    s["n_pages_out"].copy_(torch.where(gone, torch.zeros_like(have), torch.maximum(have, want)))
    s["state_out"].copy_(torch.stack([(head + need.sum()) % size, count - need.sum() + back.sum()]))
    cu = s["cu"]
    cu.zero_()
    cu[1:] = new.cumsum(0)
    i = torch.arange(slots.numel(), device=slots.device)
    of = torch.searchsorted(cu[1:].long(), i, right=True)
    live = of < ctx.numel()
    of = of.clamp(max=ctx.numel() - 1)
    pos = torch.where(live, ctx[of] + i - cu[of], torch.zeros_like(i))
    slots.copy_(torch.where(live, table[of, pos // page].long() * page + pos % page, torch.full_like(i, -1)))


def _to_e4m3(x):
    """Codes of 64-bit values: the nearest of 4 significant bits and of steps no finer
    than 2^-9, ties to even, largest 448 (quotients can lie next to a border of 32 bits)."""
    step = torch.exp2(torch.frexp(x)[1].clamp(min=-5).double() - 4)
    return (torch.round(x / step) * step).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def _plain_append(s):
    slots = s["slots"]
    rows = torch.arange(slots.numel(), device=slots.device) if s["rows"] is None else s["rows"].long()
    live = slots >= 0
    rows, slots = rows[live], slots[live]
    for_k, for_v = s["k_new"][rows], s["v_new"][rows]
    if s["ks"] is not None:
        for_k, for_v = _to_e4m3(for_k.double() / s["ks"].double()[:, None]), _to_e4m3(for_v.double() / s["vs"].double()[:, None])
    s["k"].flatten(0, 1)[slots] = for_k
    s["v"].flatten(0, 1)[slots] = for_v


def _map_outputs(s):
    return dict(table=s["table"], free=s["free"], n_pages=s["n_pages_out"], state=s["state_out"], cu=s["cu"], slots=s["slots"])


def _append_outputs(s):
    if s["ks"] is None:
        return dict(k=s["k"], v=s["v"])
    return dict(k=s["k"].view(torch.float8_e4m3fn), v=s["v"].view(torch.float8_e4m3fn))


def run(s):
    if s["op"] == "attend":
        if own:
            s["cache"].attend_into(s["q"], s["ctx"], s["cu"], s["out"], mask=s["mask"], max_nodes=s["most"])
            return s["out"]
        return _plain_attend(s)
    if s["op"] == "map":
        if own:
            s["pages"].map_into(s["ctx"], s["new"], s["n_pages"], s["free"], s["state"], s["cu"], s["slots"],
                                s["n_pages_out"], s["state_out"])
        else:
            _plain_map(s)
        return _map_outputs(s)
    if own:
        s["cache"].append_into(s["k_new"], s["v_new"], s["slots"], rows=s["rows"])
    else:
        _plain_append(s)
    return _append_outputs(s)


# ---------------------------------------------------------------- work and the definition in 64 bits

def work(case):
    """Bytes and operations of one pass, from the expected lengths of the case's recipe."""
    if case["op"] == "map":
        live = 1 + 0.9 * (case["requests"] - 1)
        tokens = live * (1 + case["new"]) / 2
        # three lengths in, two counts and a prefix out per request; a table entry per page; a slot per token
        return dict(bytes=int(24 * case["requests"] + 4 * tokens / case["page"] + 8 * (case["requests"] * case["new"] + 3)), flops=int(4 * tokens))
    row = KV_HEADS * case["dim"]
    size = 2 if case["dtype"] == "bf16" else 1
    if case["op"] == "append":
        live = case["tokens"] * (0.3 if case["accepted"] else 1.0)
        return dict(bytes=int(live * 2 * row * (2 + size) + case["tokens"] * (12 if case["accepted"] else 8)),
                    flops=int(live * 2 * row))
    b = case["requests"]
    rest = b - 1
    tokens = case["ctx"] + rest * case["ctx"] * 0.625
    nodes = case["nodes"] + rest * (0.6 * case["nodes"] + 0.4 * (1 + 0.8 * (case["nodes"] - 1)))
    heads = KV_HEADS * case["group"]
    return dict(bytes=int((tokens + nodes) * 2 * row * size + 2 * nodes * heads * case["dim"] * 2),
                flops=int(4 * (nodes / b) * tokens * heads * case["dim"]))


def _exact_attend(case, seed):
    s = _prepare_attend(case, seed)
    ctx, cu = s["ctx"].tolist(), s["cu"].tolist()
    q, dim, page = s["q"], case["dim"], case["page"]
    out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")

    def stretch(pool, scale, ids, h):
        x = pool[ids, :, h]
        x = x.double() if scale is None else x.view(torch.float8_e4m3fn).double() * scale[h].double()
        return x.reshape(-1, dim)

    for r in range(case["requests"]):
        n, end = cu[r + 1] - cu[r], ctx[r] + cu[r + 1] - cu[r]
        ids = s["table"][r, :-(-end // page)].long()
        hide = torch.ones(n, n, dtype=torch.bool)
        masks = None if s["mask"] is None else s["mask"][cu[r]:cu[r + 1]].tolist()
        for i in range(n):
            for j in range(n):
                if masks is None:
                    hide[i, j] = j > i
                else:
                    hide[i, j] = not (masks[i][j // 64] >> (j % 64)) & 1
        hide = hide.cuda()
        for h in range(KV_HEADS):
            k, v = stretch(s["k"], s["ks"], ids, h)[:end], stretch(s["v"], s["vs"], ids, h)[:end]
            for g in range(h * case["group"], (h + 1) * case["group"]):
                z = q[cu[r]:cu[r + 1], g].double() @ k.T / math.sqrt(dim)
                z[:, ctx[r]:].masked_fill_(hide, -math.inf)
                out[cu[r]:cu[r + 1], g] = torch.softmax(z, -1) @ v
    return out


def _exact_append(case, seed):
    s = _prepare_append(case, seed)
    slots = s["slots"].tolist()
    rows = list(range(len(slots))) if s["rows"] is None else s["rows"].tolist()
    done = {}
    for name, new, scale in (("k", s["k_new"], s["ks"]), ("v", s["v_new"], s["vs"])):
        pool = s[name].double() if scale is None else s[name].view(torch.float8_e4m3fn).double()
        flat = pool.view(-1, KV_HEADS, case["dim"])
        keep = [(a, r) for a, r in zip(slots, rows) if a >= 0]
        if keep:
            x = new[torch.tensor([r for _, r in keep], device="cuda")].double()
            if scale is not None:
                x = x / scale.double()[None, :, None]
                # the 8-bit grid: 4 significant bits down to steps of 2^-9, largest 448, ties to even
                step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
                x = (torch.round(x / step) * step).clamp(-448, 448)
            flat[torch.tensor([a for a, _ in keep], device="cuda")] = x
        done[name] = pool
    return done


def exact(case, seed):
    if case["op"] == "map":
        return None          # whole numbers, held equal to the plain form's
    return _exact_attend(case, seed) if case["op"] == "attend" else _exact_append(case, seed)
