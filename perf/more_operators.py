"""Measured cases of the operators around the paged cache in a speculative
serving step.

  rotate   heads of queries and keys normalised and rotated by their positions, keys
           and values written into the cache's pages in the same pass
           (PagedKV.rotate_append_into);
  verify   drafted trees, or chains, walked against the target's probabilities with
           given random numbers: the accepted path, the next token, and what the
           cache needs to keep the path (Verifier.verify_into);
  move     the accepted tokens' rows moved together inside the pages
           (PagedKV.move_into);
  fork     requests that go on from other requests' tokens: whole pages shared, the
           begun ones copied, pages that nobody holds freed (PageTable.fork_into,
           PagedKV.copy_into);
  compact  live pages moved to the front of the pool (PageTable.compact_into,
           PagedKV.copy_into).

The shapes are the repository's own KV caches (8 KV heads of 128 channels, bf16
or e4m3, 256-token pages) and generic ones around them; vocabularies are that of
its models and generic ones, odd sizes among them.

`own` False computes the plain form of each operator in elementary torch
operations; True calls the library.
"""
import math

import torch

own = False

KV_HEADS = 8
UNIT = 2.0 ** 44                     # probabilities are summed as whole numbers of 2^-44


def listed():
    return [
        # the next tokens of a small batch: pure latency
        dict(name="rotate_decode", op="rotate", tokens=8, group=4, page=256, dtype="bf16", dim=128, rot=128, axes=1, pairs="halves", norm=True),
        # prompts with images: three position axes, 8-bit cache, pages that end inside any power-of-two tile
        dict(name="rotate_image_fp8", op="rotate", tokens=7001, group=5, page=24, dtype="e4m3", dim=128, rot=128, axes=3, pairs="halves", norm=True),
        # a long prompt, admitted at once
        dict(name="rotate_prompt", op="rotate", tokens=65536, group=4, page=256, dtype="bf16", dim=128, rot=128, axes=1, pairs="halves", norm=True),
        # one request with a short drafted chain: latency, one row of the vocabulary
        dict(name="verify_chain", op="verify", requests=1, nodes=5, vocab=151936, dtype="f32", draft="drawn", tree=False),
        # trees of the draft's best tokens, whose siblings differ and whose draft has no probabilities; odd vocabulary
        dict(name="verify_best", op="verify", requests=24, nodes=27, vocab=50257, dtype="f32", draft="best", tree=True),
        # a batch of wide trees drawn from the draft's probabilities
        dict(name="verify_batch", op="verify", requests=64, nodes=60, vocab=151936, dtype="f32", draft="drawn", tree=True),
        # the accepted rows of a small batch
        dict(name="move_small", op="move", requests=8, nodes=16, accepted=4, page=256, dtype="bf16", dim=128),
        # long accepted paths of many requests, 8-bit cache
        dict(name="move_batch", op="move", requests=256, nodes=60, accepted=13, page=64, dtype="e4m3", dim=128),
        # one step of a beam search of eight beams
        dict(name="fork_beams", op="fork", requests=8, live=8, ctx=4000, page=256, dtype="bf16", dim=128),
        # several answers sampled from each of many prompts: most rows go on from another one
        dict(name="fork_samples", op="fork", requests=700, live=90, ctx=3000, page=64, dtype="e4m3", dim=128),
        # a small pool after some requests have ended
        dict(name="compact_small", op="compact", requests=6, ctx=4000, page=256, fill=0.5, dtype="bf16", dim=64),
        # a large pool, half of it free
        dict(name="compact_pool", op="compact", requests=200, ctx=3000, page=64, fill=0.5, dtype="e4m3", dim=128),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["rotate", "rotate", "verify", "verify", "move", "fork", "compact"])
    page, dtype = rng.choice([16, 24, 64, 256]), rng.choice(["bf16", "e4m3"])
    if op == "rotate":
        dim = rng.choice([64, 96, 128])
        return dict(op=op, tokens=_log_int(rng, 1, 65536), group=rng.choice([1, 2, 4]), page=page, dtype=dtype, dim=dim,
                    rot=rng.choice([dim, 32]), axes=rng.choice([1, 1, 3]), pairs=rng.choice(["halves", "neighbours"]), norm=rng.random() < 0.7)
    if op == "verify":
        return dict(op=op, requests=_log_int(rng, 1, 64), nodes=rng.choice([1, rng.randint(2, 8), rng.randint(9, 60)]),
                    vocab=_log_int(rng, 1000, 151936), dtype=rng.choice(["f32", "f32", "bf16"]), draft=rng.choice(["drawn", "distinct", "best"]),
                    tree=rng.random() < 0.7)
    if op == "move":
        accepted = rng.randint(1, 13)
        return dict(op=op, requests=_log_int(rng, 1, 256), nodes=rng.randint(2 * accepted, 60), accepted=accepted, page=page, dtype=dtype,
                    dim=rng.choice([64, 96, 128]))
    if op == "fork":
        requests = _log_int(rng, 1, 700)
        return dict(op=op, requests=requests, live=rng.randint(max(1, requests // 10), max(1, requests // 7)) if requests > 32 else requests,
                    ctx=_log_int(rng, 1, 3000), page=page, dtype=dtype, dim=64)
    return dict(op=op, requests=_log_int(rng, 1, 200), ctx=_log_int(rng, 16, 3000), page=page, fill=rng.uniform(0.3, 0.9), dtype=dtype, dim=64)


# ---------------------------------------------------------------- inputs

def _host_gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def _dev_gen(seed):
    g = torch.Generator("cuda")
    g.manual_seed(seed)
    return g


def _i32(v):
    return torch.as_tensor(v).to(torch.int32).cuda()


def _ints(gen, lo, hi, n):
    """n whole numbers of [lo, hi]."""
    return (lo + torch.rand(n, generator=gen, dtype=torch.float64) * (hi + 1 - lo)).long().clamp(lo, hi)


def _spread(gen, hi, n):
    """n lengths spread evenly over [1, hi], in the seed's order behind the longest."""
    rest = [1 + (hi - 1) * i // n for i in range(1, n)]
    return [hi] + [rest[i] for i in torch.randperm(n - 1, generator=gen).tolist()]


def _pool(pages, case, gen):
    shape = (pages, case["page"], KV_HEADS, case["dim"])
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.bfloat16)
    if case["dtype"] == "bf16":
        return x
    return (x * 64.0).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def _scales(case, gen):
    """An 8-bit cache's scale of each head, for values of about 1 to 4."""
    if case["dtype"] == "bf16":
        return None, None
    u = torch.rand(2, KV_HEADS, generator=gen, device="cuda")
    return (0.004 + 0.01 * u[0]).contiguous(), (0.004 + 0.01 * u[1]).contiguous()


def _prepare_rotate(case, seed):
    hg, gen = _host_gen(seed), _dev_gen(seed)
    n, page, dim, rot, axes = case["tokens"], case["page"], case["dim"], case["rot"], case["axes"]
    heads = KV_HEADS * case["group"]
    pages = -(-n // page) + 8
    k, v = _pool(pages, case, gen), _pool(pages, case, gen)
    ks, vs = _scales(case, gen)
    # rows of a fused projection: queries, keys and values side by side
    wide = torch.randn(n, heads + 2 * KV_HEADS, dim, generator=gen, device="cuda")
    wide *= torch.exp(0.5 * torch.randn(heads + 2 * KV_HEADS, dim, generator=gen, device="cuda"))
    wide = wide.to(torch.bfloat16)
    norms = (1.0 + 0.2 * torch.randn(2, dim, generator=gen, device="cuda")) if case["norm"] else (None, None)
    freq = [1.0e6 ** (-2.0 * i / rot) for i in range(rot // 2)]
    # positions of stretches of text, anywhere in long contexts; with more axes, stretches of
    # image patches in rows of 40 between them
    starts = _ints(hg, 0, 131072, -(-n // 997))
    i = torch.arange(n)
    pos = starts[i // 997] + i % 997
    if axes == 3:
        patch = (i // 997) % 2 == 1
        base = starts[i // 997]
        pos = torch.stack([torch.where(patch, base, pos), torch.where(patch, base + i % 997 // 40, pos),
                           torch.where(patch, base + i % 997 % 40, pos)])
    axis_of = [min(2, j * 8 // (rot // 2) // 2 if rot >= 16 else 0) for j in range(rot // 2)] if axes == 3 else None
    order = torch.randperm(pages, generator=hg)
    slots = order[i // page] * page + i % page
    if n > 20:
        slots[_ints(hg, 0, n - 1, n // 20)] = -1               # tokens of a padded batch
    s = dict(q=wide[:, :heads], k_new=wide[:, heads:heads + KV_HEADS], v_new=wide[:, heads + KV_HEADS:], k=k, v=v, ks=ks, vs=vs,
             norms=norms, freq=freq, axis_of=axis_of, pos=_i32(pos), slots=slots.cuda(), pairs=case["pairs"], eps=1e-6,
             out=torch.empty(n, heads, dim, dtype=torch.bfloat16, device="cuda"))
    if own:
        from lossless_kv_cache_scalar_gb300 import PagedKV, Rotary
        s["rotary"] = Rotary(dim, freq, q_norm=norms[0], k_norm=norms[1], eps=1e-6, axes=axis_of, interleaved=case["pairs"] == "neighbours")
        s["cache"] = PagedKV(k, v, k_scale=ks, v_scale=vs)
    else:
        s["freq"] = torch.tensor(freq, dtype=torch.float64, device="cuda")
        s["axis_of"] = None if axis_of is None else torch.tensor(axis_of, device="cuda")
    return s


def _lengths(case, gen):
    """New tokens of each request: the first has a full tree, many others too."""
    b, n = case["requests"], case["nodes"]
    u = torch.rand(b, generator=gen, dtype=torch.float64).tolist()
    return [n if i == 0 or u[i] < 0.6 else 1 + int(u[i] * (n - 1)) for i in range(b)]


def _prepare_verify(case, seed):
    hg, gen = _host_gen(seed), _dev_gen(seed)
    b, nodes, vocab = case["requests"], case["nodes"], case["vocab"]
    new = _lengths(case, hg)
    rows = b * nodes
    cu = torch.zeros(b + 1, dtype=torch.int64)
    cu[1:] = torch.tensor(new).cumsum(0)
    # peaked probabilities, and a draft that comes near them
    logits = torch.randn(rows, vocab, generator=gen, device="cuda")
    logits *= 5.0
    noise = torch.randn(rows, vocab, generator=gen, device="cuda")
    noise *= 0.8
    noise += logits
    probs = torch.softmax(logits, -1)
    del logits
    draft = torch.softmax(noise, -1)
    del noise
    # a node's parent comes before it in its request; its token is the draft's at its parent
    r = torch.rand(rows, generator=hg, dtype=torch.float64).tolist()
    parents, rank, most = [-1] * rows, [0] * rows, 1
    for a, z in zip(cu[:-1].tolist(), cu[1:].tolist()):
        below = {}
        for i in range(1, z - a):
            p = int(r[a + i] * i) if case["tree"] else i - 1
            parents[a + i] = p
            rank[a + i] = below.get(p, 0)
            below[p] = rank[a + i] + 1
            most = max(most, below[p])
    of = torch.zeros(rows, dtype=torch.int64)
    for a, z in zip(cu[:-1].tolist(), cu[1:].tolist()):
        of[a:z] = a
    par = torch.tensor(parents)
    if case["draft"] == "best":
        choice = draft.topk(most, -1).indices
    else:
        choice = torch.multinomial(draft, most, replacement=case["draft"] == "drawn", generator=gen)
    tokens = choice[(of + par.clamp(min=0)).cuda(), torch.tensor(rank).cuda()]
    if case["dtype"] == "bf16":
        probs, draft = probs.to(torch.bfloat16), draft.to(torch.bfloat16)
    # slots of the new tokens and contexts, as the page map leaves them
    slots = torch.randperm(rows + 7, generator=hg)[:rows]
    slots[int(cu[-1]):] = -1
    s = dict(probs=probs, draft=None if case["draft"] == "best" else draft, tokens=tokens.to(torch.int32),
             parents=_i32(parents) if case["tree"] else None, cu=_i32(cu), uniform=torch.rand(rows, generator=gen, device="cuda"),
             slots=slots.cuda(), ctx=_i32(_ints(hg, 1, 131072, b)), distinct=case["draft"] == "distinct", most=nodes,
             accepted=_i32([0] * b), rows=_i32([0] * rows), next=_i32([0] * b), kept=torch.zeros(rows, dtype=torch.int64, device="cuda"),
             ctx_out=_i32([0] * b))
    if own:
        from lossless_kv_cache_scalar_gb300 import Verifier
        s["verifier"] = Verifier(b, vocab)
    return s


def _prepare_move(case, seed):
    hg, gen = _host_gen(seed), _dev_gen(seed)
    b, page = case["requests"], case["page"]
    new = _lengths(case, hg)
    rows = b * case["nodes"]
    cu = torch.zeros(b + 1, dtype=torch.int64)
    cu[1:] = torch.tensor(new).cumsum(0)
    # each request's new tokens fill consecutive places from the middle of a page on
    width = -(-case["nodes"] // page) + 1
    order = torch.randperm(b * width, generator=hg).view(b, width)
    start = _ints(hg, 0, page - 1, b)
    slots = torch.full((rows,), -1, dtype=torch.int64)
    kept = torch.full((rows,), -1, dtype=torch.int64)
    path = torch.full((rows,), -1, dtype=torch.int64)
    for r in range(b):
        a, n = int(cu[r]), new[r]
        at = int(start[r]) + torch.arange(n)
        slots[a:a + n] = order[r, at // page] * page + at % page
        # the root stays; the rest of the path is spread over the wider levels behind it
        m = min(case["accepted"], max(1, n // 2))
        far = m + torch.randperm(n - m, generator=hg)[:m - 1].sort().values
        path[a:a + m] = a + torch.cat([torch.zeros(1, dtype=torch.int64), far])
        kept[a:a + m] = slots[a:a + m]
    s = dict(k=_pool(b * width, case, gen), v=_pool(b * width, case, gen), cu=_i32(cu), slots=slots.cuda(), kept=kept.cuda(), path=_i32(path))
    if own:
        from lossless_kv_cache_scalar_gb300 import PagedKV
        s["cache"] = PagedKV(s["k"], s["v"])
    return s


def _prepare_fork(case, seed):
    hg, gen = _host_gen(seed), _dev_gen(seed)
    b, page, live = case["requests"], case["page"], case["live"]
    ctx = _spread(hg, case["ctx"], live) + [-1] * (b - live)
    have = [-(-c // page) if c >= 0 else 0 for c in ctx]
    width = -(-case["ctx"] // page) + 1
    # some rows hold a page more than their tokens need (drafted ones that were not accepted)
    have = [h + (i < live and i % 3 == 1) for i, h in enumerate(have)]
    used = sum(have)
    pool = used + b
    perm = torch.randperm(pool, generator=hg)
    table = torch.full((b, width), -1, dtype=torch.int64)
    at = 0
    for i, n in enumerate(have):
        table[i, :n] = perm[at:at + n]
        at += n
    head = int(_ints(hg, 0, pool - 1, 1))
    free = torch.full((pool,), -1, dtype=torch.int64)
    free[(head + torch.arange(pool - used)) % pool] = perm[used:]
    # a row goes on from itself or from another live one; some rows end
    parents = torch.where(torch.rand(b, generator=hg) < 0.3, torch.arange(b), _ints(hg, 0, live - 1, b))
    parents[torch.rand(b, generator=hg) < 0.05] = -1
    s = dict(page=page, pool=pool, k=_pool(pool, case, gen), v=_pool(pool, case, gen), table=_i32(table), ctx=_i32(ctx), have=_i32(have),
             free=_i32(free), state=_i32([head, pool - used]), parents=_i32(parents), table_out=_i32(torch.full((b, width), -1)),
             n_out=_i32([0] * b), ctx_out=_i32([0] * b), state_out=_i32([0, 0]), src=_i32([0] * b), dst=_i32([0] * b), count=_i32([0] * b))
    if own:
        from lossless_kv_cache_scalar_gb300 import PagedKV, PageTable
        s["pages"], s["cache"] = PageTable(s["table"], page, pool, workspace=True), PagedKV(s["k"], s["v"])
    return s


def _prepare_compact(case, seed):
    hg, gen = _host_gen(seed), _dev_gen(seed)
    b, page = case["requests"], case["page"]
    have = [-(-c // page) for c in _spread(hg, case["ctx"], b)]
    used, width = sum(have), max(have)
    pool = max(used + 1, int(used / case["fill"]))
    perm = torch.randperm(pool, generator=hg)
    table = torch.full((b, width), -1, dtype=torch.int64)
    at = 0
    for i, n in enumerate(have):
        table[i, :n] = perm[at:at + n]
        at += n
    # some requests share another's first pages
    for i in range(1, b):
        if i % 5 == 0:
            m = min(have[i], have[i - 1]) // 2
            table[i, :m] = table[i - 1, :m]
    s = dict(page=page, pool=pool, k=_pool(pool, case, gen), v=_pool(pool, case, gen), table=_i32(table), have=_i32(have),
             free=_i32([-1] * pool), state=_i32([0, 0]), table_out=_i32(torch.full((b, width), -1)), state_out=_i32([0, 0]),
             src=_i32([0] * used), dst=_i32([0] * used))
    if own:
        from lossless_kv_cache_scalar_gb300 import PagedKV, PageTable
        s["pages"], s["cache"] = PageTable(s["table"], page, pool, workspace=True), PagedKV(s["k"], s["v"])
    return s


def prepare(case, seed):
    s = {"rotate": _prepare_rotate, "verify": _prepare_verify, "move": _prepare_move, "fork": _prepare_fork,
         "compact": _prepare_compact}[case["op"]](case, seed)
    s["op"] = case["op"]
    return s


# ---------------------------------------------------------------- plain forms

def _to_e4m3(x):
    """Codes of 64-bit values: the nearest of 4 significant bits and of steps no finer
    than 2^-9, ties to even, largest 448 (quotients can lie next to a border of 32 bits)."""
    step = torch.exp2(torch.frexp(x)[1].clamp(min=-5).double() - 4)
    return (torch.round(x / step) * step).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def _plain_rotate(s):
    half = s["freq"].numel()
    pos = s["pos"].double()
    if s["axis_of"] is None:
        angle = pos[:, None] * s["freq"]
    else:
        angle = pos[s["axis_of"]].T * s["freq"]
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]

    def turned(x, weight):
        x = x.float()
        if weight is not None:
            x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + s["eps"]) * weight
        lead, rest = x[..., :2 * half], x[..., 2 * half:]
        if s["pairs"] == "halves":
            a, b = lead[..., :half], lead[..., half:]
            lead = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
        else:
            a, b = lead[..., 0::2], lead[..., 1::2]
            lead = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
        return torch.cat([lead, rest], -1)

    s["out"].copy_(turned(s["q"], s["norms"][0]))
    live = s["slots"] >= 0
    slots = s["slots"][live]
    k, v = turned(s["k_new"], s["norms"][1])[live], s["v_new"][live]
    if s["ks"] is None:
        k = k.to(torch.bfloat16)
    else:
        k, v = _to_e4m3(k.double() / s["ks"].double()[:, None]), _to_e4m3(v.double() / s["vs"].double()[:, None])
    s["k"].flatten(0, 1)[slots] = k
    s["v"].flatten(0, 1)[slots] = v


def _units(x):
    return torch.round(x.double() * UNIT).long()


def _plain_verify(s):
    probs, draft, tokens, cu = s["probs"], s["draft"], s["tokens"].long(), s["cu"].long()
    b, rows = s["accepted"].numel(), s["rows"].numel()
    base, count = cu[:-1], cu[1:] - cu[:-1]
    u = s["uniform"].double()
    each = torch.arange(b, device=cu.device)
    cur, c = torch.zeros_like(base), torch.zeros(b, dtype=torch.float64, device=cu.device)
    left, unseen = torch.ones_like(c), torch.ones_like(c)         # what is left of the target's and of the draft's mass
    gone = torch.zeros(b, probs.shape[1], dtype=torch.bool, device=cu.device) if draft is None else None
    path = torch.zeros(b, s["most"], dtype=torch.int64, device=cu.device)
    taken = (count > 0).long()

    def weights(c):
        p = probs[(base + cur).clamp(max=rows - 1)].double().clamp(0, 1)
        if draft is None:
            return _units(p.masked_fill(gone, 0))
        q = draft[(base + cur).clamp(max=rows - 1)].double().clamp(0, 1)
        return _units((p - c[:, None] * q).float().clamp(min=0))

    for i in range(1, s["most"]):
        row = (base + i).clamp(max=rows - 1)
        at = (base + cur).clamp(max=rows - 1)
        turn = (i < count) & ((i - 1 if s["parents"] is None else s["parents"][row].long()) == cur)
        tok = tokens[row].clamp(0, probs.shape[1] - 1)
        p = probs[at, tok].double().clamp(0, 1)
        if draft is None:
            p = p.masked_fill(gone[each, tok], 0)
            take = turn & (u[row] * left < p)
            lose = turn & ~take
            left = torch.where(lose, (left - p).clamp(min=0), left)
            gone[each, tok] |= lose
            gone &= ~take[:, None]
        else:
            q = draft[at, tok].double().clamp(0, 1)
            rest = (p - c * q).float().clamp(min=0).double()
            take = turn & (u[row] * q * left < rest * unseen)
            lose = turn & ~take
            c = torch.where(lose, (c + left / torch.where(unseen > 0, unseen, torch.full_like(unseen, math.inf))).float().double(), c)
            if s["distinct"]:
                unseen = torch.where(lose, (unseen - q).clamp(min=0), unseen)
            left = torch.where(lose, weights(c).sum(1).double() / UNIT, left)
            c, unseen = c.masked_fill(take, 0), unseen.masked_fill(take, 1)
        left = left.masked_fill(take, 1)
        cur = torch.where(take, i, cur)
        path[each, torch.where(take, taken, 0)] = torch.where(take, i, path[:, 0])
        taken = taken + take.long()
    w = weights(c)
    none = w.sum(1) == 0
    if draft is None:
        gone &= ~none[:, None]
    w = torch.where(none[:, None], weights(c.masked_fill(none, 0)), w)
    run = w.cumsum(1)
    total = run[:, -1]
    t = torch.floor(u[base.clamp(max=rows - 1)] * total.double()).long()
    token = torch.searchsorted(run, torch.minimum(t, total - 1).clamp(min=0)[:, None], right=True)[:, 0]
    live = count > 0
    s["accepted"].copy_(taken)
    s["next"].copy_(torch.where(live & (total > 0), token, -1))
    s["ctx_out"].copy_(s["ctx"] + taken)
    i = torch.arange(rows, device=cu.device)
    of = torch.searchsorted(cu[1:], i, right=True).clamp(max=b - 1)
    j = i - base[of]
    inside, on = i < cu[-1], (i < cu[-1]) & (j < taken[of])
    s["rows"].copy_(torch.where(on, base[of] + path[of, j.clamp(0, s["most"] - 1)], torch.where(inside, -1, s["rows"].long())))
    s["kept"].copy_(torch.where(on, s["slots"], torch.where(inside, -1, s["kept"])))


def _plain_move(s):
    live = s["kept"] >= 0
    to = s["kept"][live]
    frm = s["slots"][s["path"][live].long()]
    for pool in (s["k"], s["v"]):
        flat = pool.flatten(0, 1)
        flat[to] = flat[frm]


def _copy_pages(s, src, dst, count):
    """Pages src >= 0 to pages dst, the first `count` tokens of each (None: all)."""
    live = src >= 0
    src, dst = src[live].long(), dst[live].long()
    for pool in (s["k"], s["v"]):
        if count is None:
            pool[dst] = pool[src]
        else:
            keep = torch.arange(s["page"], device=src.device) < count[live][:, None]
            pool[dst] = torch.where(keep[:, :, None, None], pool[src], pool[dst])


def _plain_fork(s):
    page, pool, table, free = s["page"], s["pool"], s["table"].long(), s["free"].long()
    ctx, have, state, parents = s["ctx"].long(), s["have"].long(), s["state"].long(), s["parents"].long()
    b, width = table.shape
    head, count, size = state[0], state[1], free.numel()
    each = torch.arange(b, device=table.device)
    frm = parents.clamp(min=0)
    on = (parents >= 0) & (ctx[frm] >= 0)
    # the row that keeps its parent's pages whole: the parent itself, else the first
    key = torch.where(on, torch.where(parents == each, -1, each), b)
    first = torch.full((b,), b, device=table.device).scatter_reduce(0, frm, key, "amin")
    heir = on & (key == first[frm])
    c = torch.where(on, ctx[frm], 0)
    whole, part = c // page, c % page
    copies = on & ~heir & (part > 0)
    n = torch.where(heir, have[frm], torch.where(on, whole + copies, 0))
    rank = copies.cumsum(0) - copies.long()
    fresh = free[(head + rank) % size]
    j = torch.arange(width, device=table.device)
    old = table[frm]
    rows = torch.where(copies[:, None] & (j == whole[:, None]), fresh[:, None], old)
    inside = j < n[:, None]
    was = torch.zeros(pool + 1, dtype=torch.bool, device=table.device)
    was[torch.where(j < have[:, None], table, pool).flatten()] = True
    now = torch.zeros_like(was)
    now[torch.where(inside, rows, pool).flatten()] = True
    freed = (was & ~now)[:pool]
    order = freed.cumsum(0) - freed.long()
    longer = torch.cat([free, free.new_zeros(1)])
    longer[torch.where(freed, (head + count + order) % size, size)] = torch.arange(pool, device=table.device)
    s["free"].copy_(longer[:-1])
    s["table_out"].copy_(torch.where(inside, rows, s["table_out"].long()))
    s["n_out"].copy_(n)
    s["ctx_out"].copy_(torch.where(on, c, -1))
    took = copies.sum()
    s["state_out"].copy_(torch.stack([(head + took) % size, count - took + freed.sum()]))
    s["src"].copy_(torch.where(copies, old.gather(1, whole.clamp(max=width - 1)[:, None])[:, 0], -1))
    s["dst"].copy_(torch.where(copies, fresh, -1))
    s["count"].copy_(torch.where(copies, part, 0))
    _copy_pages(s, s["src"], s["dst"], s["count"])


def _plain_compact(s):
    pool, table, have = s["pool"], s["table"].long(), s["have"].long()
    width, room = table.shape[1], s["src"].numel()
    j = torch.arange(width, device=table.device)
    inside = j < have[:, None]
    held = torch.zeros(pool + 1, dtype=torch.bool, device=table.device)
    held[torch.where(inside, table, pool).flatten()] = True
    held = held[:pool]
    live = held.sum()
    page = torch.arange(pool, device=table.device)
    hole, far = ~held & (page < live), held & (page >= live)
    # the k-th far page goes to the k-th hole
    holes = torch.full((pool + 1,), -1, device=table.device)
    holes[torch.where(hole, hole.cumsum(0) - 1, pool)] = page
    rank = far.cumsum(0) - 1
    to = torch.where(far, holes[rank.clamp(min=0)], page)
    s["table_out"].copy_(torch.where(inside, to[table.clamp(min=0)], s["table_out"].long()))
    s["free"].copy_(torch.where(page < pool - live, live + page, s["free"].long()))
    s["state_out"].copy_(torch.stack([torch.zeros_like(live), pool - live]))
    at = torch.where(far, rank, room)
    for name, what in (("src", page), ("dst", to)):
        out = torch.full((room + 1,), -1, device=table.device)
        out[at] = what
        s[name].copy_(out[:-1])
    _copy_pages(s, s["src"], s["dst"], None)


# ---------------------------------------------------------------- one pass

def _own_pass(s):
    op = s["op"]
    if op == "rotate":
        s["cache"].rotate_append_into(s["rotary"], s["q"], s["k_new"], s["v_new"], s["pos"], s["slots"], s["out"])
    elif op == "verify":
        s["verifier"].verify_into(s["probs"], s["tokens"], s["cu"], s["uniform"], s["accepted"], s["rows"], s["next"],
                                  parents=s["parents"], draft_probs=s["draft"], distinct=s["distinct"], slots=s["slots"], kept=s["kept"],
                                  ctx_len=s["ctx"], ctx_out=s["ctx_out"])
    elif op == "move":
        s["cache"].move_into(s["cu"], s["path"], s["slots"], s["kept"])
    elif op == "fork":
        s["pages"].fork_into(s["parents"], s["ctx"], s["have"], s["free"], s["state"], s["table_out"], s["n_out"], s["ctx_out"],
                             s["state_out"], s["src"], s["dst"], s["count"])
        s["cache"].copy_into(s["src"], s["dst"], tokens=s["count"])
    else:
        s["pages"].compact_into(s["have"], s["free"], s["state"], s["table_out"], s["state_out"], s["src"], s["dst"])
        s["cache"].copy_into(s["src"], s["dst"])


def run(s):
    op = s["op"]
    if own:
        _own_pass(s)
    else:
        {"rotate": _plain_rotate, "verify": _plain_verify, "move": _plain_move, "fork": _plain_fork, "compact": _plain_compact}[op](s)
    if op == "verify":
        return dict(accepted=s["accepted"], rows=s["rows"], next=s["next"], kept=s["kept"], ctx=s["ctx_out"])
    if op == "rotate":
        values = torch.bfloat16 if s["ks"] is None else torch.float8_e4m3fn
        return dict(q=s["out"], k=s["k"].view(values), v=s["v"].view(values))
    # bits that are only moved, and whole numbers
    bits = torch.int16 if s["k"].element_size() == 2 else torch.uint8
    moved = dict(k=s["k"].view(bits), v=s["v"].view(bits))
    if op == "fork":
        moved.update(table=s["table_out"], n=s["n_out"], ctx=s["ctx_out"], state=s["state_out"], free=s["free"], src=s["src"], dst=s["dst"],
                     count=s["count"])
    elif op == "compact":
        moved.update(table=s["table_out"], state=s["state_out"], free=s["free"], src=s["src"], dst=s["dst"])
    return moved


# ---------------------------------------------------------------- work and the definition in 64 bits

def work(case):
    """Bytes and operations of one pass, from the expected counts of the case's recipe."""
    op = case["op"]
    if op == "verify":
        b, nodes = case["requests"], 1 + (case["requests"] - 1) * 0.8
        size = 2 if case["dtype"] == "bf16" else 4
        # the row that the last token is drawn from, the draft's beside it; a few words a node
        rows = b * case["vocab"] * size * (1 if case["draft"] == "best" or case["nodes"] == 1 else 2)
        return dict(bytes=int(rows + nodes * case["nodes"] * 40 + b * 32), flops=int(4 * b * case["vocab"]))
    row = KV_HEADS * case["dim"]
    size = 2 if case["dtype"] == "bf16" else 1
    if op == "rotate":
        n, heads = case["tokens"], KV_HEADS * case["group"]
        return dict(bytes=int(n * (4 * heads * case["dim"] + row * 2 * (2 + size) + 8 + 4 * case["axes"])),
                    flops=int(n * (heads + KV_HEADS) * case["dim"] * (7 if case["norm"] else 3)))
    if op == "move":
        rows = case["requests"] * max(0, case["accepted"] - 1)
        return dict(bytes=int(rows * 4 * row * size + case["requests"] * 24 * case["nodes"]), flops=0)
    b, width = case["requests"], -(-case["ctx"] // case["page"])
    if op == "fork":
        copied = 0.5 * b * (1 if b > 1 else 0)
        return dict(bytes=int(copied * case["page"] * 0.5 * 4 * row * size + 8 * b * width * 0.5 + 32 * b), flops=0)
    live = b * (0.5 * width + 0.5)
    pool = live / case["fill"]
    return dict(bytes=int(live * (1 - case["fill"]) * case["page"] * 4 * row * size + 8 * live + 4 * pool), flops=0)


def exact(case, seed):
    if case["op"] != "rotate":
        return None          # whole numbers and moved bits, held equal to the plain form's
    s = _prepare_rotate(case, seed)
    n, dim, half, page = case["tokens"], case["dim"], case["rot"] // 2, case["page"]
    pos = s["pos"].double().view(case["axes"], n)
    spin = torch.zeros(n, half, dtype=torch.complex128, device="cuda")
    for j in range(half):
        axis = 0 if s["axis_of"] is None else int(s["axis_of"][j])
        # the angle of far positions: reduced to one turn before its sine is taken
        turn = torch.remainder(pos[axis] * (float(s["freq"][j]) / (2 * math.pi)), 1.0)
        spin[:, j] = torch.polar(torch.ones_like(turn), turn * (2 * math.pi))

    def head(x, weight):
        x = x.double()
        if weight is not None:
            x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / dim + s["eps"]) * weight.double()
        first = torch.arange(half, device="cuda") if case["pairs"] == "halves" else 2 * torch.arange(half, device="cuda")
        second = first + (half if case["pairs"] == "halves" else 1)
        z = torch.complex(x[:, first], x[:, second]) * spin
        y = x.clone()
        y[:, first], y[:, second] = z.real, z.imag
        return y

    q = torch.stack([head(s["q"][:, g], s["norms"][0]) for g in range(s["q"].shape[1])], 1)
    slots = s["slots"].tolist()
    rows = torch.tensor([i for i, t in enumerate(slots) if t >= 0], dtype=torch.int64, device="cuda")
    where = torch.tensor([t for t in slots if t >= 0], dtype=torch.int64, device="cuda")
    pools = {}
    for name, new, weight, scale in (("k", s["k_new"], s["norms"][1], s["ks"]), ("v", s["v_new"], None, s["vs"])):
        pool = s[name].double() if scale is None else s[name].view(torch.float8_e4m3fn).double()
        for h in range(KV_HEADS):
            y = head(new[:, h], weight) if name == "k" else new[:, h].double()
            if scale is not None:
                y = (y / scale[h].double()).clamp(-448, 448)
            pool[torch.div(where, page, rounding_mode="floor"), where % page, h] = y[rows]
        pools[name] = pool
    return dict(q=q, **pools)
