"""The paged-cache operators on the GPU against plain 64-bit statements of them
(_pagedtest.py): page maps, row writes, tree attention, their refusals on the
device, and the three together over pages of a decoded bitstream."""
import math
import random

import pytest
import torch

from tests import _pagedtest as P
from lossless_kv_cache_scalar_gb300 import Coder, Layout, PagedKV, PagePool, PageTable, SKVError, synth

pytestmark = pytest.mark.gpu


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ page map

def map_inputs(rng, b, page, max_ctx, max_new, ended, spare=3, head=None):
    ctx, new, have = [], [], []
    for _ in range(b):
        c, w = rng.randint(0, max_ctx), rng.randint(0, max_new)
        h = -(-c // page) + rng.choice([0, 0, 1, 2])
        if rng.random() < ended:
            c, w = -1 - rng.randint(0, 5), 0
        ctx.append(c), new.append(w), have.append(h)
    width = max([1] + [max(h, -(-(max(c, 0) + w) // page)) for c, w, h in zip(ctx, new, have)]) + 1
    need = sum(max(0, -(-(c + w) // page) - h) for c, w, h in zip(ctx, new, have) if c >= 0)
    used = sum(have)
    pool = used + need + spare
    perm = list(range(pool))
    rng.shuffle(perm)
    table = [[-1] * width for _ in range(b)]
    at = 0
    for r, h in enumerate(have):
        table[r][:h] = perm[at:at + h]
        at += h
    free = [-1] * max(pool, 1)
    head = rng.randrange(len(free)) if head is None else head
    for i, p in enumerate(perm[at:]):
        free[(head + i) % len(free)] = p
    return ctx, new, have, table, free, [head, pool - at], pool, width


def run_map(page, pool, width, cap, ctx, new, table, have, free, state, status=0):
    t = i32(table) if table else torch.empty(0, width, dtype=torch.int32, device="cuda")
    pt = PageTable(t, page, pool)
    f = i32(free)
    out, so = i32([7] * len(ctx)), i32([7, 7])
    cu = i32([7] * (len(ctx) + 1))
    slots = torch.full((cap,), 7, dtype=torch.int64, device="cuda")
    pt.map_into(i32(ctx), i32(new), i32(have), f, i32(state), cu, slots, out, so)
    torch.cuda.synchronize()
    assert int(pt.status.item()) == status
    return t.tolist(), out.tolist(), f.tolist(), so.tolist(), cu.tolist(), slots.tolist()


@pytest.mark.parametrize("b,page,max_ctx,max_new,ended", [
    (1, 1, 0, 1, 0.0), (1, 256, 1000, 1, 0.0), (3, 16, 100, 0, 0.5), (8, 256, 4000, 1, 0.0), (33, 7, 50, 20, 0.3),
    (257, 16, 300, 64, 0.1), (1023, 5, 40, 9, 0.2), (1024, 1, 10, 3, 0.2), (1025, 64, 500, 30, 0.2), (2500, 24, 90, 61, 0.1),
    (5, 1000, 5000, 30000, 0.0), (40, 3, 20, 5, 1.0)])
def test_page_map(b, page, max_ctx, max_new, ended):
    rng = random.Random(b * 1000 + page)
    for cap_more in (0, 5, 9001):
        ctx, new, have, table, free, state, pool, width = map_inputs(rng, b, page, max_ctx, max_new, ended)
        cap = sum(new) + cap_more
        want = P.page_map(page, pool, width, cap, ctx, new, table, have, free, state)
        got = run_map(page, pool, width, cap, ctx, new, table, have, free, state)
        for name, x, y in zip(("table", "n_pages", "free", "state", "cu", "slots"), got, want):
            assert x == y, name


def test_page_map_without_requests():
    got = run_map(16, 4, 3, 5, [], [], [], [], [0, 1, 2, 3], [1, 4])
    assert got == ([], [], [0, 1, 2, 3], [1, 4], [0], [-1] * 5)


def test_page_map_far_slots():
    """Slots beyond 2^31: pages of 2^20 tokens with large numbers."""
    big = 2 ** 31 - 8
    got = run_map(1 << 20, 2 ** 31 - 1, 2, 4, [(1 << 20) - 2], [4], [[big, -1]], [1], [big + 1, big + 2], [0, 2])
    p = (big << 20) + (1 << 20) - 2
    assert got[5] == [p, p + 1, (big + 1) << 20, ((big + 1) << 20) + 1]
    assert got[0] == [[big, big + 1]] and got[1] == [2] and got[3] == [1, 1]


BAD_MAPS = [
    (1, dict(new=[2, -1])), (1, dict(ctx=[-1, 3], new=[1, 1])), (1, dict(have=[-1, 1])), (1, dict(have=[9, 1])),
    (1, dict(ctx=[33, 3])), (1, dict(ctx=[2 ** 31 - 1, 3], new=[1, 1])), (1, dict(state=[8, 4])), (1, dict(state=[-1, 4])),
    (1, dict(state=[0, 9])), (1, dict(state=[0, -1])), (6, dict(state=[0, 0])), (6, dict(new=[17, 1])),
    (6, dict(new=[60, 1], state=[0, 8])), (6, dict(ctx=[-1, 3], new=[0, 1], state=[0, 8]))]


@pytest.mark.parametrize("cap", [16, 20000])
@pytest.mark.parametrize("status,change", BAD_MAPS)
def test_page_map_refuses_bad_lengths(status, change, cap):
    """Nothing but the counts is written, and those as they were (one CTA and many)."""
    s = dict(ctx=[30, 3], new=[4, 1], have=[2, 1], state=[2, 4])
    s.update(change)
    if cap > 16 and change == dict(new=[17, 1]):
        pytest.skip("fits the larger slot map")
    table, free = [[0, 1, -1, -1], [2, -1, -1, -1]], [5, 6, 3, 4, 5, 6, 7, 7]
    got = run_map(16, 8, 4, cap, s["ctx"], s["new"], table, s["have"], free, s["state"], status)
    assert got == (table, s["have"], free, s["state"], [0, 0, 0], [-1] * cap)


@pytest.mark.parametrize("cap", [16, 20000])
def test_page_map_bad_page_numbers(cap):
    """Slots on pages outside the pool are -1 and reported; the rest of the map stands."""
    table, free = [[0, 1, -1], [9, -1, -1], [-5, 2, -1]], [4, 8, -7, 3]
    got = run_map(4, 8, 3, cap, [7, 3, -1], [3, 1, 0], table, [2, 1, 1], free, [1, 2], 7)
    # request 0: position 7 on page 1, 8 and 9 on a new page 8 (outside); request 1 on page 9
    assert got[0] == [[0, 1, 8], [9, -1, -1], [-5, 2, -1]]
    assert got[5] == [7, -1, -1, -1] + [-1] * (cap - 4)
    assert got[1] == [3, 1, 0] and got[3] == [2, 2] and got[2] == [4, 8, -7, -5]


def test_page_pool_steps():
    """Several steps of a pool with requests that grow, end and start again: no page is
    held twice, and every step's map is the plain one's."""
    rng = random.Random(5)
    b, page, pool = 6, 4, 40
    pp = PagePool(b, 12, page, pool)
    ctx = [0] * b
    for step in range(30):
        new = [rng.randint(0, 5) for _ in range(b)]
        n_pages, state = pp.n_pages.tolist(), pp.free_state.tolist()
        for r in range(b):
            if ctx[r] + new[r] > 40 or rng.random() < 0.1:
                ctx[r], new[r] = -1, 0
        room = state[1]
        for r in range(b):
            if ctx[r] >= 0:
                grow = max(0, -(-(ctx[r] + new[r]) // page) - n_pages[r])
                if grow > room:
                    new[r] = 0
                else:
                    room -= grow
        want = P.page_map(page, pool, 12, 32, ctx, new, pp.block_table.tolist(), n_pages, pp.free_pages.tolist(), state)
        cu, slots = pp.step(i32(ctx), i32(new), 32)
        assert (pp.block_table.tolist(), pp.n_pages.tolist(), pp.free_pages.tolist(), pp.free_state.tolist(), cu.tolist(),
                slots.tolist()) == want
        held = [p for r, n in enumerate(want[1]) for p in want[0][r][:n]]
        head, count = want[3]
        held += [want[2][(head + i) % pool] for i in range(count)]
        assert sorted(held) == list(range(pool))
        ctx = [0 if c < 0 else c + rng.randint(0, w) for c, w in zip(ctx, new)]


# ------------------------------------------------------------------ append

def pool_of(pages, page, heads, dim, dtype, gen, layout="thd"):
    """A pool of random codes in one of several orders and strides."""
    shape = {"thd": (pages, page, heads, dim), "htd": (pages, heads, page, dim), "wide": (pages, page, heads + 1, dim + 16),
             "kv": (pages, 2, page, heads, dim)}[layout]
    x = torch.randn(shape, generator=gen, device="cuda")
    t = x.to(torch.bfloat16) if dtype == "bf16" else (x * 100).clamp(-448, 448).to(P.E4M3).view(torch.uint8)
    if layout == "htd":
        return t.permute(0, 2, 1, 3)
    if layout == "wide":
        return t[:, :, :heads, :dim]
    if layout == "kv":
        return t[:, 1]
    return t


def gen_of(seed):
    g = torch.Generator("cuda")
    g.manual_seed(seed)
    return g


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("n,page,heads,dim,layout,use_rows", [
    (0, 16, 2, 64, "thd", False), (1, 1, 1, 16, "thd", False), (8, 256, 8, 128, "thd", False), (61, 7, 3, 48, "htd", True),
    (300, 24, 8, 128, "kv", False), (2049, 16, 2, 80, "wide", True), (5000, 64, 4, 256, "thd", False)])
def test_append(dtype, n, page, heads, dim, layout, use_rows):
    g = gen_of(n + dim)
    rng = random.Random(n)
    pages = n // page + 3
    k, v = (pool_of(pages, page, heads, dim, dtype, g, layout) for _ in range(2))
    ks = vs = None
    if dtype == "e4m3":
        ks, vs = (torch.rand(heads, generator=g, device="cuda") * 0.02 + 0.003 for _ in range(2))
    n_src = n + 5
    wide = torch.randn(n_src, 3 * heads + 1, dim, generator=g, device="cuda").to(torch.bfloat16)
    if n_src * dim > 64:                              # the values that rounding and saturation meet
        wide[0, :, 0], wide[0, :, 1], wide[0, :, 2], wide[0, :, 3] = math.inf, -math.inf, math.nan, -0.0
        wide[0, :, 4], wide[0, :, 5] = 1e-30, 3e38
    new_k, new_v = wide[:, heads:2 * heads], wide[:, 2 * heads:3 * heads]
    slots = rng.sample(range(pages * page), n)
    for i in range(0, n, 9):
        slots[i] = -1 if i % 2 else slots[i]
    rows = [rng.randrange(n_src) for _ in range(n)] if use_rows else None
    cache = PagedKV(k, v, k_scale=ks, v_scale=vs)
    want_k, want_v = k.cpu().clone(), v.cpu().clone()
    for want, new, sc in ((want_k, new_k, ks), (want_v, new_v, vs)):
        for i, s in enumerate(slots):
            if s >= 0:
                x = new[rows[i] if rows else i].cpu()
                if sc is not None:
                    x = P.to_e4m3(x.double() / sc.cpu().double()[:, None])
                want[s // page, s % page] = x
    cache.append(new_k, new_v, torch.tensor(slots, dtype=torch.int64, device="cuda"), None if rows is None else i32(rows))
    bits = torch.int16 if dtype == "bf16" else torch.uint8
    for got, want in ((k, want_k), (v, want_v)):
        got, want = got.cpu().contiguous().view(bits), want.contiguous().view(bits)
        if dtype == "e4m3":                           # NaN: either sign
            got, want = (torch.where((t & 127) == 127, torch.full_like(t, 127), t) for t in (got, want))
        assert torch.equal(got, want)


def test_append_rounds_the_real_quotient():
    """Scales s for which some bf16 x has x / s next to a tie of the 8-bit grid, nearer
    than binary32 resolves: the code is the real quotient's."""
    xs = torch.arange(0x3F80, 0x4000, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)   # 1 .. 2
    ties = torch.tensor([1.0625, 1.1875, 1.3125, 1.4375, 1.5625, 1.6875, 1.8125], dtype=torch.float64)
    s = (xs.double()[:, None] / ties).flatten().float()                     # fl32(x / tie): quotients all but ties
    s = torch.cat([s, torch.nextafter(s, torch.full_like(s, 9.0)), torch.nextafter(s, torch.zeros_like(s))])
    heads = s.numel()
    k = torch.zeros(1, 1, heads, 16, dtype=torch.uint8, device="cuda")
    v = torch.zeros_like(k)
    near = xs.repeat_interleave(7).repeat(3)
    new = near.view(1, heads, 1).expand(1, heads, 16).contiguous().cuda()
    PagedKV(k, v, k_scale=s.cuda(), v_scale=s.cuda()).append(new, -new, torch.zeros(1, dtype=torch.int64, device="cuda"))
    want = P.to_e4m3(near.double() / s.double())
    assert torch.equal(k[0, 0, :, 0].cpu(), want) and torch.equal(v[0, 0, :, 5].cpu(), want | 128)


@pytest.mark.parametrize("n", [40, 3000])
@pytest.mark.parametrize("what", ["slot", "row", "short"])
def test_append_reports_bad_slots_and_rows(n, what):
    g = gen_of(3)
    k, v = (pool_of(n // 16 + 2, 16, 2, 64, "bf16", g) for _ in range(2))
    cache = PagedKV(k, v)
    new = torch.randn(n if what != "short" else n - 1, 2, 64, generator=g, device="cuda").to(torch.bfloat16)
    slots = torch.arange(n, dtype=torch.int64, device="cuda")
    rows = None
    if what == "slot":
        slots[n - 3] = (n // 16 + 2) * 16
    if what == "row":
        rows = torch.arange(n, dtype=torch.int32, device="cuda")
        rows[n - 3] = n
    before = k.clone()
    with pytest.raises(SKVError) as e:
        cache.append(new, new, slots, rows)
    assert e.value.name == "INVALID_ARG"
    bad = n - 1 if what == "short" else n - 3
    flat, old = k.view(-1, 2, 64), before.view(-1, 2, 64)
    good = torch.tensor([i for i in range(n) if i != bad], device="cuda")
    assert torch.equal(flat[good], new[good])
    assert torch.equal(flat[bad], old[bad]) and torch.equal(flat[n:], old[n:])
    cache.append(new[:1], new[:1], slots[:1])           # the next call's status is its own


# ------------------------------------------------------------------ attention

def attend_case(seed, ctx, new, page, heads, group, dim, dtype, layout="thd", tree=True, words=None, garbage=None,
                spread=2.0):
    """Random pools, tables, queries and trees; pages past the lengths hold `garbage`."""
    g, rng = gen_of(seed), random.Random(seed)
    b = len(ctx)
    need = [-(-(max(c, 0) + n) // page) for c, n in zip(ctx, new)]
    width, total = max(need + [1]) + 1, sum(need) + 2
    perm = list(range(total))
    rng.shuffle(perm)
    table, at = [[-1] * width for _ in range(b)], 0
    for r in range(b):
        table[r][:need[r]] = perm[at:at + need[r]]
        at += need[r]
    k, v = (pool_of(total, page, heads, dim, dtype, g, layout) for _ in range(2))
    if garbage is not None:
        code = {"bf16": torch.tensor(garbage, dtype=torch.bfloat16), "e4m3": torch.tensor(127, dtype=torch.uint8)}[dtype]
        for pool in (k, v):
            for p in perm[at:]:
                pool[p] = code
            for r in range(b):
                end = max(ctx[r], 0) + new[r]
                if need[r] and end % page:
                    pool[table[r][end // page], end % page:] = code
    ks = vs = None
    if dtype == "e4m3":
        ks, vs = (torch.rand(heads, generator=g, device="cuda") * 0.01 + 0.005 for _ in range(2))
    rows = sum(new) + 3
    q = (torch.randn(rows, heads * group + 2, dim, generator=g, device="cuda") * spread).to(torch.bfloat16)[:, 1:-1]
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    mask = None
    if tree:
        bits = []
        for n in new:
            bits += P.tree_bits([rng.randint(-1, i - 1) for i in range(n)])
        mask = P.mask_tensor(bits + [0] * 3, words or max(1, -(-max(new + [1]) // 64))).cuda()
    return dict(q=q, k=k, v=v, ks=ks, vs=vs, table=i32(table), ctx=i32(ctx), cu=i32(cu), mask=mask)


def check_attend(s, scale=None, max_nodes=None, want_status=0):
    heads, dim = s["q"].shape[1], s["q"].shape[2]
    sc = 1.0 / math.sqrt(dim) if scale is None else scale
    cache = PagedKV(s["k"], s["v"], s["table"], k_scale=s["ks"], v_scale=s["vs"])
    out = torch.full(s["q"].shape, 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full(s["q"].shape[:2], 7.0, device="cuda")
    cache.attend_into(s["q"], s["ctx"], s["cu"], out, mask=s["mask"], max_nodes=max_nodes, scale=scale, lse=lse)
    torch.cuda.synchronize()
    assert int(cache.status.item()) == want_status
    # an 8-bit cache: weights in fp16, and queries that may be carried in fp16 below 2^-25 of their largest
    eps = dict(q_eps=2.0 ** -16, p_eps=2.0 ** -11) if s["ks"] is not None else {}
    o, tol, l, l_tol = P.attention(s["q"], s["k"], s["v"], s["ks"], s["vs"], s["table"], s["ctx"], s["cu"], s["mask"], sc, **eps)
    got, gl = out.cpu().double(), lse.cpu().double()
    dead = torch.isnan(l) & torch.isnan(l_tol)
    assert (got[dead] == 7.0).all() and (gl[dead] == 7.0).all()
    live = ~dead
    assert not torch.isnan(got[live] - o[live]).any()
    over = ((got - o).abs() - tol)[live]
    assert (over <= 0).all(), float(over.max())
    fin = live & torch.isfinite(l)
    assert ((gl - l).abs() <= l_tol)[fin].all()
    assert (gl[live & ~fin] == -math.inf).all()
    again = torch.full_like(out, 7.0)
    cache.attend_into(s["q"], s["ctx"], s["cu"], again, mask=s["mask"], max_nodes=max_nodes, scale=scale)
    assert torch.equal(again, out)                       # the same bits, with and without lse
    return out


SHAPES = [
    # ctx, new, page, heads, group, dim
    ([0], [1], 16, 1, 1, 16), ([1], [1], 1, 2, 4, 64), ([1000], [1], 256, 8, 4, 128), ([127, 0, 5], [1, 1, 1], 64, 2, 8, 128),
    ([63, 64, 65, 128], [1, 2, 16, 3], 16, 2, 2, 64), ([300, 17], [27, 9], 24, 2, 5, 128), ([0, 0], [33, 64], 7, 1, 8, 96),
    ([511, 40], [60, 61], 64, 2, 8, 128), ([700], [64], 256, 1, 8, 256), ([50, -1, 20, 90], [3, 0, 0, 70], 5, 2, 3, 48),
    ([129], [130], 24, 1, 2, 128), ([37], [1], 16, 2, 16, 80), ([90], [5], 32, 1, 71, 64), ([200] * 40, [2] * 40, 16, 2, 4, 64)]


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("tree", [True, False])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_attend(shape, tree, dtype):
    ctx, new, page, heads, group, dim = SHAPES[shape]
    s = attend_case(shape + 100, ctx, new, page, heads, group, dim, dtype, tree=tree)
    check_attend(s, max_nodes=max(new))


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("hint", [1, 4, 100000])
def test_attend_max_nodes_is_only_a_hint(hint, dtype):
    s = attend_case(7, [100, 40], [21, 3], 16, 2, 4, 128, dtype)
    check_attend(s, max_nodes=hint)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("nodes", [1, 40])
@pytest.mark.parametrize("layout", ["htd", "wide", "kv"])
def test_attend_pool_orders(layout, nodes, dtype):
    s = attend_case(11, [77, 300], [nodes, nodes], 16, 2, 4, 128, dtype, layout=layout)
    check_attend(s, max_nodes=nodes)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("nodes", [2, 60])
def test_attend_empty_rows(nodes, dtype):
    """No context and masks that leave rows nothing at all: exactly 0, log-sum -inf."""
    s = attend_case(13, [0, 20, 0], [nodes, nodes, 1], 8, 2, 8, 64, dtype)
    s["mask"][0] = 0
    s["mask"][nodes - 1] = 0
    s["mask"][2 * nodes] = 0
    out = check_attend(s, max_nodes=nodes)
    assert (out[0] == 0).all() and (out[2 * nodes] == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("nodes,group", [(1, 4), (6, 2), (50, 8)])
def test_attend_ignores_what_lies_past_the_lengths(nodes, group, bad, dtype):
    s = attend_case(17, [130, 9], [nodes, nodes], 24, 2, group, 128, dtype, garbage=bad)
    check_attend(s, max_nodes=nodes)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("nodes,group,ctx", [(6, 2, 100), (50, 8, 250), (64, 8, 1), (9, 8, 0)])
def test_attend_masked_positions_have_no_effect(nodes, group, ctx, bad, dtype):
    """A node whose K and V are not finite changes nothing for the rows that do not see it,
    and spoils the ones that do."""
    s = attend_case(19, [ctx], [nodes], 16, 2, group, 128, dtype)
    hurt = 3
    s["mask"][:, 0] &= ~(1 << hurt)                  # none sees it ...
    clean = check_attend(s, max_nodes=nodes)
    pos = ctx + hurt
    code = torch.tensor(bad, dtype=torch.bfloat16) if dtype == "bf16" else torch.tensor(127, dtype=torch.uint8)
    page = int(s["table"][0, pos // 16])
    keep_k = s["k"][page, pos % 16].clone()
    s["k"][page, pos % 16] = code
    s["v"][page, pos % 16, :, 5:9] = code
    cache = PagedKV(s["k"], s["v"], s["table"], k_scale=s["ks"], v_scale=s["vs"])

    def run():
        return cache.attend(s["q"], s["ctx"], s["cu"], mask=s["mask"], max_nodes=nodes)[:nodes]

    assert torch.equal(run(), clean[:nodes])
    s["mask"][nodes - 1, 0] |= 1 << hurt             # ... now the last row does
    s["k"][page, pos % 16] = keep_k
    got = run()
    assert torch.equal(got[:nodes - 1], clean[:nodes - 1])
    seen = got[nodes - 1].float()
    assert not torch.isfinite(seen[:, 5:9]).any()
    if dtype == "bf16" and not math.isnan(bad):
        assert (seen[:, 5:9] == bad).all()
    assert torch.isfinite(seen[:, :5]).all() and torch.isfinite(seen[:, 9:]).all()


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("nodes", [1, 40])
def test_attend_scores_of_great_spread(nodes, dtype):
    """Scores in the thousands: the running maximum moves, most weights vanish; and scale 0
    and a negative scale."""
    s = attend_case(23, [500, 33], [nodes, nodes], 16, 2, 4, 64, dtype, spread=200.0)
    check_attend(s, max_nodes=nodes)
    check_attend(s, max_nodes=nodes, scale=0.0)
    check_attend(s, max_nodes=nodes, scale=-0.01)


@pytest.mark.parametrize("nodes", [1, 40])
def test_attend_lowest_values(nodes):
    """Keys that push scores to -infinity and to the type's lowest: rows keep the rest."""
    s = attend_case(29, [40], [nodes], 16, 1, 4, 64, "bf16", spread=1.0)
    low = torch.finfo(torch.bfloat16).min
    page = int(s["table"][0, 0])
    s["q"][:, :, 0] = 1.0
    s["k"][page, 3, :, :], s["k"][page, 5, :, :] = 0.0, 0.0
    s["k"][page, 3, :, 0] = low                       # a score of about -4e37
    s["k"][page, 5, :, 0] = -math.inf                 # a score of -infinity: weight 0
    s["v"][page, 5] = 0.0
    out = torch.full(s["q"].shape, 7.0, dtype=torch.bfloat16, device="cuda")
    cache = PagedKV(s["k"], s["v"], s["table"])
    cache.attend_into(s["q"], s["ctx"], s["cu"], out, mask=s["mask"], max_nodes=nodes)
    cache.check_status("attend")
    # the same with those two positions' weights made 0 by a finite, very low score
    s["k"][page, 3, :, 0], s["k"][page, 5, :, 0] = -1e30, -1e30
    check_attend(s, max_nodes=nodes)
    o, tol, _, _ = P.attention(s["q"], s["k"], s["v"], None, None, s["table"], s["ctx"], s["cu"], s["mask"], 0.125)
    assert ((out.cpu().double() - o).abs() <= tol)[:nodes].all()


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("nodes,ctx", [(1, 20000), (63, 9000)])
def test_attend_long_contexts(nodes, ctx, dtype):
    """Work split over the context and joined."""
    s = attend_case(31, [ctx], [nodes], 256, 1, 2, 128, dtype)
    check_attend(s, max_nodes=nodes)


def test_attend_beyond_32_bits():
    """A pool of more than 2^32 bytes and codes, with the pages in use at its far end."""
    page, heads, dim = 256, 8, 128
    pages = 16500                                     # 4.3e9 codes
    k = torch.zeros(pages, page, heads, dim, dtype=torch.uint8, device="cuda")
    g = gen_of(37)
    small = attend_case(37, [400, 30], [3, 40], page, heads, 2, dim, "e4m3")
    n = small["k"].shape[0]
    k[-n:] = small["k"]
    v = torch.zeros_like(k)
    v[-n:] = small["v"]
    far = PagedKV(k, v, torch.where(small["table"] >= 0, small["table"] + pages - n, small["table"]), k_scale=small["ks"],
                  v_scale=small["vs"])
    near = PagedKV(small["k"], small["v"], small["table"], k_scale=small["ks"], v_scale=small["vs"])
    args = (small["q"], small["ctx"], small["cu"], small["mask"], 40)
    assert torch.equal(far.attend(*args), near.attend(*args))
    new = torch.randn(5, heads, dim, generator=g, device="cuda").to(torch.bfloat16)
    at = torch.tensor([pages * page - 1 - 7 * i for i in range(5)], dtype=torch.int64, device="cuda")
    far.append(new, new, at)
    near.append(new, new, at - (pages - n) * page)
    assert torch.equal(k[-n:], small["k"]) and torch.equal(v[-n:], small["v"])


@pytest.mark.parametrize("nodes", [1, 40])
def test_attend_bad_requests_are_reported_and_left_alone(nodes):
    base = attend_case(41, [90, 50, 30], [nodes, nodes, nodes], 16, 2, 4, 64, "bf16")
    good = check_attend(base, max_nodes=nodes)
    cache = PagedKV(base["k"], base["v"], base["table"])

    def run(**kw):
        s = dict(base, **kw)
        out = torch.full_like(good, 7.0)
        cache.attend_into(s["q"], s["ctx"], s["cu"], out, mask=s["mask"], max_nodes=nodes)
        torch.cuda.synchronize()
        return out, int(cache.status.item())

    def close(x, y):
        # each is within 2^-8 (|o| + A) of the truth and a little more, A < 5.5
        return ((x.float() - y.float()).abs() <= 2.0 ** -7 * (y.float().abs() + 6)).all()

    out, st = run(ctx=i32([90, -2, 30]))
    assert st == 1 and (out[nodes:2 * nodes] == 7).all()
    assert close(out[:nodes], good[:nodes]) and close(out[2 * nodes:], good[2 * nodes:])
    out, st = run(ctx=i32([90, 100000, 30]))
    assert st == 1 and (out[nodes:2 * nodes] == 7).all() and close(out[:nodes], good[:nodes])
    out, st = run(ctx=i32([90, 2 ** 31 - 1, 30]))
    assert st == 1 and close(out[2 * nodes:], good[2 * nodes:])
    out, st = run(cu=i32([0, nodes, 10 ** 6, 3 * nodes]))
    assert st == 1 and close(out[:nodes], good[:nodes]) and (out[nodes:] == 7).all()
    out, st = run(cu=i32([-5, nodes, 2 * nodes, 3 * nodes]))
    assert st == 1 and (out[:nodes] == 7).all() and close(out[nodes:], good[nodes:])
    table = base["table"].clone()
    for bad in (-1, 10 ** 6, 2 ** 31 - 1):
        base["table"][1, 2] = bad
        out, st = run()
        assert st == 7
        assert torch.equal(out[:nodes], good[:nodes]) and torch.equal(out[2 * nodes:], good[2 * nodes:])
    base["table"].copy_(table)
    out, st = run()
    assert st == 0 and torch.equal(out, good)


def test_attend_more_nodes_than_mask_bits():
    s = attend_case(43, [10], [65], 16, 1, 1, 64, "bf16")
    s["mask"] = s["mask"][:, :1].contiguous()
    cache = PagedKV(s["k"], s["v"], s["table"])
    with pytest.raises(SKVError) as e:
        cache.attend(s["q"], s["ctx"], s["cu"], mask=s["mask"])
    assert e.value.name == "INVALID_ARG"


@pytest.mark.parametrize("nodes", [1, 33])
def test_on_another_stream_and_in_a_graph(nodes):
    """All three captured on a stream of their own, replayed on changed inputs."""
    b, page, heads, group, dim, pool = 3, 16, 2, 4, 128, 64
    g = gen_of(47)
    table = torch.full((b, 20), -1, dtype=torch.int32, device="cuda")
    pt = PageTable(table, page, pool)
    k, v = (pool_of(pool, page, heads, dim, "bf16", g) for _ in range(2))
    cache = PagedKV(k, v, table, q_heads=heads * group)
    free, state, state2 = torch.arange(pool, dtype=torch.int32, device="cuda"), i32([0, pool]), i32([0, 0])
    ctx, new, have, have2, cu = i32([0] * b), i32([0] * b), i32([0] * b), i32([0] * b), i32([0] * (b + 1))
    rows = b * nodes
    slots = torch.empty(rows, dtype=torch.int64, device="cuda")
    kn, vn = (torch.zeros(rows, heads, dim, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q = torch.zeros(rows, heads * group, dim, dtype=torch.bfloat16, device="cuda")
    out = torch.zeros_like(q)

    def step():
        pt.map_into(ctx, new, have, free, state, cu, slots, have2, state2)
        cache.append_into(kn, vn, slots)
        cache.attend_into(q, ctx, cu, out, max_nodes=nodes)
        have.copy_(have2)
        state.copy_(state2)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    lens = [0] * b
    for turn in range(4):
        n = [nodes if (turn + r) % 3 else 1 for r in range(b)]
        new.copy_(i32(n))
        ctx.copy_(i32(lens))
        for t in (kn, vn, q):
            t.copy_(torch.randn(t.shape, generator=g, device="cuda"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert int(pt.status.item()) == 0 and int(cache.status.item()) == 0
        total = sum(n)
        assert cu.tolist()[-1] == total
        o, tol, _, _ = P.attention(q, k, v, None, None, table, ctx, cu, None, 1.0 / math.sqrt(dim))
        assert ((out.cpu().double() - o).abs() <= tol)[:total].all()
        flat = k.view(-1, heads, dim)
        assert torch.equal(flat[slots[:total]], kn[:total])
        lens = [l + x for l, x in zip(lens, n)]


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_over_decoded_pages(dtype):
    """The coder's pages are the cache: K and V pages decoded out of order into one
    buffer, read in place by the attention of a drafted tree appended behind them."""
    T, page, heads, group, dim, nodes = 600, 256, 8, 2, 128, 12
    cfg = synth.CONFIGS["tiny" if dtype == "bf16" else "fp8_32b"].scaled(n_layers=1, n_tokens=T)
    w = {k: v.cuda() for k, v in synth.generate(cfg).items()}
    lay = Layout(dtype, 1, 2, heads, dim, T, tokens_per_chunk=page)
    coder = Coder(lay)
    w["kv"] = w["mu"].clone()                         # no outlier codes: scores in the usual range
    bits, offs = coder.encode(w["kv"], w["mu"], w["sigma"], w["counts"])
    ids = i32([2, 0, 1, 5, 3, 4])                     # pages 2 0 1 of K, then of V
    got = coder.decode_chunks(bits, offs, w["mu"], w["sigma"], w["counts"], ids)
    pool = got.view(2, 3, page, heads, dim)
    table = i32([[1, 2, 0]])
    scale = torch.full((heads,), 0.01, device="cuda") if dtype == "e4m3" else None
    cache = PagedKV(pool[0], pool[1], table, k_scale=scale, v_scale=scale)
    g = gen_of(53)
    new_k, new_v = (torch.randn(nodes, heads, dim, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    q = torch.randn(nodes, heads * group, dim, generator=g, device="cuda").to(torch.bfloat16)
    slots = torch.arange(T - 2 * page, T - 2 * page + nodes, dtype=torch.int64, device="cuda")       # page 0 of the pool
    cache.append(new_k, new_v, slots)
    full = torch.cat([w["kv"].view(2, T, heads, dim), torch.stack([pool[0], pool[1]])[:, 0, T - 2 * page:T - 2 * page + nodes]
                      .view(w["kv"].dtype)], 1)
    mask = P.mask_tensor(P.tree_bits([-1, 0, 0, 1, 1, 2, -1, 6, 7, 7, 4, 10]), 1).cuda()
    ctx, cu = i32([T]), i32([0, nodes])
    out = cache.attend(q, ctx, cu, mask=mask, max_nodes=nodes)
    whole = full.unsqueeze(1)                          # one page of T + nodes tokens each
    codes = torch.uint8 if dtype == "e4m3" else torch.bfloat16
    eps = dict(q_eps=2.0 ** -16, p_eps=2.0 ** -11) if dtype == "e4m3" else {}
    o, tol, _, _ = P.attention(q, whole[0].view(codes), whole[1].view(codes), scale, scale, i32([[0]]), ctx, cu, mask,
                               1.0 / math.sqrt(dim), **eps)
    assert ((out.cpu().double() - o).abs() <= tol).all()


@pytest.mark.parametrize("dtype,dim", [("bf16", 128), ("bf16", 48), ("e4m3", 128), ("e4m3", 64)])
@pytest.mark.parametrize("page", [1, 8, 12, 40, 48, 72, 104, 120, 136, 256])
def test_attend_page_lengths(page, dtype, dim):
    """Tiles of whole pages, of parts of pages, and of rows one by one, over several tiles and
    with rows past the pages' ends that hold NaN."""
    s = attend_case(59 + page, [333, 130, 7], [9, 33, 40], page, 2, 4, dim, dtype, garbage=math.nan)
    check_attend(s, max_nodes=40)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("hint", [1, 1000])
def test_attend_many_requests(hint, dtype):
    """More requests than a CTA has threads, some idle, and far more than there are shares."""
    rng = random.Random(61)
    ctx = [rng.choice([0, 1, 5, 30, 140]) for _ in range(1300)]
    new = [rng.choice([0, 1, 1, 2]) for _ in range(1300)]
    ctx = [-1 if n == 0 and c == 5 else c for c, n in zip(ctx, new)]
    s = attend_case(61, ctx, new, 16, 1, 1, 64, dtype)
    check_attend(s, max_nodes=hint)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("ctx,new", [([0], [1]), ([0, 0, 0], [1, 0, 2]), ([127], [1]), ([128], [1])])
def test_attend_least_work(ctx, new, dtype):
    """One or two tiles in all, through the kernel for many rows."""
    s = attend_case(67, ctx, new, 16, 1, 2, 128, dtype)
    check_attend(s, max_nodes=1000)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_attend_wide_and_narrow_row_tiles(dtype):
    """Row tiles of 256, 129, 128 and 1 rows in one call, cut by the shares' ends."""
    s = attend_case(71, [3000, 2500, 1400, 700], [96, 43, 32, 65], 64, 1, 4, 64, dtype)
    check_attend(s, max_nodes=96)



def test_wrappers_refuse_wrong_tensors():
    """Types, shapes, strides and devices that the C ABI cannot see are refused before a call."""
    s = attend_case(73, [9, 3], [2, 1], 16, 2, 2, 64, "bf16")
    cache = PagedKV(s["k"], s["v"], s["table"], q_heads=4)
    q, ctx, cu, mask = s["q"], s["ctx"], s["cu"], s["mask"]
    out = torch.empty(q.shape, dtype=torch.bfloat16, device="cuda")
    for bad in (dict(q=q.float()), dict(q=q.cpu()), dict(q=q[:, :3]), dict(q=q[..., :32]), dict(q=q.transpose(0, 1)),
                dict(out=out.float()), dict(out=out[:-1]), dict(out=out.transpose(0, 1)), dict(ctx=ctx.long()), dict(ctx=ctx[:1]),
                dict(cu=cu[:-1]), dict(cu=cu.cpu()), dict(mask=mask[:-1]), dict(mask=mask.int()), dict(mask=mask[:, :0]),
                dict(lse=torch.empty(3, device="cuda"))):
        a = dict(dict(q=q, ctx=ctx, cu=cu, out=out, mask=mask, lse=None), **bad)
        with pytest.raises(ValueError):
            cache.attend_into(a["q"], a["ctx"], a["cu"], a["out"], mask=a["mask"], lse=a["lse"])
    with pytest.raises(ValueError):
        PagedKV(s["k"], s["v"]).attend_into(q, ctx, cu, out)
    new, slots = torch.zeros(3, 2, 64, dtype=torch.bfloat16, device="cuda"), torch.arange(3, dtype=torch.int64, device="cuda")
    rows = i32([0, 1, 2])
    for k, v, sl, r in ((new.float(), new.float(), slots, None), (new, new[:2], slots, None), (new[:, :1], new[:, :1], slots, None),
                        (new, new.cpu(), slots, None), (new, new, slots.int(), None), (new, new, slots, rows[:2]),
                        (new, new, slots, rows.long())):
        with pytest.raises(ValueError):
            cache.append_into(k, v, sl, rows=r)
    for k, v in ((s["k"].float(), s["v"].float()), (s["k"][:-1], s["v"]), (s["k"].view(torch.int16)[..., ::2], s["v"].view(torch.int16)[..., ::2])):
        with pytest.raises(ValueError):
            PagedKV(k, v, s["table"])
    with pytest.raises(ValueError):
        PagedKV(s["k"], s["v"], s["table"].t())
    with pytest.raises(SKVError):                      # scales of a bf16 cache
        one = torch.ones(2, device="cuda")
        PagedKV(s["k"], s["v"], s["table"], k_scale=one, v_scale=one)
    pt = PageTable(s["table"], 16, s["k"].shape[0])
    with pytest.raises(ValueError):
        pt.map_into(ctx.long(), ctx, ctx, ctx, ctx, cu, slots, ctx, ctx)
    with pytest.raises(SKVError):                      # counts read and written in place
        pt.map_into(ctx, ctx, ctx, i32([0]), i32([0, 1]), cu, slots, ctx, i32([0, 0]))
