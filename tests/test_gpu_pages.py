"""Forks, compaction, copies and moves of pages and tokens, against plain lists."""
import random

import pytest
import torch

from tests._servetest import compact, fork
from lossless_kv_cache_scalar_gb300 import PagedKV, PagePool, PageTable, SKVError

pytestmark = pytest.mark.gpu


def i32(v):
    return torch.tensor(v, dtype=torch.int32).cuda()


def tables(rng, n, width, page, share=True, idle=0.2, extra=0.3):
    """Random rows over a pool, some of them with a common beginning, and what is free."""
    ctx, have, rows = [], [], []
    pool = n * width + rng.randint(1, 20)
    order = list(range(pool))
    rng.shuffle(order)
    for r in range(n):
        c = -1 if rng.random() < idle else rng.randint(0, width * page - 1)
        h = 0 if c < 0 and rng.random() < 0.7 else max(0, -(-c // page))
        if h < width and rng.random() < extra:
            h += rng.randint(1, width - h)
        row = [order.pop() for _ in range(h)]
        if share and r and rng.random() < 0.4:
            o = rng.randrange(r)
            m = min(h, max(0, c) // page, max(0, ctx[o]) // page, have[o])
            row[:m] = rows[o][:m]
        ctx.append(c)
        have.append(h)
        rows.append(row)
    held = {p for row in rows for p in row}
    free = [p for p in range(pool) if p not in held]
    rng.shuffle(free)
    return ctx, have, rows, free, pool


def block_table(rows, width):
    return i32([r + [-9] * (width - len(r)) for r in rows]) if width else torch.zeros(len(rows), 0, dtype=torch.int32, device="cuda")


def ring_of(rng, free, size):
    head = rng.randrange(size)
    ring = [-5] * size
    for i, p in enumerate(free):
        ring[(head + i) % size] = p
    return ring, [head, len(free)]


def call_fork(page, pool, parents, ctx, rows, have, width, ring, state, trim):
    n = len(ctx)
    t = PageTable(block_table(rows, width), page, pool, workspace=True)
    t.workspace.fill_(255)
    out = dict(table_out=torch.full((n, width), -9, dtype=torch.int32, device="cuda"), n_pages_out=i32([-9] * n), ctx_out=i32([-9] * n),
               free_state_out=i32([-9, -9]), copy_src=i32([-9] * n), copy_dst=i32([-9] * n), copy_tokens=i32([-9] * n))
    free = i32(ring)
    t.fork_into(None if parents is None else i32(parents), i32(ctx), i32(have), free, i32(state), trim=trim, **out)
    torch.cuda.synchronize()
    got = {k: v.tolist() for k, v in out.items()}
    got["free"] = free.tolist()
    return got, int(t.status)


def check_fork(got, want, width):
    rows, have, ctx, ring, state, copies = want
    assert got["n_pages_out"] == have
    assert got["ctx_out"] == ctx
    assert got["table_out"] == [r + [-9] * (width - len(r)) for r in rows]
    assert got["free"] == ring
    assert got["free_state_out"] == state
    assert list(zip(got["copy_src"], got["copy_dst"], got["copy_tokens"])) == copies


@pytest.mark.parametrize("n,width,page", [(1, 1, 1), (2, 3, 16), (8, 20, 256), (33, 7, 5), (100, 30, 24), (700, 50, 64), (1300, 3, 16), (5, 900, 2), (40, 1000, 4), (1024, 20, 8), (2100, 40, 8)])
def test_fork(n, width, page):
    for seed in range(12 if n < 500 else 4):
        rng = random.Random(1000 * n + seed)
        ctx, have, rows, free, pool = tables(rng, n, width, page)
        kind = seed % 4
        parents = ([rng.randrange(-1, n) for _ in range(n)] if kind == 0 else [r if rng.random() < 0.8 else -1 for r in range(n)] if kind == 1
                   else None if kind == 2 else [min(range(n), key=lambda r: (ctx[r] < 0, r))] * n)
        # room for every copy
        spare = list(range(pool, pool + n))
        ring, state = ring_of(rng, free + spare, pool + n + rng.randint(0, 3))
        got, status = call_fork(page, pool + n, parents, ctx, rows, have, width, ring, state, trim=bool(seed & 1))
        assert status == 0
        check_fork(got, fork(page, pool + n, parents, ctx, rows, have, ring, state, bool(seed & 1)), width)


def unchanged(got, ctx, rows, have, width, ring, state):
    n = len(ctx)
    assert got["table_out"] == [r + [-9] * (width - len(r)) for r in rows]
    assert got["n_pages_out"] == have and got["ctx_out"] == ctx and got["free"] == ring and got["free_state_out"] == state
    assert got["copy_src"] == [-1] * n and got["copy_dst"] == [-1] * n and got["copy_tokens"] == [0] * n


@pytest.mark.parametrize("n", [6, 600, 1100])
def test_fork_errors_leave_everything(n):
    rng = random.Random(n)
    width, page = 12, 8
    ctx, have, rows, free, pool = tables(rng, n, width, page, idle=0.0, extra=0.0)
    ctx[0] = max(ctx[0], 1)
    have[0] = max(have[0], -(-ctx[0] // page))
    while len(rows[0]) < have[0]:
        rows[0].append(free.pop())
    ctx = [c if c % page or not c else c - 1 for c in ctx]
    ring, state = ring_of(rng, free, pool)
    same = list(range(n))
    for parents, c, h, st, code in ((same[:-1] + [n], ctx, have, state, 1), (same[:-1] + [-2], ctx, have, state, 1),
                                    (same, ctx, have[:-1] + [width + 1], state, 1), (same, ctx, have[:-1] + [-1], state, 1),
                                    (same, ctx[:-1] + [width * page + 1], have, state, 1), (same, ctx, have, [pool, 1], 1), (same, ctx, have, [0, pool + 1], 1),
                                    (same, ctx, have, [-1, 1], 1), (same, ctx, have, [0, -1], 1),
                                    ([0] * n, ctx, have, [state[0], n - 2], 6)):
        got, status = call_fork(page, pool, parents, c, rows, h, width, ring, st, False)
        assert status == code
        clamped = [r[:max(0, x)] for r, x in zip(rows, h)]
        n_ok = [len(r) for r in clamped]
        got["table_out"] = [t[:k] + [-9] * (width - k) for t, k in zip(got["table_out"], n_ok)]
        unchanged(got, c, clamped, h, width, ring, st)
    # a ring that is too short for what comes free
    if free:
        short, st = ring_of(rng, free, len(free))
        got, status = call_fork(page, pool, [-1] * n, ctx, rows, have, width, short, st, False)
        assert status == 6
        unchanged(got, ctx, rows, have, width, short, st)


def test_fork_with_pages_outside_the_pool():
    """Handed on as they are and reported; their copies are left out, everything else comes as it should."""
    rows, ctx, have = [[3, 99, 1], [2, -4], [0]], [9, 7, 4], [3, 2, 1]
    got, status = call_fork(4, 8, [0, 0, 1], ctx, rows, have, 3, [5, 6, 99, 4, -1, -1, -1, -1], [0, 4], False)
    assert status == 7
    assert got["table_out"] == [[3, 99, 1], [3, 99, 5], [2, -4, -9]]
    assert (got["copy_src"], got["copy_dst"], got["copy_tokens"]) == ([-1, 1, -1], [-1, 5, -1], [0, 1, 0])
    assert got["free_state_out"] == [1, 4] and got["free"][1:5] == [6, 99, 4, 0]
    got, status = call_fork(4, 8, [1, 1, 2], ctx, rows, have, 3, [5, 6, 7, 4, -1, -1, -1, -1], [0, 4], False)
    assert status == 7 and got["copy_src"] == [-1, -1, -1] and got["table_out"][:2] == [[2, 5, -9], [2, -4, -9]] and got["n_pages_out"] == [2, 2, 1]


def call_compact(pool, rows, have, width, ring, state, room):
    n = len(have)
    t = PageTable(block_table(rows, width), 16, pool, workspace=True)
    t.workspace.fill_(255)
    out = dict(table_out=torch.full((n, width), -9, dtype=torch.int32, device="cuda"), free_state_out=i32([-9, -9]), copy_src=i32([-9] * room),
               copy_dst=i32([-9] * room))
    free = i32(ring)
    t.compact_into(i32(have), free, i32(state), **out)
    torch.cuda.synchronize()
    got = {k: v.tolist() for k, v in out.items()}
    got["free"] = free.tolist()
    return got, int(t.status)


@pytest.mark.parametrize("n,width", [(1, 1), (2, 3), (8, 20), (33, 7), (100, 30), (700, 50), (1300, 3), (3, 2000), (40, 1000), (16, 2046), (2100, 40)])
def test_compact(n, width):
    for seed in range(10 if n < 500 else 3):
        rng = random.Random(77 * n + seed)
        _, have, rows, free, pool = tables(rng, n, width, 16)
        ring, state = ring_of(rng, free, pool)
        want, tail, moves = compact(pool, rows, have)
        room = len(moves) + seed % 3
        got, status = call_compact(pool, rows, have, width, ring, state, room)
        assert status == 0
        assert got["table_out"] == [r + [-9] * (width - len(r)) for r in want]
        assert got["free"] == tail + ring[len(tail):]
        assert got["free_state_out"] == [0, len(tail)]
        assert list(zip(got["copy_src"], got["copy_dst"])) == moves + [(-1, -1)] * (room - len(moves))


@pytest.mark.parametrize("n", [40, 1100])
def test_compact_errors_leave_everything(n):
    rng = random.Random(5)
    _, have, rows, free, pool = tables(rng, n, 10, 16, idle=0.0)
    ring, state = ring_of(rng, free, pool)
    _, tail, moves = compact(pool, rows, have)
    assert len(moves) > 1
    table = [r + [-9] * (10 - len(r)) for r in rows]
    for h, rg, room, code in ((have, ring, len(moves) - 1, 6), (have, ring[:len(tail) - 1], len(moves), 6), (have[:-1] + [11], ring, len(moves), 1),
                              (have[:-1] + [-1], ring, len(moves), 1)):
        got, status = call_compact(pool, rows, h, 10, rg, state, room)
        assert status == code
        assert [t for t in got["table_out"][:-1]] == table[:-1]
        assert got["free"] == rg and got["free_state_out"] == state and got["copy_src"] == [-1] * room and got["copy_dst"] == [-1] * room
    rows[0][0] = pool
    got, status = call_compact(pool, rows, have, 10, ring, state, 10 * n)
    assert status == 7 and got["table_out"][0][0] == pool


# ---------------------------------------------------------------- bytes

def pools(dtype, pages, page, heads, dim, turns=False):
    """K and V pools of random bits; turns: pages of K and V in turn, heads before tokens."""
    size = torch.int16 if dtype == "bf16" else torch.uint8
    top = 2 ** (8 * (2 if dtype == "bf16" else 1) - (1 if dtype == "bf16" else 0))
    if turns:
        x = torch.randint(0, top, (pages, 2, heads, page, dim), dtype=size, device="cuda")
        return x[:, 0].transpose(1, 2), x[:, 1].transpose(1, 2)
    return tuple(torch.randint(0, top, (pages, page, heads, dim), dtype=size, device="cuda") for _ in range(2))


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("pages,page,heads,dim,turns", [(9, 256, 8, 128, False), (7, 1, 1, 16, False), (40, 24, 2, 80, True), (11, 7, 3, 256, False),
                                                        (300, 16, 8, 64, True), (5, 1000, 5, 96, False)])
def test_copy(pages, page, heads, dim, turns, dtype):
    g = torch.Generator()
    g.manual_seed(pages)
    k, v = pools(dtype, pages, page, heads, dim, turns)
    k0, v0 = k.clone(), v.clone()
    order = torch.randperm(pages, generator=g)
    m = pages // 2
    src, dst = order[:m].clone(), order[m:2 * m]
    src = src[torch.randint(0, m, (m,), generator=g)]                    # one source may go to several places
    src[torch.rand(m, generator=g) < 0.3] = -1
    tokens = torch.randint(0, page + 1, (m,), generator=g)
    cache = PagedKV(k, v)
    for t in (tokens, None):
        k.copy_(k0), v.copy_(v0)
        cache.copy(src.int().cuda(), dst.int().cuda(), None if t is None else t.int().cuda())
        wk, wv = k0.clone(), v0.clone()
        for i in range(m):
            if src[i] >= 0:
                n = page if t is None else int(t[i])
                wk[dst[i], :n], wv[dst[i], :n] = k0[src[i], :n], v0[src[i], :n]
        assert torch.equal(k, wk) and torch.equal(v, wv)


def test_copy_of_many_pairs_and_errors():
    k, v = pools("bf16", 6000, 4, 1, 16)
    k0 = k.clone()
    cache = PagedKV(k, v)
    src, dst = torch.full((2999,), -1, dtype=torch.int32), torch.arange(3000, 5999, dtype=torch.int32)
    src[::7] = torch.arange(0, 2999, 7, dtype=torch.int32)
    cache.copy(src.cuda(), dst.cuda())
    assert torch.equal(k[3000:5999:7], k0[:2999:7]) and torch.equal(k[3001], k0[3001])
    for n in (3, 2999):
        for what, x in (("src", 6000), ("dst", 6000), ("dst", -1), ("tokens", 5), ("tokens", -1)):
            k.copy_(k0)
            a = dict(src=src[:n].clone(), dst=dst[:n].clone(), tokens=torch.full((n,), 4, dtype=torch.int32))
            a["src"][:2] = torch.tensor([0, 1], dtype=torch.int32)
            a[what][0] = x
            with pytest.raises(SKVError, match="INVALID_ARG"):
                cache.copy(**{key: t.cuda() for key, t in a.items()})
            assert torch.equal(k[3000], k0[3000]) and torch.equal(k[3001], k0[1])
    empty = torch.zeros(0, dtype=torch.int32, device="cuda")
    cache.copy(empty, empty)
    with pytest.raises(ValueError):
        cache.copy_into(src.cuda(), dst.cuda()[:5])
    with pytest.raises(ValueError):
        cache.copy_into(src.cuda().long(), dst.cuda().long())


def move_plain(pool, cu, rows, slots, kept, page):
    out = pool.clone()
    for r in range(len(cu) - 1):
        for i in range(cu[r], cu[r + 1]):
            if kept[i] >= 0:
                a, b = slots[rows[i]], kept[i]
                out[b // page, b % page] = out[a // page, a % page].clone()
    return out


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("counts,page,heads,dim,turns", [([1], 1, 1, 16, False), ([16] * 5, 16, 8, 128, False), ([60, 0, 3, 90, 33], 24, 2, 80, True),
                                                         ([7] * 300, 5, 3, 64, False), ([40, 41], 7, 8, 256, False)])
def test_move(counts, page, heads, dim, turns, dtype):
    """Accepted paths in order, and arbitrary lists, whose entries are moved one after the other."""
    for seed in range(4):
        rng = random.Random(seed + len(counts))
        n = sum(counts)
        pages = -(-n // page) + 2
        k, v = pools(dtype, pages, page, heads, dim, turns)
        place = list(range(pages * page))
        rng.shuffle(place)
        slots = place[:n] + [-1] * 3
        cu, rows, kept = [0], [-1] * (n + 3), [-1] * (n + 3)
        for c in counts:
            a = cu[-1]
            cu.append(a + c)
            if seed < 2:
                path = sorted(rng.sample(range(c), rng.randint(0, c)))
                for i, p in enumerate(path):
                    rows[a + i], kept[a + i] = a + p, slots[a + i]
            else:
                for i in range(c):
                    if rng.random() < 0.7:
                        rows[a + i], kept[a + i] = a + rng.randrange(c), slots[a + rng.randrange(c)]
        wk, wv = (move_plain(p.cpu(), cu, rows, slots, kept, page) for p in (k, v))
        PagedKV(k, v).move(i32(cu), i32(rows), torch.tensor(slots).cuda(), torch.tensor(kept).cuda())
        assert torch.equal(k.cpu(), wk) and torch.equal(v.cpu(), wv)


@pytest.mark.parametrize("many", [False, True])
def test_move_errors(many):
    k, v = pools("bf16", 300, 16, 2, 64)
    k0 = k.clone()
    n = 1500 if many else 4
    cache = PagedKV(k, v)
    slots = torch.arange(2 * n).cuda() if not many else torch.arange(2 * n).cuda() % 4800
    cu = torch.arange(0, 2 * n + 1, 2, dtype=torch.int32).cuda()
    for what, i, x in (("rows", 2, 2 * n), ("rows", 2, -1), ("kept", 2, 4800), ("slots", 3, 4800), ("slots", 3, -1), ("cu", 2, 2 * n + 1)):
        k.copy_(k0)
        a = dict(cu=cu.clone(), rows=torch.arange(2 * n, dtype=torch.int32).cuda(), slots=slots.clone(), kept=torch.full((2 * n,), -1).cuda())
        a["rows"][0::2] += 1
        a["kept"][0::2] = slots[0::2]
        a[what][i] = x
        with pytest.raises(SKVError, match="INVALID_ARG"):
            cache.move(a["cu"], a["rows"], a["slots"], a["kept"])
        flat, old = k.flatten(0, 1), k0.flatten(0, 1)
        assert torch.equal(flat[0], old[1]) and torch.equal(flat[2], old[2])
        if what != "cu":
            assert torch.equal(flat[4], old[5])


def test_more_entries_than_one_block_looks_through():
    k, v = pools("e4m3", 70000, 1, 1, 16)
    k0, cache = k.clone(), PagedKV(k, v)
    n = 69000
    src, dst = torch.full((n,), -1, dtype=torch.int32), torch.arange(1000, 70000, dtype=torch.int32)
    src[::701] = torch.arange(len(src[::701]), dtype=torch.int32)
    cache.copy(src.cuda(), dst.cuda())
    assert torch.equal(k[1000::701], k0[:len(src[::701])]) and torch.equal(k[1001:1701], k0[1001:1701])
    src[5] = 70000
    with pytest.raises(SKVError, match="INVALID_ARG"):
        cache.copy(src.cuda(), dst.cuda())
    k.copy_(k0)
    cu, rows = torch.arange(35001, dtype=torch.int32).cuda() * 2, torch.arange(70000, dtype=torch.int32).cuda()
    slots, kept = torch.arange(70000).cuda(), torch.full((70000,), -1).cuda()
    rows[0::2] += 1
    kept[0::2] = slots[0::2]
    cache.move(cu, rows, slots, kept)
    assert torch.equal(k[0::2], k0[1::2]) and torch.equal(k[1::2], k0[1::2])
    rows[69998] = -2
    with pytest.raises(SKVError, match="INVALID_ARG"):
        cache.move(cu, rows, slots, kept)


def test_far_pages_are_copied_and_moved():
    pool = torch.empty(4200, 2, 64, 8, 128, dtype=torch.bfloat16, device="cuda")         # 11 GB
    pool[7].normal_(), pool[4100].normal_()
    cache = PagedKV(pool[:, 0], pool[:, 1])
    want = pool[7].clone()
    cache.copy(i32([7]), i32([4199]))
    assert torch.equal(pool[4199], want)
    cache.copy(i32([4199]), i32([4198]), i32([3]))
    assert torch.equal(pool[4198, :, :3], want[:, :3])
    cache.move(i32([0, 2]), i32([1, -1]), torch.tensor([4197 * 64 + 5, 4100 * 64 + 63]).cuda(), torch.tensor([4197 * 64 + 5, -1]).cuda())
    assert torch.equal(pool[4197, :, 5], pool[4100, :, 63])


# ---------------------------------------------------------------- a pool in use

def test_pool_over_many_steps():
    """Admissions, forks, ends and compactions in turn: pages are held by the rows that should hold them, and the
    ring has every other one once; tokens stay what they were (each slot holds the history it stands for)."""
    rng = random.Random(3)
    n, width, page, pages = 9, 14, 4, 80
    pool = PagePool(n, width, page, pages)
    k = torch.zeros(pages, page, 1, 16, dtype=torch.int16, device="cuda")
    cache = PagedKV(k, torch.zeros_like(k))
    history = [[] for _ in range(n)]                       # what each row should read back
    ctx = [-1] * n
    stamp = 1

    def audit():
        have, table = pool.n_pages.tolist(), pool.block_table.tolist()
        held = {p for r in range(n) for p in table[r][:have[r]]}
        head, count = pool.free_state.tolist()
        ring = pool.free_pages.tolist()
        free = [ring[(head + i) % pages] for i in range(count)]
        assert sorted(free + sorted(held)) == list(range(pages))
        for r in range(n):
            got = [int(k[table[r][t // page], t % page, 0, 0]) for t in range(len(history[r]))]
            assert got == history[r], r
        # a page that tokens may still be added to is one row's own
        for r in range(n):
            if ctx[r] >= 0 and ctx[r] % page:
                p = table[r][ctx[r] // page]
                assert sum(p in table[s][:have[s]] for s in range(n)) == 1

    for step in range(60):
        act = rng.choice(["step", "step", "step", "fork", "fork", "end", "compact"])
        if act == "fork":
            live = [r for r in range(n) if ctx[r] >= 0]
            parents = [rng.choice(live) if live and (ctx[r] < 0 and rng.random() < 0.5 or rng.random() < 0.2) else r for r in range(n)]
            lens, src, dst, tokens = pool.fork(i32(parents), i32(ctx), trim=rng.random() < 0.5)
            cache.copy(src, dst, tokens)
            ctx = [ctx[p] for p in parents]
            history = [list(history[p]) if ctx[r] >= 0 else [] for r, p in enumerate(parents)]
            assert lens.tolist() == ctx
        elif act == "compact":
            src, dst = pool.compact()
            cache.copy(src, dst)
            have, table = pool.n_pages.tolist(), pool.block_table.tolist()
            held = {p for r in range(n) for p in table[r][:have[r]]}
            assert held == set(range(len(held)))
        else:
            if act == "end":
                gone = rng.randrange(n)
                ctx[gone], history[gone] = -1, []
            new = []
            for r in range(n):
                if ctx[r] < 0 and rng.random() < 0.3 and act == "step":
                    ctx[r] = 0
                new.append(rng.randint(0, 5) if ctx[r] >= 0 and ctx[r] + 5 <= width * page else 0)
            spare = pages - len({p for r in range(n) for p in pool.block_table.tolist()[r][:pool.n_pages.tolist()[r]]})
            if sum(-(-x // page) + 1 for x in new if x) > spare:
                new = [0] * n
            cu, slots = pool.step(i32(ctx), i32(new), 64)
            slots = slots.tolist()
            at = 0
            for r in range(n):
                for _ in range(new[r]):
                    k.view(-1, 16)[slots[at]] = stamp
                    history[r].append(stamp)
                    stamp += 1
                    at += 1
                ctx[r] += new[r] if ctx[r] >= 0 else 0
        audit()


def test_pool_calls_on_another_stream_and_in_a_capture():
    pool, side = PagePool(4, 6, 4, 30), torch.cuda.Stream()
    ctx, new = i32([0, 0, -1, -1]), i32([10, 3, 0, 0])
    pool.step(ctx, new, 16)
    now = i32([10, 3, -1, -1])
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)
    lens, src, dst, tokens = pool.fork(i32([0, 1, 0, 1]), now, stream=side)
    assert lens.tolist() == [10, 3, 10, 3]
    assert (src.tolist(), dst.tolist(), tokens.tolist()) == ([-1, -1, 2, 3], [-1, -1, 4, 5], [0, 0, 2, 3])
    assert pool.block_table.tolist()[2][:3] == [0, 1, 4] and pool.n_pages.tolist() == [3, 1, 3, 1]
    torch.cuda._sleep(200_000_000)
    lens2, _, _, _ = pool.fork(None, i32([-1, 3, 10, 3]), check=False, stream=side)
    torch.cuda.synchronize()
    assert lens2.tolist() == [-1, 3, 10, 3] and pool.free_state.tolist()[1] == 30 - 5
    src, dst = pool.compact(stream=side)
    assert sorted(p for r, h in zip(pool.block_table.tolist(), pool.n_pages.tolist()) for p in r[:h]) == [0, 1, 2, 3, 4]
    for call in (lambda: pool.fork(None, now), pool.compact):
        with pytest.raises(ValueError, match="host"):
            with torch.cuda.graph(torch.cuda.CUDAGraph()):
                call()
    t = PageTable(pool.block_table.clone(), 4, 30)
    with pytest.raises(ValueError, match="workspace"):
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            t.compact_into(pool.n_pages, pool.free_pages.clone(), pool.free_state, torch.empty_like(t.block_table), torch.empty_like(pool.free_state),
                           torch.empty_like(pool.free_pages), torch.empty_like(pool.free_pages))


def test_plans_in_a_graph():
    rng = random.Random(8)
    n, width, page = 50, 60, 8
    ctx, have, rows, free, pool = tables(rng, n, width, page)
    ring, state = ring_of(rng, free + list(range(pool, pool + n)), pool + n)
    parents = [rng.randrange(-1, n) for _ in range(n)]
    t = PageTable(block_table(rows, width), page, pool + n, workspace=True)
    free, st = i32(ring), i32(state)
    out = [torch.full((n, width), -9, dtype=torch.int32, device="cuda"), i32([0] * n), i32([0] * n), i32([0, 0]), i32([0] * n), i32([0] * n), i32([0] * n)]
    args = (i32(parents), i32(ctx), i32(have), free, st)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        t.fork_into(*args, *out)
    for _ in range(3):                                     # the ring's front and the old rows are as they were
        g.replay()
    t.check_status("fork")
    got = dict(zip(("table_out", "n_pages_out", "ctx_out", "free_state_out", "copy_src", "copy_dst", "copy_tokens"), (o.tolist() for o in out)))
    got["free"] = free.tolist()
    check_fork(got, fork(page, pool + n, parents, ctx, rows, have, ring, state, False), width)


def test_tables_with_wider_rows_and_an_empty_ring():
    """Rows of wider tensors, in and out; what lies beside them stays."""
    wide = torch.full((3, 9), 77, dtype=torch.int32, device="cuda")
    wide[:, 2:6] = i32([[4, 1, -9, -9], [0, -9, -9, -9], [4, 3, 2, -9]])
    other = torch.full((3, 12), 55, dtype=torch.int32, device="cuda")
    t = PageTable(wide[:, 2:6], 4, 6)
    empty, st, st2 = i32([]), i32([0, 0]), i32([-9, -9])
    ctx, have = i32([8, 4, 11]), i32([2, 1, 3])
    out = [i32([0] * 3) for _ in range(5)]
    t.fork_into(i32([0, 0, 2]), ctx, have, empty, st, other[:, 1:5], out[0], out[1], st2, *out[2:])
    torch.cuda.synchronize()
    assert int(t.status) == 6                              # page 0 comes free, and the ring has no room
    t.fork_into(i32([0, 1, 0]), ctx, have, empty, st, other[:, 1:5], out[0], out[1], st2, *out[2:])
    torch.cuda.synchronize()
    assert int(t.status) == 6
    t.fork_into(None, ctx, have, empty, st, other[:, 1:5], out[0], out[1], st2, *out[2:])
    t.check_status("fork")
    assert other.tolist() == [[55, 4, 1] + [55] * 9, [55, 0] + [55] * 10, [55, 4, 3, 2] + [55] * 8]
    assert out[0].tolist() == [2, 1, 3] and st2.tolist() == [0, 0]
    ring, other = i32([-1] * 6), other.fill_(55)
    t.compact_into(have, ring, st, other[:, 3:7], st2, out[2], out[3])
    t.check_status("compact")
    assert other.tolist() == [[55] * 3 + [4, 1] + [55] * 7, [55] * 3 + [0] + [55] * 8, [55] * 3 + [4, 3, 2] + [55] * 6]
    assert ring.tolist() == [5] + [-1] * 5 and st2.tolist() == [0, 1] and out[2].tolist() == [-1] * 3
    assert wide[:, :2].eq(77).all() and wide[:, 6:].eq(77).all()


def test_what_the_wrappers_refuse():
    t = PageTable(i32([[0, 1], [2, 3]]), 4, 8)
    a = dict(parents=i32([0, 1]), ctx_len=i32([5, 6]), n_pages=i32([2, 2]), free_pages=i32([4, 5, 6, 7]), free_state=i32([0, 4]),
             table_out=i32([[0, 0], [0, 0]]), n_pages_out=i32([0, 0]), ctx_out=i32([0, 0]), free_state_out=i32([0, 0]), copy_src=i32([0, 0]),
             copy_dst=i32([0, 0]), copy_tokens=i32([0, 0]))
    t.fork_into(**a)
    t.check_status("fork")
    for kw in (dict(parents=i32([0])), dict(ctx_len=i32([0])), dict(table_out=t.block_table), dict(table_out=i32([[0], [0]])),
               dict(free_state=i32([0])), dict(copy_src=i32([0, 0, 0])), dict(parents=i32([0, 1]).long()), dict(free_pages=a["free_pages"][::2])):
        with pytest.raises(ValueError):
            t.fork_into(**dict(a, **kw))
    for kw in (dict(n_pages_out=a["n_pages"]), dict(ctx_out=a["ctx_len"]), dict(free_state_out=a["free_state"])):
        with pytest.raises(SKVError):
            t.fork_into(**dict(a, **kw))
    c = {k: a[k] for k in ("n_pages", "free_pages", "free_state", "table_out", "free_state_out", "copy_src", "copy_dst")}
    t.compact_into(**c)
    for kw in (dict(n_pages=i32([1])), dict(copy_dst=i32([0])), dict(table_out=t.block_table), dict(free_state=i32([0, 0, 0]))):
        with pytest.raises(ValueError):
            t.compact_into(**dict(c, **kw))
