"""PagePool.step where rows share pages: rows that go back or are admitted anew, errors, and pools that
share nothing any more."""
import pytest
import torch

from lossless_kv_cache_scalar_gb300 import PagePool, SKVError

pytestmark = pytest.mark.gpu

PAGE = 4


def i32(v):
    return torch.tensor(v, dtype=torch.int32).cuda()


def rows_of(pool):
    return [row[:h] for row, h in zip(pool.block_table.tolist(), pool.n_pages.tolist())]


def ring_of(pool):
    head, count = pool.free_state.tolist()
    ring = pool.free_pages.tolist()
    return [ring[(head + i) % len(ring)] for i in range(count)]


def audit(pool):
    """Every page of the pool is held or on the ring, once."""
    held = {p for row in rows_of(pool) for p in row}
    assert sorted(ring_of(pool) + sorted(held)) == list(range(pool.pool_pages))


def shared_pool(tokens=10, rows=3, pages=24):
    """`rows` rows of `tokens` tokens that share the first row's full pages, and an idle row."""
    pool = PagePool(rows + 1, 8, PAGE, pages)
    pool.step(i32([0] + [-1] * rows), i32([tokens] + [0] * rows), tokens)
    pool.fork(i32([0] * rows + [-1]), i32([tokens] + [-1] * rows))
    audit(pool)
    return pool


@pytest.mark.parametrize("back", [0, 4])
@pytest.mark.parametrize("check", [True, False])
def test_a_row_that_starts_again_leaves_the_shared_pages_alone(back, check):
    """A row that ends and is admitted anew in one step, or goes back to a page's border: its new tokens fall into
    pages that are its own."""
    pool = shared_pool()
    before = rows_of(pool)
    cu, slots = pool.step(i32([back, 10, 10, -1]), i32([9, 1, 1, 0]), 11, check=check)
    pool.check_status("step")
    after, cu, slots = rows_of(pool), cu.tolist(), slots.tolist()
    audit(pool)
    assert after[1] == before[1] and after[2] == before[2]
    for r in range(3):
        for at in slots[cu[r]:cu[r + 1]]:
            assert at // PAGE in after[r] and not any(at // PAGE in after[s] for s in range(4) if s != r), (r, at)
    assert after[0][:back // PAGE] == before[0][:back // PAGE]


def test_an_idle_row_is_admitted_beside_shared_ones():
    pool = shared_pool()
    pool.step(i32([-1, 10, 10, 0]), i32([0, 3, 0, 17]), 32)
    audit(pool)
    assert [len(r) for r in rows_of(pool)] == [0, 4, 3, 5]


def state(pool):
    return rows_of(pool), pool.n_pages.tolist(), pool.free_state.tolist(), ring_of(pool)


@pytest.mark.parametrize("ctx,new,room,error", [([-1, 10, 10, -1], [0, 1, 1, 2], 8, "INVALID_ARG"), ([10, -1, 13, -1], [0, 0, 1, 0], 8, "INVALID_ARG"),
                                                ([-1, 8, 10, 0], [0, 1, 1, 99], 101, "CAPACITY"), ([-1, 8, -1, 0], [0, 20, 0, 9], 29, "CAPACITY")])
def test_a_refused_step_leaves_a_shared_pool_as_it_was(ctx, new, room, error):
    pool = shared_pool(pages=9)
    before = state(pool)
    for _ in range(2):
        with pytest.raises(SKVError, match=error):
            pool.step(i32(ctx), i32(new), room)
        assert state(pool) == before
    pool.step(i32([-1, 10, 10, -1]), i32([0, 1, 3, 0]), 4)
    audit(pool)
    assert [len(r) for r in rows_of(pool)] == [0, 3, 4, 0]


@pytest.mark.parametrize("check", [True, False])
def test_a_bad_page_that_only_the_shared_rows_show(check):
    """A page number outside the pool in a row without new tokens, before its last page: nothing but the walk over the shared
    rows comes past it."""
    pool = shared_pool()
    good = int(pool.block_table[2, 0])
    pool.block_table[2, 0] = 99
    ctx, new = i32([10, 10, 10, -1]), i32([1, 0, 0, 0])
    if check:
        with pytest.raises(SKVError, match="CORRUPT"):
            pool.step(ctx, new, 4)
    else:
        pool.step(ctx, new, 4, check=False)
        with pytest.raises(SKVError, match="CORRUPT"):
            pool.check_status("step")
    pool.block_table[2, 0] = good
    pool.step(i32([11, 10, 10, -1]), i32([1, 0, 0, 0]), 4)
    pool.check_status("step")
    pool.compact()
    audit(pool)


@pytest.mark.parametrize("check", [True, False])
def test_a_step_on_another_stream(check):
    pool, side = shared_pool(), torch.cuda.Stream()
    ctx, new = i32([-1, 10, 0, -1]), i32([0, 1, 9, 0])
    torch.cuda.synchronize()
    for _ in range(2):
        torch.cuda._sleep(100_000_000)
        cu, slots = pool.step(ctx, new, 10, check=check, stream=side)
        torch.cuda.synchronize()
        pool.check_status("step", side)
        audit(pool)
        assert cu.tolist() == [0, 0, 1, 10, 10] and [len(r) for r in rows_of(pool)] == [0, 3, 3, 0]
        held = rows_of(pool)
        assert [at // PAGE for at in slots.tolist()] == [held[1][2]] + [held[2][i // PAGE] for i in range(9)]


def test_a_pool_that_shares_nothing_any_more_ends_its_rows_in_one_launch():
    """Launches of a step are those of a pool that was never forked, some steps after the last sharing row has ended; while
    rows share pages they stay two."""
    pool = shared_pool()
    two = []

    class Ends:
        def __init__(self, ends):
            self.ends = ends

        def __getattr__(self, name):
            if name == "fork_into":
                two.append(1)
            return getattr(self.ends, name)

    pool._ends = Ends(pool._ends)
    length = 10
    for step in range(40):                                 # two rows share pages
        pool.step(i32([length, length, -1, -1]), i32([step % 2, step % 2, 0, 0]), 2)
        length += step % 2
    assert len(two) == 40
    for step in range(40):                                 # one row's pages are its own
        pool.step(i32([length, -1, -1, -1]), i32([0, 0, 0, 0]), 2)
    assert 40 < len(two) <= 40 + 16
    audit(pool)
    pool.step(i32([-1, 0, -1, -1]), i32([0, 9, 0, 0]), 9)
    audit(pool)
    assert [len(r) for r in rows_of(pool)] == [0, 3, 0, 0]
    pool.fork(None, i32([-1, 9, -1, -1]))                  # nobody shares: still one launch
    n = len(two)
    pool.step(i32([-1, 9, -1, -1]), i32([0, 9, 0, 0]), 9)
    assert len(two) == n
    pool.fork(i32([1, 1, -1, -1]), i32([-1, 18, -1, -1]))
    pool.step(i32([-1, 18, -1, -1]), i32([0, 9, 0, 0]), 9)
    assert len(two) == n + 1
    audit(pool)
