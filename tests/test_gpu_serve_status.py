"""Errors are reported, and the rest is done, whichever way a call of that size writes its status: a block of its own that
looks through all entries, or any block behind a launch that clears it. Sizes on both sides of each border, and a wrong entry at either
end."""
import pytest
import torch

from lossless_kv_cache_scalar_gb300 import PagedKV, Rotary, SKVError, Verifier

pytestmark = pytest.mark.gpu


def i32(v):
    return torch.tensor(v, dtype=torch.int32).cuda()


@pytest.mark.parametrize("draft", [True, False])
@pytest.mark.parametrize("requests,nodes", [(512, 8), (1023, 4), (1024, 4), (241, 17), (900, 9)])
def test_verification(requests, nodes, draft):
    vocab, rows = 16, requests * nodes
    g = torch.Generator()
    g.manual_seed(rows)
    probs = torch.softmax(torch.randn(rows, vocab, generator=g), -1).cuda()
    q = torch.softmax(torch.randn(rows, vocab, generator=g), -1).cuda() if draft else None
    tokens = torch.randint(0, vocab, (rows,), generator=g, dtype=torch.int32).cuda()
    u, cu = torch.rand(rows, generator=g).cuda(), torch.arange(requests + 1, dtype=torch.int32, device="cuda") * nodes
    v = Verifier(requests, vocab)
    want = v.verify(probs, tokens, cu, u, draft_probs=q)
    for r in (0, requests // 2, requests - 1):
        bad = tokens.clone()
        bad[r * nodes + nodes - 1] = vocab
        out = [torch.full((requests,), -7, dtype=torch.int32, device="cuda"), torch.full((rows,), -7, dtype=torch.int32, device="cuda"),
               torch.full((requests,), -7, dtype=torch.int32, device="cuda")]
        v.verify_into(probs, bad, cu, u, *out, draft_probs=q)
        with pytest.raises(SKVError, match="INVALID_ARG"):
            v.check_status("verify")
        rest = torch.arange(requests, device="cuda") != r
        assert torch.equal(out[0][rest], want[0][rest]) and torch.equal(out[2][rest], want[2][rest])
        assert int(out[0][r]) == 0 and int(out[2][r]) == -1
    again = v.verify(probs, tokens, cu, u, draft_probs=q)
    assert all(torch.equal(a, b) for a, b in zip(again, want))


@pytest.mark.parametrize("n", [512, 513, 16384, 16385, 40000])
def test_copies(n):
    pool = torch.randint(0, 1 << 15, (2 * n + 2, 2, 1, 16), dtype=torch.int16, device="cuda")
    v = pool.clone()
    c = PagedKV(pool, v)
    g = torch.Generator()
    g.manual_seed(n)
    src = torch.randperm(n, generator=g, dtype=torch.int32)
    src[torch.rand(n, generator=g) < 0.6] = -1
    src[0], src[n - 1] = n, n + 1                          # (no destinations below)
    dst = (n + 2 + torch.randperm(n, generator=g)).int()
    for bad in (None, 0, n - 1):
        before = pool.clone()
        d = dst.clone()
        if bad is not None:
            d[bad] = 2 * n + 2
        live = (src >= 0) & (d < 2 * n + 2)
        c.copy_into(src.cuda(), d.cuda())
        if bad is None:
            c.check_status("copy")
        else:
            with pytest.raises(SKVError, match="INVALID_ARG"):
                c.check_status("copy")
        before[d[live].long().cuda()] = before[src[live].long().cuda()]
        assert torch.equal(pool, before) and torch.equal(v, before)


@pytest.mark.parametrize("requests,nodes", [(1024, 16), (1025, 16), (16384, 1), (16385, 1), (300, 130), (70000, 1)])
def test_moves(requests, nodes):
    n = requests * nodes
    pool = torch.randint(0, 1 << 15, (n // 4 + 1, 8, 1, 16), dtype=torch.int16, device="cuda")
    v = pool.clone()
    c = PagedKV(pool, v)
    cu = torch.arange(requests + 1, dtype=torch.int32, device="cuda") * nodes
    # every request's last token to the place behind its tokens
    slots = torch.arange(n, device="cuda") // nodes * 2 * nodes + torch.arange(n, device="cuda") % nodes
    rows = torch.full((n,), -1, dtype=torch.int32, device="cuda")
    kept = torch.full((n,), -1, dtype=torch.int64, device="cuda")
    at = torch.arange(requests, device="cuda") * nodes
    rows[at], kept[at] = (at + nodes - 1).int(), slots[at] + nodes
    for bad in (None, 0, requests - 1):
        flat = pool.flatten(0, 1).clone()
        k = kept.clone()
        if bad is not None:
            k[at[bad]] = pool.shape[0] * 8
        live = torch.ones(requests, dtype=torch.bool, device="cuda")
        if bad is not None:
            live[bad] = False
        c.move_into(cu, rows, slots, k)
        if bad is None:
            c.check_status("move")
        else:
            with pytest.raises(SKVError, match="INVALID_ARG"):
                c.check_status("move")
        flat[kept[at[live]]] = flat[slots[at[live] + nodes - 1]]
        assert torch.equal(pool.flatten(0, 1), flat) and torch.equal(v.flatten(0, 1), flat)


@pytest.mark.parametrize("n,q_heads,heads,dim", [(2048, 2, 1, 64), (2049, 2, 1, 64), (2049, 16, 4, 64), (4252, 4, 2, 128), (4253, 40, 4, 128), (6000, 4, 2, 128),
                                                 (8600, 40, 4, 128), (65536, 1, 1, 16), (65537, 1, 1, 16)])
def test_rotated_rows(n, q_heads, heads, dim):
    """And each row is what it is among a few, whatever the number of warps that a row's heads go to."""
    g = torch.Generator()
    g.manual_seed(n)
    q = torch.randn(n, q_heads, dim, generator=g).bfloat16().cuda()
    k, v = (torch.randn(n, heads, dim, generator=g).bfloat16().cuda() for _ in range(2))
    w = 1 + 0.1 * torch.randn(2, dim, generator=g)
    rotary = Rotary(dim, [1e4 ** (-2.0 * i / dim) for i in range(dim // 2)], w[0], w[1])
    pos, slots = torch.randint(0, 1 << 17, (n,), generator=g, dtype=torch.int32).cuda(), torch.randperm(n, generator=g).cuda()
    pool = torch.zeros(2, -(-n // 16), 16, heads, dim, dtype=torch.bfloat16, device="cuda")
    c = PagedKV(pool[0], pool[1])
    out = c.rotate_append(rotary, q, k, v, pos, slots)
    whole = pool.clone()
    few = torch.tensor([0, 1, n // 3, n - 2, n - 1], device="cuda")
    got = c.rotate_append(rotary, q[few], k[few], v[few], pos[few], slots[few])
    assert torch.equal(got, out[few]) and torch.equal(pool, whole)
    for bad in (0, n - 1):
        s = slots.clone()
        s[bad] = pool.shape[1] * 16
        pool.zero_()
        c.rotate_append_into(rotary, q, k, v, pos, s, got_all := torch.empty_like(out))
        with pytest.raises(SKVError, match="INVALID_ARG"):
            c.check_status("rotate")
        assert torch.equal(got_all, out)
        want = whole.clone().flatten(1, 2)
        want[:, slots[bad]] = 0
        assert torch.equal(pool.flatten(1, 2), want)
