"""Verification of drafted trees, against its statement in whole numbers."""
import math

import numpy as np
import pytest
import torch

from tests._servetest import verify
from lossless_kv_cache_scalar_gb300 import SKVError, Verifier

pytestmark = pytest.mark.gpu


def gen_of(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def i32(v):
    return torch.tensor(v, dtype=torch.int32).cuda()


def made(seed, counts, vocab, dtype="f32", draft="drawn", tree=True, pad=3, spread=3.0, noise=0.7):
    g = gen_of(seed)
    rows = sum(counts) + pad
    z = spread * torch.randn(rows, vocab, generator=g)
    p = torch.softmax(z, -1)
    q = torch.softmax(z + noise * torch.randn(rows, vocab, generator=g), -1)
    if dtype == "bf16":
        p, q = p.bfloat16(), q.bfloat16()
    cu = [0]
    parents = []
    for n in counts:
        cu.append(cu[-1] + n)
        parents += [-1] + [int(torch.randint(0, i, (1,), generator=g)) if tree else i - 1 for i in range(1, n)] if n else []
    parents += [0] * pad
    tokens = torch.zeros(rows, dtype=torch.int64)
    for a, n in zip(cu, counts):
        used = {}
        for i in range(1, n):
            par = parents[a + i]
            w = q[a + par].float().clone()
            if draft != "drawn":
                w[used.get(par, [])] = 0
            if draft == "best" or float(w.sum()) == 0:
                tokens[a + i] = int(w.argmax())
            else:
                tokens[a + i] = int(torch.multinomial(w, 1, generator=g))
            used.setdefault(par, []).append(int(tokens[a + i]))
    return dict(probs=p, draft=None if draft == "best" else q, tokens=tokens.int(), parents=torch.tensor(parents, dtype=torch.int32) if tree else None,
                uniform=torch.rand(rows, generator=g), cu=cu, vocab=vocab, distinct=draft == "distinct", rows=rows)


def to_np(t):
    return t.float().numpy()


def plain(s):
    return verify(to_np(s["probs"]), None if s["draft"] is None else to_np(s["draft"]), s["tokens"].numpy(),
                  None if s["parents"] is None else s["parents"].numpy(), s["uniform"].numpy(), s["cu"], s["vocab"], s["distinct"])


def call(s, stream=None):
    n = len(s["cu"]) - 1
    slots = torch.arange(s["rows"], dtype=torch.int64, device="cuda") * 3 + 1
    ctx = torch.arange(n, dtype=torch.int32, device="cuda") * 100
    out = dict(accepted=i32([-7] * n), rows=i32([-7] * s["rows"]), next_tokens=i32([-7] * n),
               kept=torch.full((s["rows"],), -7, dtype=torch.int64, device="cuda"), ctx_out=i32([-7] * n))
    v = Verifier(n, s["vocab"])
    dev = lambda t: None if t is None else t if t.is_cuda else t.cuda()          # noqa: E731
    v.verify_into(dev(s["probs"]), dev(s["tokens"]), i32(s["cu"]), dev(s["uniform"]), parents=dev(s["parents"]), draft_probs=dev(s["draft"]),
                  distinct=s["distinct"], slots=slots, ctx_len=ctx, stream=stream, **out)
    v.check_status("verify", stream)
    return {k: t.cpu() for k, t in out.items()}, slots.cpu(), ctx.cpu()


def compare(s):
    out, slots, ctx = call(s)
    accepted, paths, nxt = plain(s)
    assert out["accepted"].tolist() == accepted
    assert out["next_tokens"].tolist() == nxt
    assert out["ctx_out"].tolist() == [int(c) + a for c, a in zip(ctx, accepted)]
    rows, kept = [-7] * s["rows"], [-7] * s["rows"]
    for r, path in enumerate(paths):
        for j in range(s["cu"][r], s["cu"][r + 1]):
            i = j - s["cu"][r]
            rows[j] = path[i] if i < len(path) else -1
            kept[j] = int(slots[j]) if i < len(path) else -1
    assert out["rows"].tolist() == rows
    assert out["kept"].tolist() == kept
    return accepted, nxt


CASES = [([1], 1, False), ([1, 1, 1], 7, False), ([5], 1000, False), ([5, 0, 2, 1, 0], 33, True), ([9, 3, 12], 4097, True), ([20] * 6, 513, True),
         ([27, 1, 60], 50257, True), ([4], 151936, False), ([6, 3], 1 << 19, True), ([64] * 12, 100, True), ([33], 32, True)]


@pytest.mark.parametrize("draft", ["drawn", "distinct", "best"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("counts,vocab,tree", CASES)
def test_against_whole_numbers(counts, vocab, tree, dtype, draft):
    for seed in range(2 if vocab > 10000 else 6):
        compare(made(100 * seed + vocab % 97, counts, vocab, dtype, draft, tree, spread=1.0 + seed))


@pytest.mark.parametrize("draft", ["drawn", "distinct", "best"])
def test_many_siblings(draft):
    """Wide levels: many rejections, each with its sum over what is left."""
    for seed in range(4):
        s = made(seed, [40, 25], 300, draft=draft, spread=0.7, noise=2.5)
        s["parents"] = torch.tensor([0] * 20 + [3] * 10 + [0] * 10 + [0] * 12 + [2] * 13 + [0] * 3, dtype=torch.int32)
        s["uniform"] = s["uniform"] ** 0.25
        acc, _ = compare(s)


@pytest.mark.parametrize("draft,n", [("drawn", 1500), ("distinct", 700), ("best", 1300)])
def test_more_nodes_than_are_gathered_at_once(draft, n):
    """Chains of children of late nodes, and a walk that goes past the first batch."""
    for seed in range(3):
        s = made(seed, [n, 3], 50, draft="drawn", spread=0.5, noise=0.1)
        if draft == "best":
            s["draft"] = None
        s["distinct"] = draft == "distinct"
        g = gen_of(seed + 50)
        par = [max(0, i - 1 - int(torch.randint(0, 3, (1,), generator=g))) for i in range(n)]
        if seed == 1:
            par[600:] = [0] * (n - 600)
        s["parents"] = torch.tensor(par + [0, 0, 1] + [0] * 3, dtype=torch.int32)
        s["uniform"] = s["uniform"] * (1.0 if seed == 2 else 0.02)
        compare(s)


@pytest.mark.parametrize("draft,dtype", [("best", "f32"), ("best", "bf16"), ("drawn", "f32")])
def test_many_requests_of_a_large_vocabulary(draft, dtype):
    """Few CTAs to a request: a part of the row comes in several pieces."""
    compare(made(3, [2, 1, 3, 0] * 25, 60001, dtype, draft, spread=4.0))


@pytest.mark.parametrize("draft", ["drawn", "best"])
def test_the_same_in_any_company(draft):
    """The number of requests chooses how a row is split; the answer does not depend on it."""
    s = made(21, [7], 70000, draft=draft, pad=0)
    want = plain(s)
    for n in (1, 9, 20, 70):
        t = dict(s, probs=s["probs"].cuda().repeat(n, 1), tokens=s["tokens"].repeat(n), parents=s["parents"].repeat(n), uniform=s["uniform"].repeat(n),
                 cu=list(range(0, 7 * n + 1, 7)), rows=7 * n)
        if draft == "drawn":
            t["draft"] = s["draft"].cuda().repeat(n, 1)
        out, _, _ = call(t)
        assert out["accepted"].tolist() == want[0] * n and out["next_tokens"].tolist() == want[2] * n


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("draft", ["drawn", "best"])
def test_full_sums_over_the_largest_vocabulary(draft, dtype):
    """150 requests, the fewest CTAs to each: the longest runs of a warp, of probabilities of one (0.75 left of each behind a
    rejection), whose sums pass 2^62."""
    vocab, n = 1 << 19, 150
    for seed, first in enumerate((0.0, 0.5, 0.999999)):
        s = made(31 + seed, [2], vocab, dtype, draft, tree=False, pad=0)
        s["probs"] = torch.ones_like(s["probs"])
        if draft == "drawn":
            s["draft"] = torch.full_like(s["probs"], 0.25)
        if seed:
            s["probs"][0, int(s["tokens"][1])] = 0           # the only drafted token is rejected
        s["uniform"] = torch.tensor([first, 0.75])
        want = plain(s)
        t = dict(s, probs=s["probs"].cuda().repeat(n, 1), tokens=s["tokens"].repeat(n), uniform=s["uniform"].repeat(n),
                 cu=list(range(0, 2 * n + 1, 2)), rows=2 * n)
        if draft == "drawn":
            t["draft"] = s["draft"].cuda().repeat(n, 1)
        out, _, _ = call(t)
        assert out["accepted"].tolist() == want[0] * n and out["next_tokens"].tolist() == want[2] * n
        assert want[0] == [1 if seed else 2]


def test_rows_far_into_a_large_tensor():
    """More than 2^32 probabilities: the last rows of 29,000."""
    rows, vocab = 29000, 151937
    s = made(22, [4], vocab, dtype="bf16", pad=0)
    big = torch.empty(rows, vocab, dtype=torch.bfloat16, device="cuda")
    big[-4:] = s["probs"].cuda()
    tokens, uniform, parents = torch.zeros(rows, dtype=torch.int32), torch.zeros(rows), torch.zeros(rows, dtype=torch.int32)
    tokens[-4:], uniform[-4:], parents[-4:] = s["tokens"], s["uniform"], s["parents"]
    draft = torch.empty(rows, vocab, dtype=torch.bfloat16, device="cuda")
    draft[-4:] = s["draft"].cuda()
    v = Verifier(1, vocab)
    got = v.verify(big, tokens.cuda(), i32([rows - 4, rows]), uniform.cuda(), parents=parents.cuda(), draft_probs=draft)
    want = plain(s)
    assert got[0].tolist() == want[0] and got[2].tolist() == want[2]
    assert got[1][-4:].tolist() == [p + rows - 4 for p in want[1][0]] + [-1] * (4 - want[0][0])


def test_no_rows():
    v = Verifier(3, 100)
    e = torch.zeros(0, dtype=torch.int32, device="cuda")
    acc, rows, nxt, after = v.verify(torch.zeros(0, 100, device="cuda"), e, i32([0, 0, 0, 0]), e.float(), ctx_len=i32([4, 5, -1]))
    assert acc.tolist() == [0, 0, 0] and nxt.tolist() == [-1, -1, -1] and rows.numel() == 0 and after.tolist() == [4, 5, -1]
    v = Verifier(0, 100)
    assert v.verify(torch.zeros(2, 100, device="cuda"), i32([1, 1]), i32([0]), torch.zeros(2, device="cuda"))[1].tolist() == [-1, -1]


def test_uniform_numbers_at_the_ends():
    for u in (0.0, 1.0 - 2.0 ** -24, 2.0 ** -149, 0.5):
        for draft in ("drawn", "distinct", "best"):
            s = made(8, [6, 1, 4], 200, draft=draft)
            s["uniform"].fill_(u)
            compare(s)


def test_borders_of_the_cumulative_sum():
    """Probabilities that are whole eighths: the drawn number falls on borders exactly."""
    s = made(1, [1] * 8, 5, pad=0, tree=False)
    s["probs"] = torch.tensor([0.25, 0.0, 0.125, 0.5, 0.125]).repeat(8, 1)
    s["uniform"] = torch.arange(8) / 8.0
    _, nxt = compare(s)
    assert nxt == [0, 0, 2, 3, 3, 3, 3, 4]


def test_rows_without_weight_and_strange_values():
    s = made(2, [3, 3, 2, 1, 1], 64, tree=False, pad=0)
    p, q = s["probs"], s["draft"]
    p[0], q[0] = 0.5 * p[0], p[0].clone()                  # a rejection leaves nothing of the target: its row again
    s["uniform"][1] = 0.9
    p[3] = 0
    q[3] = 0
    p[6] = -p[6]
    p[8, 5] = math.nan
    p[8, 6] = -3.0
    p[9] = 0
    p[9, 11] = math.inf
    q[6, 3] = math.nan
    acc, nxt = compare(s)
    assert acc[0] == 1 and nxt[0] >= 0 and nxt[1] == -1 and nxt[4] == 11


def test_the_same_token_among_siblings():
    for draft in ("drawn", "best"):
        s = made(3, [6, 6], 10, draft=draft)
        s["parents"] = torch.zeros(15, dtype=torch.int32)
        s["tokens"] = torch.tensor([0, 4, 4, 4, 5, 4, 0, 1, 1, 2, 1, 2, 0, 0, 0], dtype=torch.int32)
        s["uniform"].fill_(0.999)
        compare(s)


def test_strided_rows():
    s = made(4, [5, 7], 321)
    wide = torch.randn(s["rows"], 2, 400).cuda()
    wide[:, 0, 3:324], wide[:, 1, 5:326] = s["probs"].cuda(), s["draft"].cuda()
    want = plain(s)
    s["probs"], s["draft"] = wide[:, 0, 3:324], wide[:, 1, 5:326]
    out, _, _ = call(s)
    assert out["accepted"].tolist() == want[0] and out["next_tokens"].tolist() == want[2]


@pytest.mark.parametrize("draft", ["drawn", "distinct", "best"])
def test_tokens_come_out_as_the_target_gives_them(draft):
    """40,000 requests with the same distributions and trees drawn by the draft: the first token behind
    the root is distributed as the target's row. Within 5.5 standard deviations for each of 6 tokens
    (a chance of 2e-7 for all three drafts)."""
    n, vocab = 40000, 6
    g = gen_of(17)
    p = torch.tensor([0.05, 0.3, 0.2, 0.25, 0.15, 0.05])
    q = torch.tensor([0.3, 0.1, 0.2, 0.05, 0.05, 0.3])
    probs = p.repeat(4 * n, 1)
    if draft == "best":
        t = torch.tensor([1, 3, 2]).repeat(n, 1)
    else:
        t = torch.multinomial(q.repeat(n, 1), 3, replacement=draft == "drawn", generator=g)
    tokens = torch.zeros(n, 4, dtype=torch.int32)
    tokens[:, 1:] = t
    s = dict(probs=probs, draft=None if draft == "best" else q.repeat(4 * n, 1), tokens=tokens.flatten(),
             parents=torch.tensor([-1, 0, 0, 0], dtype=torch.int32).repeat(n), uniform=torch.rand(4 * n, generator=g),
             cu=list(range(0, 4 * n + 1, 4)), vocab=vocab, distinct=draft == "distinct", rows=4 * n)
    out, _, _ = call(s)
    took = out["accepted"] == 2
    second = out["rows"].view(n, 4)[:, 1].long()
    first = torch.where(took, tokens.flatten()[second.clamp(min=0)].long(), out["next_tokens"].long())
    got = torch.bincount(first, minlength=vocab).double() / n
    sd = torch.sqrt(p.double() * (1 - p.double()) / n)
    assert ((got - p.double()).abs() <= 5.5 * sd).all(), got
    assert 0.2 < took.double().mean() < 0.999


def test_errors_stay_with_their_request():
    for many in (False, True):
        counts = [4, 3, 5, 2, 3] + ([1] * 1100 if many else [])
        good = made(6, counts, 40, pad=0)
        want = plain(good)
        for what in ("token", "parent", "later", "cu"):
            s = dict(good, tokens=good["tokens"].clone(), parents=good["parents"].clone(), cu=list(good["cu"]))
            bad = {2}
            if what == "token":
                s["tokens"][s["cu"][2] + 4] = 40
            elif what == "parent":
                s["parents"][s["cu"][2] + 1] = 1
            elif what == "later":
                s["tokens"][s["cu"][2] + 3] = -1
            else:
                s["cu"][3] = s["cu"][2] - 1                       # request 2 descends, request 3 has more rows
                bad = {2, 3}
            n = len(s["cu"]) - 1
            v = Verifier(n, 40)
            out = [i32([-7] * n), i32([-7] * s["rows"]), i32([-7] * n)]
            v.verify_into(s["probs"].cuda(), s["tokens"].cuda(), i32(s["cu"]), s["uniform"].cuda(), *out, parents=s["parents"].cuda(),
                          draft_probs=s["draft"].cuda())
            with pytest.raises(SKVError, match="INVALID_ARG"):
                v.check_status("verify")
            acc, nxt = out[0].tolist(), out[2].tolist()
            assert acc[2] == 0 and nxt[2] == -1
            for r in range(n):
                if r not in bad:
                    assert acc[r] == want[0][r] and nxt[r] == want[2][r], (what, r)
            # the next call is sound
            v.verify_into(good["probs"].cuda(), good["tokens"].cuda(), i32(good["cu"]), good["uniform"].cuda(), *out,
                          parents=good["parents"].cuda(), draft_probs=good["draft"].cuda())
            v.check_status("verify")
            assert out[0].tolist() == want[0] and out[2].tolist() == want[2]


def test_too_many_nodes_without_draft_probabilities():
    n = 4097
    v = Verifier(1, 8)
    out = [i32([-7]), i32([-7] * n), i32([-7])]
    v.verify_into(torch.full((n, 8), 0.125).cuda(), i32([1] * n), i32([0, n]), torch.rand(n).cuda(), *out)
    with pytest.raises(SKVError, match="INVALID_ARG"):
        v.check_status("verify")
    assert out[0].tolist() == [0] and out[2].tolist() == [-1] and (out[1] == -1).all()
    v.verify_into(torch.full((n, 8), 0.125).cuda(), i32([1] * n), i32([0, n - 1]), torch.rand(n).cuda(), *out)
    v.check_status("verify")
    assert out[1][-1] == -1


def test_rejections_of_every_sibling_without_draft_probabilities():
    """4,095 children, all rejected, most of them seen before: what is left is drawn from."""
    n, vocab = 4096, 5000
    g = gen_of(4)
    p = torch.zeros(n, vocab)
    p[0] = torch.rand(vocab, generator=g)
    p[0] /= p[0].sum()
    s = dict(probs=p, draft=None, tokens=torch.randint(0, 3000, (n,), generator=g, dtype=torch.int32), parents=torch.zeros(n, dtype=torch.int32),
             uniform=torch.full((n,), 0.9999), cu=[0, n], vocab=vocab, distinct=False, rows=n)
    s["uniform"][0] = 0.4
    compare(s)


def test_in_a_graph_and_on_another_stream():
    s = made(9, [6, 9, 1], 5000, pad=0)
    want = plain(s)
    n = 3
    v = Verifier(n, 5000)
    args = (s["probs"].cuda(), s["tokens"].cuda(), i32(s["cu"]), s["uniform"].cuda())
    kw = dict(parents=s["parents"].cuda(), draft_probs=s["draft"].cuda())
    out = [i32([-7] * n), i32([-7] * s["rows"]), i32([-7] * n)]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        v.verify_into(*args, *out, **kw)
    for _ in range(3):
        for t in out:
            t.fill_(-7)
        g.replay()
        v.check_status("graph")
        assert out[0].tolist() == want[0] and out[2].tolist() == want[2]
    side = torch.cuda.Stream()
    torch.cuda._sleep(200_000_000)
    got = v.verify(*args, stream=side, **kw)
    assert got[0].tolist() == want[0] and got[2].tolist() == want[2] and len(got) == 3


def test_what_the_wrapper_refuses():
    s = made(9, [6, 9], 50, pad=0)
    v = Verifier(2, 50)
    good = dict(probs=s["probs"].cuda(), tokens=s["tokens"].cuda(), cu_new=i32(s["cu"]), uniform=s["uniform"].cuda(), accepted=i32([0, 0]),
                rows=i32([0] * 15), next_tokens=i32([0, 0]), parents=s["parents"].cuda(), draft_probs=s["draft"].cuda())
    v.verify_into(**good)
    v.check_status("verify")
    slots = torch.zeros(15, dtype=torch.int64, device="cuda")
    for kw in (dict(probs=s["probs"]), dict(probs=good["probs"][:, :49]), dict(probs=good["probs"].half()), dict(draft_probs=good["probs"].bfloat16()),
               dict(tokens=good["tokens"].long()), dict(cu_new=i32([0, 15])), dict(uniform=good["uniform"].double()), dict(accepted=i32([0])),
               dict(rows=i32([0] * 14)), dict(slots=slots), dict(kept=slots), dict(ctx_len=i32([0, 0])), dict(slots=slots, kept=slots[:3]),
               dict(parents=good["parents"][:5]), dict(probs=good["probs"].t().contiguous().t())):
        with pytest.raises(ValueError):
            v.verify_into(**dict(good, **kw))
    assert np.isfinite(float(v.status))
