"""Verification: requests of more nodes than are gathered at once, whose later nodes take the first ones' places."""
import pytest
import torch

from tests.test_gpu_verify import compare, i32
from lossless_kv_cache_scalar_gb300 import Verifier

pytestmark = pytest.mark.gpu


def long_requests(draft, n, nodes, vocab, seed):
    """Node 0's only child is rejected at once, and no other node is looked at: the walk passes all batches of nodes in no time.
    Node 0's u draws one token, those of the nodes that take its place draw another."""
    g = torch.Generator()
    g.manual_seed(seed)
    rows = n * nodes
    first = torch.rand(n, generator=g) < 0.5
    probs = torch.full((rows, vocab), 0.0)
    probs[:, 3], probs[:, vocab - 2] = 0.5, 0.5
    tokens = torch.full((rows,), 7, dtype=torch.int32)
    parents = torch.arange(-1, nodes - 1, dtype=torch.int32).repeat(n)
    uniform = torch.empty(n, nodes)
    uniform[:] = torch.where(first, 0.75, 0.25)[:, None]
    uniform[:, 0] = torch.where(first, 0.25, 0.75)
    uniform[:, 1] = 0.9
    s = dict(probs=probs, draft=None, tokens=tokens, parents=parents, uniform=uniform.flatten(), cu=list(range(0, rows + 1, nodes)), vocab=vocab,
             distinct=False, rows=rows)
    if draft:
        q = torch.zeros(rows, vocab)
        q[:, 7] = 1.0
        s["draft"] = q
    return s, torch.where(first, 3, vocab - 2).tolist()


@pytest.mark.parametrize("draft", [False, True])
@pytest.mark.parametrize("n,nodes,vocab", [(1, 257, 64), (40, 300, 64), (6, 1025, 5000), (3, 4096, 40)])
def test_the_first_nodes_number_draws_the_token(n, nodes, vocab, draft):
    s, want = long_requests(draft, n, nodes, vocab, n)
    accepted, nxt = compare(s)
    assert accepted == [1] * n and nxt == want


def test_many_times():
    n, nodes, vocab = 60, 300, 64
    s, want = long_requests(False, n, nodes, vocab, 5)
    v = Verifier(n, vocab)
    args = (s["probs"].cuda(), s["tokens"].cuda(), i32(s["cu"]), s["uniform"].cuda())
    parents, want = s["parents"].cuda(), i32(want)
    acc, rows, nxt = i32([0] * n), i32([0] * s["rows"]), i32([0] * n)
    wrong = torch.zeros(1, dtype=torch.int64, device="cuda")
    for _ in range(500):
        nxt.fill_(-7)
        v.verify_into(*args, acc, rows, nxt, parents=parents)
        wrong += (nxt != want).sum()
    v.check_status("verify")
    assert int(wrong) == 0
