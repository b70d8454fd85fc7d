"""The example of a drafted step over so short a context that the drafted tokens hold much of
the weight: what is written where, and that a wrong path, mask or place would show."""
import importlib.util
import math
import os

import pytest
import torch

from tests import _pagedtest as P

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    at = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "draft_step.py")
    spec = importlib.util.spec_from_file_location("draft_step_path", at)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("tokens", [1, 3])
def test_the_accepted_path(example, tokens):
    s = example.step(tokens=tokens)
    cache, pool, path, n = s["cache"], s["pool"], s["path"], len(s["parents"])
    heads, dim = s["k"].shape[1:]
    flat_k, flat_v = (p.view(torch.bfloat16).reshape(-1, heads, dim) for p in (cache.k_pages, cache.v_pages))
    # the accepted rows lie, bit for bit and in order, behind the context; the other drafted rows where they were
    assert s["slots"].tolist() == list(range(tokens, tokens + n))
    at = s["slots"][:len(path)]
    assert torch.equal(flat_k[at], s["k"][path]) and torch.equal(flat_v[at], s["v"][path])
    rest = s["slots"][len(path):]
    assert torch.equal(flat_k[rest], s["k"][len(path):]) and torch.equal(flat_v[rest], s["v"][len(path):])

    scale, ctx = 1.0 / math.sqrt(dim), i32([tokens])
    node = path[-1]

    def exact(rows):
        """The last accepted token over the context and these drafted rows, in 64 bits."""
        k, v = (torch.cat([f[:tokens], new[rows]])[None] for f, new in ((flat_k, s["k"]), (flat_v, s["v"])))
        o, tol, _, _ = P.attention(s["q"][node:node + 1], k, v, None, None, i32([[0]]), i32([tokens + len(rows) - 1]), i32([0, 1]),
                                   None, scale)
        return o[0], tol[0]

    o, tol = exact(path)
    tree, single = s["out"][node].cpu().double(), s["again"][0].cpu().double()
    assert ((tree - o).abs() <= tol).all() and ((single - o).abs() <= tol).all()
    # the same check tells every other path from this one
    for wrong in ([0, 1, 2, 3, 4], path[:-1], [node], [9, 10, 5, 7, 4], list(range(n))):
        assert ((exact(wrong)[0] - o).abs() > 4 * tol).float().mean() > 0.3, wrong
    # and a cache that holds another path gives another answer
    cache.append(s["k"], s["v"], at, rows=i32([9, 10, 5, 7, 4]))
    ctx.fill_(tokens + len(path) - 1)
    other = cache.attend(s["q"][node:node + 1], ctx, i32([0, 1]), max_nodes=1)[0].cpu().double()
    assert ((other - o).abs() > tol).float().mean() > 0.3
