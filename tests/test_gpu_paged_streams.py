"""The paged-cache calls on a stream that is not the current one, and what an object keeps
between calls: nothing that a call needs may still wait on another stream, and nothing
that a captured graph holds may be given away."""
import pytest
import torch
from tests.test_gpu_paged import attend_case
from lossless_kv_cache_scalar_gb300 import PagedKV
pytestmark = pytest.mark.gpu


def busy():
    """Keeps the current stream at work for some 0.2 s."""
    torch.cuda._sleep(400_000_000)


def case(nodes, dtype, seed=81):
    return attend_case(seed, [1500, 300], [nodes, nodes], 16, 2, 4, 128, dtype)


def cache_of(s, **kw):
    return PagedKV(s["k"], s["v"], s["table"], k_scale=s["ks"], v_scale=s["vs"], **kw)


def expected(s, nodes):
    """The result where every stream is the current one, rows outside every request 0."""
    out = cache_of(s, q_heads=8).attend(s["q"], s["ctx"], s["cu"], mask=s["mask"], max_nodes=nodes)
    torch.cuda.synchronize()
    assert out.abs().sum() > 0
    return out


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("nodes", [1, 40])
def test_attend_fills_its_output_on_the_given_stream(nodes, dtype):
    s = case(nodes, dtype)
    want, cache, side = expected(s, nodes), cache_of(s, q_heads=8), torch.cuda.Stream()
    torch.cuda.synchronize()
    busy()
    got = cache.attend(s["q"], s["ctx"], s["cu"], mask=s["mask"], max_nodes=nodes, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
