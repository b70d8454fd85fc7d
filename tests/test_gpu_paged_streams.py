"""The paged-cache calls on a stream that is not the current one, and what an object keeps
between calls: nothing that a call needs may still wait on another stream, and nothing
that a captured graph holds may be given away."""
import pytest
import torch

from tests.test_gpu_paged import attend_case, gen_of, i32, pool_of
from lossless_kv_cache_scalar_gb300 import Coder, Layout, PagedKV, PagePool, SKVError, synth

pytestmark = pytest.mark.gpu


def busy():
    """Keeps the current stream at work for some 0.2 s."""
    torch.cuda._sleep(400_000_000)


def dirty(n_bytes, count=1):
    """Leaves blocks of that size full of ones with the allocator of the current stream."""
    blocks = [torch.full((n_bytes,), 255, dtype=torch.uint8, device="cuda") for _ in range(count)]
    torch.cuda.synchronize()
    return blocks


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


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("nodes", [1, 40])
def test_attend_makes_its_workspace_on_the_given_stream(nodes, dtype):
    """A first call without q_heads: the counters are 0 before the kernel reads them."""
    s = case(nodes, dtype)
    want, cache, side = expected(s, nodes), cache_of(s), torch.cuda.Stream()
    n_bytes = cache_of(s, q_heads=8).workspace.numel()
    blocks = dirty(n_bytes, 3)
    with torch.cuda.stream(side):
        blocks += dirty(n_bytes, 3)
    del blocks
    got = torch.zeros_like(want)
    torch.cuda.synchronize()
    busy()
    cache.status.fill_(-1)                           # behind the busy stream's work: must not be what stays
    torch.cuda.synchronize()
    busy()
    cache.attend_into(s["q"], s["ctx"], s["cu"], got, mask=s["mask"], max_nodes=nodes, stream=side)
    torch.cuda.synchronize()
    assert int(cache.status.item()) == 0
    assert torch.equal(got, want)
    cache.attend_into(s["q"], s["ctx"], s["cu"], got.zero_(), mask=s["mask"], max_nodes=nodes)
    assert torch.equal(got, want)


@pytest.mark.parametrize("nodes", [1, 40])
def test_a_new_object_is_ready_for_any_stream(nodes):
    """What a constructor fills is filled when it returns: a status that a call on another stream
    writes is not wiped by the constructor's zeros."""
    s = case(nodes, "bf16")
    s["table"][1, 2] = 10 ** 6                        # outside the pool
    out, side = torch.zeros_like(s["q"]).contiguous(), torch.cuda.Stream()
    torch.cuda.synchronize()
    busy()
    cache = cache_of(s, q_heads=8)
    cache.attend_into(s["q"], s["ctx"], s["cu"], out, mask=s["mask"], max_nodes=nodes, stream=side)
    torch.cuda.synchronize()
    assert int(cache.status.item()) == 7


def test_a_new_pool_is_ready_for_any_stream():
    ctx, new, side = i32([0, 0]), i32([20, 5]), torch.cuda.Stream()
    blocks = dirty(512, 20)
    del blocks
    torch.cuda.synchronize()
    busy()
    pool = PagePool(2, 4, 16, 8)
    cu, slots = pool.step(ctx, new, 32, stream=side)
    torch.cuda.synchronize()
    assert cu.tolist() == [0, 20, 25]
    assert slots.tolist() == list(range(20)) + list(range(32, 37)) + [-1] * 7
    assert pool.block_table[:, :2].tolist() == [[0, 1], [2, -1]]


def test_pool_step_takes_no_memory_that_the_current_stream_still_writes():
    """cu_new and slots of a step on another stream: not a block whose last use is still on its way."""
    ctx, new, side, pool = i32([0, 0]), i32([20, 5]), torch.cuda.Stream(), PagePool(2, 4, 16, 8)
    torch.cuda.synchronize()
    old = [torch.empty(n, dtype=t, device="cuda") for n, t in ((32, torch.int64), (3, torch.int32)) for _ in range(8)]
    busy()
    for t in old:
        t.fill_(77)
    del old, t
    cu, slots = pool.step(ctx, new, 32, stream=side)
    torch.cuda.synchronize()
    assert cu.tolist() == [0, 20, 25]
    assert slots.tolist() == list(range(20)) + list(range(32, 37)) + [-1] * 7


@pytest.mark.parametrize("nodes", [1, 40])
def test_a_graph_keeps_its_workspace(nodes):
    """A capture with one number of query heads, then a call with another, then other tensors:
    a replay gives what it gave, and writes to nobody else's memory."""
    s = case(nodes, "bf16")
    cache = cache_of(s, q_heads=8)
    out = torch.zeros_like(s["q"]).contiguous()
    half = s["q"][:, ::2]

    def step():
        cache.attend_into(s["q"], s["ctx"], s["cu"], out, mask=s["mask"], max_nodes=nodes)

    step()
    torch.cuda.synchronize()
    want = out.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    n_bytes = cache.workspace.numel()
    eager = cache.attend(half, s["ctx"], s["cu"], mask=s["mask"], max_nodes=nodes)
    others = dirty(n_bytes, 4)
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    for t in others:
        assert (t == 255).all()
    assert torch.equal(cache.attend(half, s["ctx"], s["cu"], mask=s["mask"], max_nodes=nodes), eager)


def test_no_workspace_is_made_in_a_capture_of_the_given_stream():
    """The capture that counts is the given stream's, not the current one's."""
    s = case(1, "bf16")
    cache = cache_of(s)
    out = torch.zeros_like(s["q"]).contiguous()
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        with torch.cuda.stream(other):
            with pytest.raises(ValueError):
                cache.attend_into(s["q"], s["ctx"], s["cu"], out, mask=s["mask"], max_nodes=1, stream=side)
    assert cache.workspace is None


def test_pool_step_refuses_a_capture():
    """A step swaps its buffers on the host: replayed, it would read the same counts for ever."""
    ctx, new, pool = i32([0, 0]), i32([20, 5]), PagePool(2, 4, 16, 8)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        with pytest.raises(ValueError):
            pool.step(ctx, new, 32, check=False)
    cu, slots = pool.step(ctx, new, 32)
    assert cu.tolist() == [0, 20, 25] and pool.n_pages.tolist() == [2, 1]


def test_decode_chunks_fills_its_pages_on_the_given_stream():
    cfg = synth.CONFIGS["tiny"].scaled(n_tokens=600)
    w = {k: v.cuda() for k, v in synth.generate(cfg).items()}
    lay = Layout("bf16", cfg.n_layers, cfg.n_kv, cfg.n_heads, cfg.head_dim, 600, tokens_per_chunk=256)
    coder, side = Coder(lay), torch.cuda.Stream()
    bits, offs = coder.encode(w["kv"], w["mu"], w["sigma"], w["counts"])
    ids = i32([2, 0, 1])
    want = coder.decode_chunks(bits, offs, w["mu"], w["sigma"], w["counts"], ids)
    torch.cuda.synchronize()
    busy()
    got = coder.decode_chunks(bits, offs, w["mu"], w["sigma"], w["counts"], ids, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(got, want)


def test_append_on_a_given_stream():
    """Rows and their status, with the current stream busy."""
    g, side = gen_of(83), torch.cuda.Stream()
    k, v = (pool_of(4, 16, 2, 64, "bf16", g) for _ in range(2))
    new = torch.randn(9, 2, 64, generator=g, device="cuda").to(torch.bfloat16)
    slots = torch.arange(9, dtype=torch.int64, device="cuda") * 7
    slots[8] = 64
    torch.cuda.synchronize()
    busy()
    cache = PagedKV(k, v)
    with pytest.raises(SKVError):
        cache.append(new, new, slots, stream=side)
    torch.cuda.synchronize()
    assert int(cache.status.item()) == 1
    assert torch.equal(k.view(-1, 2, 64)[slots[:8]], new[:8])


def test_results_may_be_used_on_the_current_stream():
    """What a call on another stream returned is read on the current one and given up there: the
    next call on the other stream takes no memory that is still read."""
    s = case(1, "bf16")
    cache, side = cache_of(s, q_heads=8), torch.cuda.Stream()
    args = (s["ctx"], s["cu"], s["mask"])
    want = cache.attend(s["q"], *args, max_nodes=1, stream=side).clone()
    pool, ctx, new = PagePool(2, 4, 16, 8), i32([0, 0]), i32([20, 5])
    cfg = synth.CONFIGS["tiny"].scaled(n_tokens=600)
    w = {k: v.cuda() for k, v in synth.generate(cfg).items()}
    coder = Coder(Layout("bf16", cfg.n_layers, cfg.n_kv, cfg.n_heads, cfg.head_dim, 600, tokens_per_chunk=256))
    bits, offs = coder.encode(w["kv"], w["mu"], w["sigma"], w["counts"])
    ids, others = i32([2, 0, 1]), i32([0, 1, 2])
    pages = coder.decode_chunks(bits, offs, w["mu"], w["sigma"], w["counts"], ids).clone()
    turned = -s["q"]
    torch.cuda.synchronize()

    out = cache.attend(s["q"], *args, max_nodes=1, stream=side)
    cu, slots = pool.step(ctx, new, 32, stream=side)
    got = coder.decode_chunks(bits, offs, w["mu"], w["sigma"], w["counts"], ids, stream=side)
    busy()
    read = [t.clone() for t in (out, cu, slots, got)]
    del out, cu, slots, got
    later = [cache.attend(turned, *args, max_nodes=1, stream=side), pool.step(i32([20, 5]), i32([1, 9]), 32, stream=side),
             coder.decode_chunks(bits, offs, w["mu"], w["sigma"], w["counts"], others, stream=side)]
    torch.cuda.synchronize()
    assert torch.equal(read[0], want) and torch.equal(read[3], pages)
    assert read[1].tolist() == [0, 20, 25]
    assert read[2].tolist() == list(range(20)) + list(range(32, 37)) + [-1] * 7
    del later


def test_pool_step_without_a_check_keeps_its_results():
    """A step that is not waited for: its results, given up at once, are not handed out while it writes."""
    pool, side = PagePool(2, 4, 16, 8), torch.cuda.Stream()
    ctx, new = i32([0, 0]), i32([20, 5])
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        busy()
    pool.step(ctx, new, 32, check=False, stream=side)
    later = [torch.full((n,), 77, dtype=t, device="cuda") for n, t in ((32, torch.int64), (3, torch.int32)) for _ in range(4)]
    torch.cuda.synchronize()
    for t in later:
        assert (t == 77).all()
