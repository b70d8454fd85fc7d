"""Corners of the paged-cache operators' arithmetic: many small weights beside a large one,
scales at the ends of binary32, wide and narrow row tiles in one long list of work,
the kernel that a call takes by default, and pools of other types."""
import math
import random
import pytest
import torch

from tests import _pagedtest as P
from tests.test_gpu_paged import attend_case, check_attend, gen_of, i32, map_inputs, run_map
from lossless_kv_cache_scalar_gb300 import PagedKV

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("nodes,requests,ctx", [(1, 40, 2000), (40, 16, 2000), (1, 1, 20000)])
@pytest.mark.parametrize("where", ["first", "last"])
@pytest.mark.parametrize("above", [27.0, 7.9])
def test_attend_small_weights_beside_a_large_one(above, where, nodes, requests, ctx, dtype):
    """One position whose score lies `above` powers of two over all others and whose value is
    0: the output is what the others hold, each with a weight of 2^-above. A batch with as many
    items as CTAs, so that one CTA has all positions of a head; and one request, split over
    many. (7.9: the largest weight against a reference that has not moved.)"""
    g = gen_of(91)
    page, heads, group, dim = 256, 16, 2, 64
    pages = -(-(ctx + nodes) // page)
    kf = torch.randn(pages * page, heads, dim, generator=g, device="cuda") * 0.25
    vf = 1.0 + 0.5 * torch.rand(pages * page, heads, dim, generator=g, device="cuda")
    kf[:, :, 0] = 0.0
    at = 0 if where == "first" else ctx - 1
    kf[at], vf[at] = 0.0, 0.0
    kf[at, :, 0] = 8.0
    kind = torch.bfloat16 if dtype == "bf16" else P.E4M3
    k, v = (t.to(kind).view(pages, page, heads, dim) for t in (kf, vf))
    if dtype == "e4m3":
        k, v = k.view(torch.uint8), v.view(torch.uint8)
    scale = 0.125
    rows = requests * nodes
    q = torch.randn(rows, heads * group, dim, generator=g, device="cuda") * 0.5
    q[:, :, 0] = above * math.log(2.0) / (8.0 * scale)
    q = q.to(torch.bfloat16)
    ones = torch.ones(heads, device="cuda") if dtype == "e4m3" else None
    # every request reads the same pages
    table, lens, cu = i32([list(range(pages))] * requests), i32([ctx] * requests), i32(list(range(0, rows + 1, nodes)))
    out = PagedKV(k, v, table, k_scale=ones, v_scale=ones).attend(q, lens, cu, max_nodes=nodes, scale=scale)
    eps = dict(q_eps=2.0 ** -16, p_eps=2.0 ** -11) if dtype == "e4m3" else {}
    for r in {0, requests // 2, requests - 1}:
        for i in {0, nodes // 2, nodes - 1}:
            # node i of a chain is a single token over ctx + i positions
            row = slice(r * nodes + i, r * nodes + i + 1)
            o, tol, _, _ = P.attention(q[row], k, v, ones, ones, table[:1], i32([ctx + i]), i32([0, 1]), None, scale, **eps)
            # an e4m3 cache: fp16 weights are off by 2^-32 of the row's largest, or 2^-11 of themselves
            if dtype == "e4m3":
                tol = tol + 2.0 ** -32 * (ctx + i + 1) * 1.5
            if above == 27.0:
                assert float(o.min()) > 4 * float(tol.max())           # the tolerance tells the output from nothing
            over = (out[row].cpu().double() - o).abs() - tol
            assert (over <= 0).all(), float(over.max())


def near_ties(exponent):
    """bf16 values of that exponent and scales for which their quotients are ties of the 8-bit
    grid, or next to one."""
    x = torch.arange(128, 256, dtype=torch.float64) * 2.0 ** (exponent - 7)
    x = x[x == x.to(torch.bfloat16).double()]
    ties = torch.tensor([1.0625, 1.1875, 1.3125, 1.4375, 1.5625, 1.6875, 1.8125], dtype=torch.float64)
    s = (x[:, None] / ties).flatten().float()
    x = x.repeat_interleave(7)
    s = torch.cat([s, torch.nextafter(s, torch.full_like(s, math.inf)), torch.nextafter(s, torch.zeros_like(s))])
    x = x.repeat(3)
    keep = (s > 0) & torch.isfinite(s)
    return x[keep].to(torch.bfloat16), s[keep]


@pytest.mark.parametrize("exponent", [-131, -126, -124, -122, -120, -110, -101, -98, 98, 101, 120, 126, 127])
def test_append_rounds_the_real_quotient_at_the_ends_of_binary32(exponent):
    x, s = near_ties(exponent)
    heads = s.numel()
    k = torch.zeros(1, 1, heads, 16, dtype=torch.uint8, device="cuda")
    v = torch.zeros_like(k)
    new = x.view(1, heads, 1).expand(1, heads, 16).contiguous().cuda()
    PagedKV(k, v, k_scale=s.cuda(), v_scale=s.cuda()).append(new, -new, torch.zeros(1, dtype=torch.int64, device="cuda"))
    want = P.to_e4m3(x.double() / s.double())
    assert torch.equal(k[0, 0, :, 0].cpu(), want) and torch.equal(v[0, 0, :, 5].cpu(), want | 128)


@pytest.mark.parametrize("scale", [1e-45, 1e-40, 1e-37, 3e-31, 3e31, 1e38, 3.4e38])
def test_append_with_scales_far_from_the_values(scale):
    """Values of any size against scales of any size: saturated, or 0 with the value's sign."""
    x = torch.tensor([0.0, -0.0, 1.0, -1.0, 3e38, -3e38, 1e-38, -1e-38, 9.2e-41, -9.2e-41, math.inf, -math.inf, math.nan, 448.0, 0.01, 7.0],
                     dtype=torch.float64).to(torch.bfloat16)
    s = torch.tensor([scale], dtype=torch.float32)
    k = torch.zeros(1, 1, 1, 16, dtype=torch.uint8, device="cuda")
    v = torch.zeros_like(k)
    PagedKV(k, v, k_scale=s.cuda(), v_scale=s.cuda()).append(x.view(1, 1, 16).cuda(), x.view(1, 1, 16).cuda(),
                                                             torch.zeros(1, dtype=torch.int64, device="cuda"))
    want = P.to_e4m3(x.double() / s.double())
    for got in (k, v):
        got = got.flatten().cpu()
        nan = (want & 127) == 127
        assert torch.equal((got & 127) == 127, nan) and torch.equal(got[~nan], want[~nan])


@pytest.mark.parametrize("dtype,dim", [("bf16", 64), ("bf16", 80), ("e4m3", 64), ("e4m3", 80)])
def test_attend_wide_and_narrow_row_tiles_in_a_long_list(dtype, dim):
    """Row tiles of 256, 4, 140 and 6 rows among 3,920 units of work, above the 2,432 from which runs
    of wide and of narrow tiles count 4 and 3, so that shares end anywhere in either."""
    ctx, new, heads, group = [3000, 1500, 700], [130, 70, 3], 16, 2
    units = sum(heads * -(-(c + n) // 128) * (4 * (n * group // 256) + (4 if n * group % 256 > 128 else 3 if n * group % 256 else 0))
                for c, n in zip(ctx, new))
    assert units > 4 * 4 * 152
    s = attend_case(93, ctx, new, 64, heads, group, dim, dtype)
    check_attend(s, max_nodes=130)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_attend_takes_single_tokens_for_single_tokens(dtype):
    """Without max_nodes a batch of single tokens is one, whatever the number of requests: the
    same bits as with max_nodes=1."""
    s = attend_case(95, [900 + 37 * i for i in range(40)], [1] * 40, 16, 2, 8, 128, dtype)
    q = s["q"][:40]
    cache = PagedKV(s["k"], s["v"], s["table"], k_scale=s["ks"], v_scale=s["vs"], q_heads=16)
    assert torch.equal(cache.attend(q, s["ctx"], s["cu"]), cache.attend(q, s["ctx"], s["cu"], max_nodes=1))


@pytest.mark.parametrize("kind", [torch.float16, torch.float8_e5m2, torch.float8_e4m3fnuz, torch.bool])
def test_pools_of_other_types_are_refused(kind):
    """Codes of the right size and the wrong meaning."""
    k = torch.zeros(2, 16, 2, 64, device="cuda").to(kind)
    with pytest.raises(ValueError):
        PagedKV(k, k.clone())


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.int16, torch.uint16, torch.uint8, torch.int8, torch.float8_e4m3fn])
def test_pools_of_codes_are_taken(kind):
    shape = (2, 16, 2, 64)
    k, v = (torch.zeros(shape, dtype=torch.int16 if kind.itemsize == 2 else torch.uint8, device="cuda").view(kind) for _ in range(2))
    new = torch.ones(1, 2, 64, dtype=torch.bfloat16, device="cuda")
    PagedKV(k, v).append(new, new, torch.zeros(1, dtype=torch.int64, device="cuda"))
    one = k.view(torch.bfloat16) if kind.itemsize == 2 else k.view(P.E4M3)
    assert (one[0, 0].float() == 1).all()


@pytest.mark.parametrize("nodes", [1, 40])
@pytest.mark.parametrize("scale", [1e-35, -1e-35, 0.0])
def test_attend_tiny_scales_of_large_values(scale, nodes):
    """Products of 1e35 and a scale that makes ordinary scores of them, or none at all."""
    s = attend_case(97, [300, 20], [nodes, nodes], 16, 2, 4, 64, "bf16")
    for name in ("q", "k"):
        s[name] = (s[name].float() * 2.0 ** 56).to(torch.bfloat16)
    check_attend(s, max_nodes=nodes, scale=scale)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("dim", [16, 32, 112])
@pytest.mark.parametrize("page", [16, 24])
def test_attend_trees_of_other_head_sizes(page, dim, dtype):
    """Heads that fill a part of a copy's box, one of their blocks or none of the second."""
    s = attend_case(99 + dim, [333, 130], [40, 9], page, 2, 4, dim, dtype, garbage=math.nan)
    check_attend(s, max_nodes=40)


def test_append_slots_beyond_31_bits():
    """A pool of 2^32 token slots (pages 16 bytes apart: nothing that is written lies twice)."""
    base_k, base_v = (torch.zeros((1 << 20) + 4096, 16, dtype=torch.uint8, device="cuda") for _ in range(2))
    k, v = (t.as_strided((4096, 1 << 20, 1, 16), (16, 16, 16, 1)) for t in (base_k, base_v))
    pages, tokens = [0, 2047, 2048, 4095, 4000], [5, 77, 1000, (1 << 20) - 1, 9]
    slots = torch.tensor([p * (1 << 20) + t for p, t in zip(pages, tokens)] + [1 << 32, -1], dtype=torch.int64, device="cuda")
    new = torch.arange(1, 8, device="cuda").view(7, 1, 1).expand(7, 1, 16).to(torch.bfloat16).contiguous()
    cache = PagedKV(k, v)
    cache.append_into(new, -new, slots)
    torch.cuda.synchronize()
    assert int(cache.status.item()) == 1                    # the slot just behind the pool
    want = torch.zeros_like(base_k).view(P.E4M3).float()
    for i, (p, t) in enumerate(zip(pages, tokens)):
        want[p + t] = float(i + 1)
    assert torch.equal(base_k.view(P.E4M3).float(), want) and torch.equal(base_v.view(P.E4M3).float(), -want)


@pytest.mark.parametrize("b,page,max_new,more", [(4096, 16, 3, 7), (4097, 24, 9, 0), (9000, 5, 20, 30000)])
def test_page_map_of_many_requests(b, page, max_new, more):
    """More requests than one scan of the block holds."""
    rng = random.Random(b)
    ctx, new, have, table, free, state, pool, width = map_inputs(rng, b, page, 60, max_new, 0.2)
    cap = sum(new) + more
    want = P.page_map(page, pool, width, cap, ctx, new, table, have, free, state)
    got = run_map(page, pool, width, cap, ctx, new, table, have, free, state)
    for name, x, y in zip(("table", "n_pages", "free", "state", "cu", "slots"), got, want):
        assert x == y, name
