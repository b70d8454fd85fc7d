"""Norms, rotation and row writes in one pass, against their 64-bit statement."""
import math

import pytest
import torch

from tests._pagedtest import E4M3, to_e4m3
from tests._servetest import angles, bf16_tol, e4m3_tol, far_angles, rotated
from lossless_kv_cache_scalar_gb300 import PagedKV, Rotary, SKVError

pytestmark = pytest.mark.gpu


def gen_of(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def freqs(rot, theta=1.0e6):
    return [theta ** (-2.0 * i / rot) for i in range(rot // 2)]


def made(seed, n, q_heads, heads, dim, page, dtype, skip=0.1):
    """Rows (slices of a fused projection), a cache of ones and slots in it."""
    g = gen_of(seed)
    wide = torch.randn(n, q_heads + 2 * heads, dim, generator=g) * torch.exp(torch.randn(q_heads + 2 * heads, dim, generator=g))
    wide = wide.to(torch.bfloat16).cuda()
    pages = -(-n // page) + 3
    slots = torch.randperm(pages * page, generator=g)[:n]
    slots[torch.rand(n, generator=g) < skip] = -1
    shape = (pages, page, heads, dim)
    if dtype == "bf16":
        k, v = (torch.full(shape, 1.0, dtype=torch.bfloat16).cuda() for _ in range(2))
        ks = vs = None
    else:
        k, v = (torch.full(shape, 0x38, dtype=torch.uint8).cuda() for _ in range(2))
        ks, vs = ((0.003 + 0.02 * torch.rand(heads, generator=g)).cuda() for _ in range(2))
    return dict(q=wide[:, :q_heads], kn=wide[:, q_heads:q_heads + heads], vn=wide[:, q_heads + heads:], k=k, v=v, ks=ks, vs=vs,
                slots=slots.cuda(), cache=PagedKV(k, v, k_scale=ks, v_scale=vs), gen=g)


def check(s, angle, q_norm, k_norm, eps, interleaved, amplitude, out):
    if out is not None:
        y, off = rotated(s["q"].cpu(), None if q_norm is None else q_norm.cpu(), eps, angle, interleaved, amplitude)
        d = (out.cpu().double() - y).abs()
        assert (d <= bf16_tol(y, off)).all(), (d / bf16_tol(y, off)).max()
    y, off = rotated(s["kn"].cpu(), None if k_norm is None else k_norm.cpu(), eps, angle, interleaved, amplitude)
    slots = s["slots"].cpu()
    live = slots >= 0
    at = slots[live]
    got_k, got_v = s["k"].flatten(0, 1).cpu(), s["v"].flatten(0, 1).cpu()
    if s["ks"] is None:
        d = (got_k[at].double() - y[live]).abs()
        assert (d <= bf16_tol(y[live], off[live])).all()
        assert torch.equal(got_v[at].view(torch.int16), s["vn"].cpu()[live].view(torch.int16))
        rest = torch.ones(got_k.shape[0], dtype=torch.bool)
        rest[at] = False
        assert (got_k[rest] == 1).all() and (got_v[rest] == 1).all()
    else:
        scale = s["ks"].cpu().double()[:, None]
        want = (y[live] / scale).clamp(-448, 448)
        d = (got_k[at].view(E4M3).double() - want).abs()
        assert (d <= e4m3_tol(want, off[live] / scale)).all()
        assert torch.equal(got_v[at], to_e4m3(s["vn"].cpu()[live].double() / s["vs"].cpu().double()[:, None]))
        rest = torch.ones(got_k.shape[0], dtype=torch.bool)
        rest[at] = False
        assert (got_k[rest] == 0x38).all() and (got_v[rest] == 0x38).all()


#        n, q heads, kv heads, dim, rot, interleaved, axes, norms, page
SHAPES = [(1, 32, 8, 128, 128, False, 1, True, 256), (1, 1, 1, 16, 16, True, 1, True, 1), (3, 5, 1, 96, 96, False, 3, True, 24),
          (7, 7, 7, 80, 32, True, 2, True, 16), (8, 32, 8, 128, 128, True, 1, False, 64), (33, 10, 2, 64, 64, False, 1, True, 7),
          (300, 40, 8, 128, 64, False, 3, True, 24), (61, 4, 4, 256, 256, False, 1, True, 16), (61, 16, 2, 256, 64, True, 4, True, 16),
          (500, 9, 3, 112, 112, False, 1, True, 33), (129, 3, 3, 32, 16, False, 1, True, 16), (2500, 6, 2, 64, 32, True, 1, True, 48),
          (2049, 8, 8, 48, 48, False, 1, False, 256), (40, 64, 1, 128, 0, False, 1, True, 16)]


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(str(int(x)) for x in s))
def test_against_64_bits(shape, dtype):
    n, qh, kh, dim, rot, inter, n_axes, norms, page = shape
    s = made(7 * n + dim, n, qh, kh, dim, page, dtype)
    g = s["gen"]
    f = freqs(rot) if rot else []
    axes = None if n_axes == 1 else [j % n_axes for j in range(rot // 2)]
    if axes is not None:
        axes[-1] = n_axes - 1
    qn, kn = ((1 + 0.3 * torch.randn(2, dim, generator=g)) if norms else (None, None))
    pos = torch.randint(0, 131072, (n_axes, n), generator=g, dtype=torch.int32)
    amp = 1.0 if n % 2 else 1.1875
    rotary = Rotary(dim, f, qn, kn, eps=1e-5, axes=axes, interleaved=inter, amplitude=amp)
    assert rotary.n_axes == n_axes
    out = s["cache"].rotate_append(rotary, s["q"], s["kn"], s["vn"], pos.cuda(), s["slots"])
    check(s, angles(pos, f, axes), qn, kn, 1e-5, inter, amp, out)


def test_far_and_negative_positions():
    pos = torch.tensor([[0, 1, -1, 131071, 1 << 20, (1 << 31) - 1, -(1 << 31), -12345678]], dtype=torch.int32)
    s = made(5, 8, 4, 2, 64, 16, "bf16", skip=0.0)
    f = [1.0, 2.5, -0.75, 1e-7] + freqs(56)
    out = s["cache"].rotate_append(Rotary(64, f), s["q"], s["kn"], s["vn"], pos.cuda(), s["slots"])
    check(s, far_angles(pos[0].tolist(), f), None, None, 0.0, False, 1.0, out)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("n", [5, 3000, 9001])
def test_without_rotation_it_is_append(n, dtype):
    """No norm and no frequencies: the pages get what append writes, bit for bit."""
    s = made(3, n, 4, 2, 96, 16, dtype)
    k2, v2 = s["k"].clone(), s["v"].clone()
    PagedKV(k2, v2, k_scale=s["ks"], v_scale=s["vs"]).append(s["kn"], s["vn"], s["slots"])
    out = s["cache"].rotate_append(Rotary(96, []), s["q"], s["kn"], s["vn"], torch.zeros(n, dtype=torch.int32, device="cuda"), s["slots"])
    assert torch.equal(out, s["q"])
    assert torch.equal(s["k"].view(torch.uint8), k2.view(torch.uint8)) and torch.equal(s["v"].view(torch.uint8), v2.view(torch.uint8))


def test_in_place_and_without_queries():
    s = made(4, 50, 4, 2, 128, 16, "bf16")
    pos = torch.arange(50, dtype=torch.int32, device="cuda") * 77
    w = 1 + 0.1 * torch.randn(128, generator=s["gen"])
    rotary = Rotary(128, freqs(128), w, w)
    want = s["cache"].rotate_append(rotary, s["q"], s["kn"], s["vn"], pos, s["slots"])
    k, v = s["k"].clone(), s["v"].clone()
    q = s["q"].contiguous()
    s["k"].fill_(1), s["v"].fill_(1)
    s["cache"].rotate_append_into(rotary, q, s["kn"], s["vn"], pos, s["slots"], q)
    assert torch.equal(q, want) and torch.equal(s["k"], k) and torch.equal(s["v"], v)
    s["k"].fill_(1), s["v"].fill_(1)
    assert s["cache"].rotate_append(rotary, None, s["kn"], s["vn"], pos, s["slots"]) is None
    assert torch.equal(s["k"], k) and torch.equal(s["v"], v)


def test_no_rows():
    s = made(4, 3, 4, 2, 128, 16, "bf16")
    e = torch.zeros(0, dtype=torch.int32, device="cuda")
    out = s["cache"].rotate_append(Rotary(128, freqs(128)), s["q"][:0], s["kn"][:0], s["vn"][:0], e, e.long())
    assert out.shape == (0, 4, 128)


def test_values_that_are_not_finite_stay_in_their_head():
    s = made(9, 6, 4, 2, 64, 16, "bf16", skip=0.0)
    pos = torch.arange(6, dtype=torch.int32, device="cuda")
    w = torch.ones(64)
    rotary = Rotary(64, freqs(32), w, w)
    want = s["cache"].rotate_append(rotary, s["q"], s["kn"], s["vn"], pos, s["slots"])
    k = s["k"].clone()
    s["q"][2, 1, 3], s["kn"][4, 0, 5] = math.nan, math.inf
    got = s["cache"].rotate_append(rotary, s["q"], s["kn"], s["vn"], pos, s["slots"])
    assert got[2, 1].isnan().all()
    got[2, 1] = want[2, 1]
    assert torch.equal(got, want)
    a = int(s["slots"][4])
    assert s["k"].flatten(0, 1)[a, 0].isnan().any()
    s["k"].flatten(0, 1)[a, 0] = k.flatten(0, 1)[a, 0]
    assert torch.equal(s["k"], k)


def test_channels_beyond_the_rotated_ones_take_nothing_from_them():
    s = made(9, 6, 4, 2, 64, 16, "bf16", skip=0.0)
    s["q"][:, :, 40] = math.inf
    out = s["cache"].rotate_append(Rotary(64, freqs(32)), s["q"], s["kn"], s["vn"], torch.arange(6, dtype=torch.int32, device="cuda"), s["slots"])
    assert (out[:, :, 40] == math.inf).all()
    assert torch.equal(out[:, :, 32:], s["q"][:, :, 32:]) and out[:, :, :32].isfinite().all()


@pytest.mark.parametrize("n,heads", [(40, 2), (2100, 2), (2100, 16), (5000, 16)])
def test_a_slot_beyond_the_pool(n, heads):
    s = made(11, n, heads, 2, 64, 16, "bf16", skip=0.0)
    pos = torch.zeros(n, dtype=torch.int32, device="cuda")
    good = s["slots"].clone()
    s["slots"][n - 2] = s["k"].shape[0] * 16
    with pytest.raises(SKVError, match="INVALID_ARG"):
        s["cache"].rotate_append(Rotary(64, freqs(64)), s["q"], s["kn"], s["vn"], pos, s["slots"])
    assert (s["k"].flatten(0, 1)[good[n - 2]] == 1).all()
    assert torch.equal(s["k"].flatten(0, 1)[good[n - 1]], s["kn"][n - 1])            # position 0
    s["slots"][n - 2] = good[n - 2]
    s["cache"].rotate_append(Rotary(64, freqs(64)), s["q"], s["kn"], s["vn"], pos, s["slots"])


def test_pools_with_strides_and_far_pages():
    """A pool of K and V pages in turn, more than 2^32 bytes of it."""
    pool = torch.empty(5000, 2, 64, 8, 128, dtype=torch.bfloat16, device="cuda")
    s = made(12, 9, 4, 8, 128, 64, "bf16", skip=0.0)
    slots = torch.tensor([4999 * 64 + 63 - i * 70 for i in range(9)], device="cuda")
    pos = torch.zeros(9, dtype=torch.int32, device="cuda")
    PagedKV(pool[:, 0], pool[:, 1]).rotate_append(Rotary(128, freqs(128)), s["q"], s["kn"], s["vn"], pos, slots)
    assert torch.equal(pool[slots // 64, 0, slots % 64], s["kn"]) and torch.equal(pool[slots // 64, 1, slots % 64], s["vn"])


def test_rows_far_into_a_large_tensor():
    """Rows whose elements lie beyond 2^31 of the first's."""
    n, wide = 3000, torch.empty(3000, 6000, 128, dtype=torch.bfloat16, device="cuda")          # 4.6 GB
    s = made(16, n, 2, 1, 128, 16, "bf16", skip=0.0)
    wide[:, 5996:5998], wide[:, 5998:5999], wide[:, 5999:] = s["q"], s["kn"], s["vn"]
    w, pos = torch.ones(128), torch.arange(n, dtype=torch.int32, device="cuda")
    rotary = Rotary(128, freqs(128), w, w)
    want = s["cache"].rotate_append(rotary, s["q"], s["kn"], s["vn"], pos, s["slots"])
    k = s["k"].clone()
    s["k"].fill_(1)
    got = s["cache"].rotate_append(rotary, wide[:, 5996:5998], wide[:, 5998:5999], wide[:, 5999:], pos, s["slots"])
    assert torch.equal(got, want) and torch.equal(s["k"], k)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_pages_with_heads_before_tokens(dtype):
    """Strides of their own for heads and tokens, K and V in one tensor: the same rows as in a plain pool."""
    s = made(15, 70, 4, 3, 96, 24, dtype)
    pages = s["k"].shape[0]
    both = torch.zeros(pages, 2, 3, 24, 96, dtype=s["k"].dtype, device="cuda")
    k, v = both[:, 0].transpose(1, 2), both[:, 1].transpose(1, 2)
    rotary, pos = Rotary(96, freqs(64), torch.ones(96), torch.ones(96)), torch.arange(70, dtype=torch.int32, device="cuda")
    want = s["cache"].rotate_append(rotary, s["q"], s["kn"], s["vn"], pos, s["slots"])
    got = PagedKV(k, v, k_scale=s["ks"], v_scale=s["vs"]).rotate_append(rotary, s["q"], s["kn"], s["vn"], pos, s["slots"])
    assert torch.equal(got, want)
    at = s["slots"][s["slots"] >= 0]
    for mine, plain in ((k, s["k"]), (v, s["v"])):
        assert torch.equal(mine[at // 24, at % 24].view(torch.uint8), plain[at // 24, at % 24].view(torch.uint8))
    left = torch.ones(pages * 24, dtype=torch.bool, device="cuda")
    left[at] = False
    assert not k.reshape(pages * 24, 3, 96)[left].float().any() and not v.reshape(pages * 24, 3, 96)[left].float().any()


def test_in_a_graph_and_on_another_stream():
    s = made(13, 30, 4, 2, 128, 16, "e4m3", skip=0.0)
    w = torch.ones(128)
    rotary = Rotary(128, freqs(128), w, w)
    pos = torch.arange(30, dtype=torch.int32, device="cuda")
    want = s["cache"].rotate_append(rotary, s["q"], s["kn"], s["vn"], pos, s["slots"])
    k = s["k"].clone()
    out, side = torch.empty_like(want), torch.cuda.Stream()
    s["k"].fill_(0)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        s["cache"].rotate_append_into(rotary, s["q"], s["kn"], s["vn"], pos, s["slots"], out)
    g.replay()
    torch.cuda.synchronize()
    s["cache"].check_status("graph")
    assert torch.equal(out, want)
    at = s["slots"]
    assert torch.equal(s["k"].flatten(0, 1)[at], k.flatten(0, 1)[at])
    torch.cuda._sleep(200_000_000)
    got = s["cache"].rotate_append(rotary, s["q"], s["kn"], s["vn"], pos, s["slots"], stream=side)
    assert torch.equal(got, want)


def test_what_the_wrapper_refuses():
    s = made(14, 4, 4, 2, 64, 16, "bf16")
    rotary, pos = Rotary(64, freqs(64)), torch.zeros(4, dtype=torch.int32, device="cuda")
    out = torch.empty(4, 4, 64, dtype=torch.bfloat16, device="cuda")
    c = s["cache"]
    good = dict(rotary=rotary, q=s["q"], k=s["kn"], v=s["vn"], positions=pos, slots=s["slots"], q_out=out)
    c.rotate_append_into(**good)
    for kw in (dict(rotary=Rotary(96, freqs(96))), dict(q=s["q"].float()), dict(q=s["q"][:3]), dict(q_out=out[:, :2]), dict(q_out=None), dict(q=None),
               dict(k=s["kn"][:, :1]), dict(v=s["vn"].contiguous()), dict(positions=pos.long()), dict(positions=pos[:3]), dict(slots=s["slots"].int()),
               dict(rotary=Rotary(64, freqs(64), axes=[0, 1] * 16)),
               dict(rotary=Rotary(64, freqs(64), axes=[0, 1] * 16), positions=torch.zeros(4, 2, dtype=torch.int32, device="cuda"))):
        with pytest.raises(ValueError):
            c.rotate_append_into(**dict(good, **kw))
    for a in (dict(inv_freq=freqs(80)), dict(inv_freq=[1.0] * 7), dict(inv_freq=[math.nan] * 8), dict(inv_freq=freqs(64), axes=[0]),
              dict(inv_freq=freqs(64), axes=[16] * 32), dict(inv_freq=freqs(64), q_norm=torch.ones(32)), dict(inv_freq=[], eps=-1.0)):
        with pytest.raises((ValueError, SKVError, RuntimeError)):
            Rotary(64, **a)
