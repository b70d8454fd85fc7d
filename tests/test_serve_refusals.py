"""The operators around a paged cache refuse bad arguments on the host, before any CUDA call
(checked here through the C ABI with addresses that are never read), and so do their Python
wrappers."""
import ctypes as C
import math

import pytest
import torch

from lossless_kv_cache_scalar_gb300 import Rotary, Verifier
from lossless_kv_cache_scalar_gb300 import _binding as B
from lossless_kv_cache_scalar_gb300.serve import _turns
from tests.test_paged_refusals import A, BAD, cache


def rotary(**kw):
    f = dict(version=1, head_dim=128, rot_dim=128, n_axes=1, interleaved=0, eps=1e-6, amplitude=1.0, turns=A, axis=None, q_norm=A, k_norm=None)
    f.update(kw)
    return B.skv_rotary(**f)


def test_good_rotaries():
    for kw in ({}, dict(rot_dim=0, turns=None), dict(axis=A + 1, n_axes=16), dict(head_dim=16, rot_dim=16), dict(eps=0.0, interleaved=1)):
        assert B.lib().skv_rotary_check(C.byref(rotary(**kw))) == 0, kw
    assert B.lib().skv_rotary_check(None) == BAD


ROTATE = dict(q=A, q_row_stride=4096, q_head_stride=128, n_q_heads=32, k=A, v=A, row_stride=1024, row_head_stride=128, positions=A, slots=A, n=4, q_out=A,
              status=A, stream=None)


@pytest.mark.parametrize("kw", [dict(version=0), dict(head_dim=0), dict(head_dim=24), dict(head_dim=272), dict(rot_dim=8), dict(rot_dim=144), dict(n_axes=0),
                                dict(n_axes=17), dict(interleaved=2), dict(eps=-1.0), dict(eps=math.nan), dict(amplitude=math.inf), dict(turns=None),
                                dict(turns=A + 4), dict(q_norm=A + 8), dict(k_norm=A + 4)])
def test_bad_rotaries(kw):
    r = rotary(**kw)
    assert B.lib().skv_rotary_check(C.byref(r)) == BAD
    assert B.lib().skv_rotate_append(C.byref(cache()), C.byref(r), *ROTATE.values()) == BAD


@pytest.mark.parametrize("kw", [dict(q=None), dict(q=A + 8), dict(q_row_stride=4), dict(q_head_stride=1), dict(n_q_heads=65536), dict(k=None), dict(v=A + 8),
                                dict(row_stride=1020), dict(row_head_stride=4), dict(positions=None), dict(positions=A + 2), dict(slots=None),
                                dict(slots=A + 4), dict(q_out=None), dict(q_out=A + 4), dict(status=None), dict(n=1 << 31), dict(q_row_stride=1 << 41)])
def test_bad_rotate_arguments(kw):
    assert B.lib().skv_rotate_append(C.byref(cache()), C.byref(rotary()), *dict(ROTATE, **kw).values()) == BAD


def test_rotary_and_cache_go_together():
    assert B.lib().skv_rotate_append(C.byref(cache()), C.byref(rotary(head_dim=64, rot_dim=64)), *ROTATE.values()) == BAD
    assert B.lib().skv_rotate_append(C.byref(cache(head_stride=0)), C.byref(rotary()), *ROTATE.values()) == BAD


VERIFY = dict(dtype=0, probs=A, probs_stride=50, draft_probs=A, draft_stride=50, vocab=50, distinct=0, n_rows=4, n_requests=2, cu_new=A, tokens=A, parents=A,
              uniform=A, slots=A, ctx_len=A, accepted=A, rows=A, kept=A, ctx_out=A, next=A, status=A, stream=None)


@pytest.mark.parametrize("kw", [dict(dtype=2), dict(probs=None), dict(probs=A + 2), dict(probs_stride=49), dict(draft_stride=49), dict(vocab=0),
                                dict(vocab=(1 << 19) + 1, probs_stride=1 << 20, draft_stride=1 << 20), dict(distinct=2), dict(n_rows=1 << 31),
                                dict(n_requests=(1 << 26) + 1), dict(cu_new=None), dict(tokens=None), dict(uniform=None), dict(slots=None), dict(kept=None),
                                dict(ctx_len=None), dict(ctx_out=None), dict(accepted=None), dict(rows=None), dict(next=None), dict(status=None),
                                dict(cu_new=A + 2), dict(parents=A + 1), dict(slots=A + 4), dict(dtype=1, draft_probs=A + 1), dict(probs_stride=1 << 41)])
def test_bad_verify_arguments(kw):
    assert B.lib().skv_tree_verify(*dict(VERIFY, **kw).values()) == BAD


MOVE = dict(n_requests=2, cu_new=A, n_rows=4, rows=A, slots=A, kept=A, status=A, stream=None)


@pytest.mark.parametrize("kw", [dict(cu_new=None), dict(cu_new=A + 2), dict(n_rows=1 << 31), dict(rows=None), dict(slots=None), dict(kept=A + 4),
                                dict(status=None), dict(n_requests=1 << 31)])
def test_bad_move_arguments(kw):
    assert B.lib().skv_cache_move(C.byref(cache()), *dict(MOVE, **kw).values()) == BAD
    assert B.lib().skv_cache_move(C.byref(cache(n_pages=0)), *MOVE.values()) == BAD


COPY = dict(src=A, dst=A, tokens=A, n=4, status=A, stream=None)


@pytest.mark.parametrize("kw", [dict(src=None), dict(dst=None), dict(dst=A + 2), dict(tokens=A + 1), dict(status=None), dict(n=1 << 31)])
def test_bad_copy_arguments(kw):
    assert B.lib().skv_cache_copy(C.byref(cache()), *dict(COPY, **kw).values()) == BAD
    assert B.lib().skv_cache_copy(C.byref(cache(dtype=3)), *COPY.values()) == BAD
    big = cache(page_tokens=1 << 20, n_heads=128, token_stride=16384, page_stride=1 << 34)        # 2^31 units of 16 bytes
    assert B.lib().skv_cache_copy(C.byref(big), *COPY.values()) == BAD


def ws(requests, pages):
    v = C.c_uint64()
    assert B.lib().skv_page_workspace_bytes(requests, pages, C.byref(v)) == 0
    return v.value


def test_workspace_bytes():
    assert ws(0, 1) >= 12 and ws(1 << 20, 1) >= 4 << 20 and ws(1, 1 << 20) >= (8 << 20) + (1 << 17)
    assert B.lib().skv_page_workspace_bytes(1, 0, C.byref(C.c_uint64())) == BAD
    assert B.lib().skv_page_workspace_bytes(1, 1, None) == BAD


FORK = dict(page_tokens=16, pool_pages=8, n_requests=2, parents=A, ctx_len=A, block_table=A, table_stride=4, max_pages=4, n_pages_in=A, trim=0,
            table_out=A + 256, table_out_stride=4, n_pages_out=A + 64, ctx_out=A + 64, free_pages=A, free_capacity=8, free_in=A, free_out=A + 64, copy_src=A,
            copy_dst=A, copy_tokens=A, status=A, workspace=A, ws_bytes=4096, stream=None)


@pytest.mark.parametrize("kw", [dict(page_tokens=0), dict(page_tokens=(1 << 20) + 1), dict(pool_pages=0), dict(pool_pages=1 << 31), dict(n_requests=1 << 31),
                                dict(ctx_len=None), dict(block_table=None), dict(table_stride=3), dict(table_out_stride=3), dict(max_pages=1 << 31),
                                dict(n_pages_in=None), dict(trim=2), dict(table_out=None), dict(table_out=A), dict(n_pages_out=A), dict(ctx_out=A),
                                dict(free_pages=None), dict(free_capacity=1 << 31), dict(free_in=None), dict(free_out=A), dict(copy_src=None),
                                dict(copy_dst=None), dict(copy_tokens=None), dict(status=None), dict(parents=A + 2), dict(workspace=None),
                                dict(workspace=A + 8), dict(ws_bytes=64)])
def test_bad_fork_arguments(kw):
    assert B.lib().skv_page_fork(*dict(FORK, **kw).values()) == BAD


COMPACT = dict(pool_pages=8, n_requests=2, block_table=A, table_stride=4, max_pages=4, n_pages=A, table_out=A + 256, table_out_stride=4, free_pages=A,
               free_capacity=8, free_in=A, free_out=A + 64, copy_src=A, copy_dst=A, copy_capacity=8, status=A, workspace=A, ws_bytes=4096, stream=None)


@pytest.mark.parametrize("kw", [dict(pool_pages=0), dict(pool_pages=1 << 31), dict(block_table=None), dict(table_stride=3), dict(table_out_stride=3),
                                dict(n_pages=None), dict(table_out=None), dict(table_out=A), dict(free_pages=None), dict(free_in=None), dict(free_out=A),
                                dict(copy_src=None), dict(copy_dst=None), dict(copy_capacity=1 << 31), dict(status=A + 2), dict(workspace=None),
                                dict(ws_bytes=64)])
def test_bad_compact_arguments(kw):
    assert B.lib().skv_page_compact(*dict(COMPACT, **kw).values()) == BAD


def test_turns():
    """Frequencies as words of 2^-64 of a turn."""
    f = [1.0, -0.75, 1e-9, 100.25, 0.0]
    for x, t in zip(f, _turns(f)):
        back = (t / 2.0 ** 64) % 1.0
        want = (x / (2 * math.pi)) % 1.0
        assert min(abs(back - want), 1 - abs(back - want)) <= 2.0 ** -48
    assert _turns([2 * math.pi * 0.25])[0] == pytest.approx(2 ** 62, abs=2 ** 11)


def test_python_refuses():
    with pytest.raises(ValueError):
        Rotary(128, [1.0] * 64, device="cpu")
    with pytest.raises(ValueError):
        Verifier(2, 8, device="cpu")
