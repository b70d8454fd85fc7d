"""The paged-cache operators refuse bad arguments on the host, before any CUDA
call (checked here through the C ABI with addresses that are never read), and
their Python wrappers refuse host tensors."""
import ctypes as C

import pytest
import torch

from lossless_kv_cache_scalar_gb300 import PagedKV, PageTable
from lossless_kv_cache_scalar_gb300 import _binding as B

A = 1 << 20                                            # an aligned address
BAD = 1                                                # SKV_ERR_INVALID_ARG


def cache(**kw):
    f = dict(version=1, dtype=0, n_heads=8, head_dim=128, page_tokens=256, n_pages=4, k_pages=A, v_pages=A, page_stride=262144,
             token_stride=1024, head_stride=128, k_scale=None, v_scale=None, block_table=A, table_stride=4, n_requests=2,
             max_pages=4)
    f.update(kw)
    return B.skv_paged(**f)


def test_a_good_cache():
    assert B.lib().skv_paged_check(C.byref(cache())) == 0
    assert B.lib().skv_paged_check(C.byref(cache(dtype=1, k_scale=A, v_scale=A))) == 0
    assert B.lib().skv_paged_check(C.byref(cache(page_tokens=1, n_heads=1, head_dim=16, token_stride=0, head_stride=0))) == 0
    assert B.lib().skv_paged_check(None) == BAD


@pytest.mark.parametrize("kw", [
    dict(version=0), dict(dtype=2), dict(n_heads=0), dict(n_heads=65536), dict(head_dim=0), dict(head_dim=24), dict(head_dim=272),
    dict(page_tokens=0), dict(page_tokens=(1 << 20) + 1), dict(n_pages=0), dict(n_pages=1 << 31), dict(k_pages=None),
    dict(v_pages=A + 8), dict(page_stride=262145), dict(token_stride=1028), dict(head_stride=0), dict(page_stride=0),
    dict(token_stride=0), dict(page_stride=(1 << 40) + 8), dict(k_scale=A, v_scale=A), dict(dtype=1, k_scale=A),
    dict(dtype=1, token_stride=1032), dict(dtype=1, k_scale=A + 2, v_scale=A)])
def test_bad_caches(kw):
    c = cache(**kw)
    n = C.c_uint64()
    assert B.lib().skv_paged_check(C.byref(c)) == BAD
    assert B.lib().skv_tree_attention_workspace_bytes(C.byref(c), 8, C.byref(n)) == BAD
    assert B.lib().skv_cache_append(C.byref(c), A, A, 1024, 128, 4, None, A, 4, A, None) == BAD


MAP = dict(page_tokens=16, pool_pages=8, n_requests=2, ctx_len=A, new_len=A, block_table=A, table_stride=4, max_pages=4,
           n_pages_in=A, n_pages_out=A + 64, free_pages=A, free_capacity=8, free_in=A, free_out=A + 64, cu_new=A, slots=A,
           slot_capacity=4, status=A, stream=None)


@pytest.mark.parametrize("kw", [
    dict(page_tokens=0), dict(page_tokens=(1 << 20) + 1), dict(pool_pages=0), dict(pool_pages=1 << 31), dict(max_pages=5),
    dict(ctx_len=None), dict(new_len=None), dict(block_table=None), dict(n_pages_in=None), dict(n_pages_out=None),
    dict(free_pages=None), dict(free_in=None), dict(free_out=None), dict(cu_new=None), dict(slots=None), dict(status=None),
    dict(n_pages_out=A), dict(free_out=A), dict(slots=A + 4), dict(ctx_len=A + 1), dict(free_capacity=1 << 31),
    dict(n_requests=1 << 31), dict(slot_capacity=(1 << 40) + 1)])
def test_bad_map_arguments(kw):
    assert B.lib().skv_page_map(*dict(MAP, **kw).values()) == BAD


APPEND = dict(k=A, v=A, row_stride=1024, row_head_stride=128, n_src=4, rows=None, slots=A, n=4, status=A, stream=None)


@pytest.mark.parametrize("kw", [dict(k=None), dict(v=A + 8), dict(row_stride=1020), dict(row_head_stride=4), dict(rows=A + 2),
                                dict(slots=None), dict(slots=A + 4), dict(status=None), dict(status=A + 2),
                                dict(row_stride=1 << 41)])
def test_bad_append_arguments(kw):
    assert B.lib().skv_cache_append(C.byref(cache()), *dict(APPEND, **kw).values()) == BAD


def attend_args(**kw):
    n = C.c_uint64()
    assert B.lib().skv_tree_attention_workspace_bytes(C.byref(cache()), 32, C.byref(n)) == 0
    f = dict(q=A, q_row_stride=4096, q_head_stride=128, n_q_heads=32, n_rows=4, ctx_len=A, cu_new=A, mask=A, mask_words=1,
             max_nodes=4, scale=0.1, out=A, lse=None, status=A, workspace=A, ws_bytes=n.value, stream=None)
    f.update(kw)
    return f


@pytest.mark.parametrize("kw", [
    dict(q=None), dict(q=A + 8), dict(q_row_stride=4097), dict(q_head_stride=4), dict(n_q_heads=0), dict(n_q_heads=33),
    dict(n_q_heads=65536), dict(n_rows=1 << 31),
    dict(n_rows=1 << 29), dict(ctx_len=None), dict(cu_new=None), dict(cu_new=A + 2), dict(mask=None), dict(mask_words=0), dict(mask=A + 4),
    dict(scale=float("nan")), dict(out=None), dict(out=A + 8), dict(lse=A + 2), dict(status=None), dict(workspace=None),
    dict(workspace=A + 128), dict(ws_bytes=0)])
def test_bad_attention_arguments(kw):
    assert B.lib().skv_tree_attention(C.byref(cache()), *attend_args(**kw).values()) == BAD


@pytest.mark.parametrize("kw", [dict(block_table=None), dict(block_table=A + 2), dict(table_stride=3), dict(max_pages=1 << 31),
                                dict(n_requests=0x7FFFFFFF)])
def test_bad_tables(kw):
    assert B.lib().skv_tree_attention(C.byref(cache(**kw)), *attend_args().values()) == BAD


def test_python_refuses_host_tensors():
    pool = torch.zeros(2, 16, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        PagedKV(pool, pool)
    with pytest.raises(ValueError):
        PageTable(torch.zeros(2, 4, dtype=torch.int32), 16, 8)
