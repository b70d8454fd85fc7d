"""Corners of the paged-cache operators' arithmetic: many small weights beside a large one,
scales at the ends of binary32, wide and narrow row tiles in one long list of work,
the kernel that a call takes by default, and pools of other types."""
import math
import pytest
import torch

from tests import _pagedtest as P
from tests.test_gpu_paged import attend_case
from lossless_kv_cache_scalar_gb300 import PagedKV

pytestmark = pytest.mark.gpu


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
