"""Norms of queries and keys without a rotation, and without positions."""
import pytest
import torch

from tests.test_gpu_rotate import check, made
from lossless_kv_cache_scalar_gb300 import Rotary

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("n,dim", [(1, 16), (77, 96), (2600, 128)])
def test_norms_alone(n, dim, dtype):
    s = made(n + dim, n, 4, 2, dim, 16, dtype)
    w = 1 + 0.3 * torch.randn(2, dim, generator=s["gen"])
    out = s["cache"].rotate_append(Rotary(dim, [], w[0], w[1], eps=1e-5), s["q"], s["kn"], s["vn"], None, s["slots"])
    check(s, torch.zeros(n, 0, dtype=torch.float64), w[0], w[1], 1e-5, False, 1.0, out)
    with pytest.raises(ValueError, match="positions"):
        s["cache"].rotate_append(Rotary(dim, [1.0] * 8), s["q"], s["kn"], s["vn"], None, s["slots"])
