"""The tree-attention kernel whose waits run out: it says so and leaves the GPU usable. The
same sources are built with a limit of 0 clocks, so that every wait that is not over at
its first look gives up; accesses stay in bounds, copies that were started are waited
for, and no other kernel runs meanwhile."""
import ctypes as C
import os
import subprocess

import pytest
import torch

from tests.test_gpu_paged import attend_case
from lossless_kv_cache_scalar_gb300 import PagedKV, SKVError
from lossless_kv_cache_scalar_gb300 import _binding as B
from lossless_kv_cache_scalar_gb300 import build as L

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def hasty(tmp_path_factory):
    """libskv's attention with waits that give up at once."""
    at = tmp_path_factory.mktemp("hasty")
    objects = []
    running = []
    for name in ("skv_paged", "skv_attend", "skv_attend_tc"):
        objects.append(str(at / (name + ".o")))
        running.append(subprocess.Popen([L.nvcc(), *L.ARCH, *L.FLAGS, "-DSKV_WAIT_CLOCKS=0ll", "-c", os.path.join(L.CSRC, name + ".cu"),
                                         "-o", objects[-1]]))
    assert [p.wait() for p in running] == [0, 0, 0]
    so = str(at / "libhasty.so")
    subprocess.run([L.nvcc(), *L.ARCH, "-shared", "-o", so, *objects, "-lcudart_static", "-ldl", "-lrt", "-lpthread"], check=True)
    lib = C.CDLL(so)
    for name in ("skv_paged_check", "skv_tree_attention_workspace_bytes", "skv_tree_attention"):
        getattr(lib, name).restype, getattr(lib, name).argtypes = B.SIGNATURES[name]
    return lib


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("page,dim", [(16, 128), (256, 64), (7, 128)])
def test_a_wait_that_runs_out_is_reported(hasty, monkeypatch, page, dim, dtype):
    s = attend_case(101, [900, 40, 300], [40, 0, 70], page, 2, 4, dim, dtype)
    cache = PagedKV(s["k"], s["v"], s["table"], k_scale=s["ks"], v_scale=s["vs"], q_heads=8)
    pools = s["k"].clone(), s["v"].clone()
    rows = s["q"].shape[0]
    guard = torch.full((rows + 64, 8, dim), 7.0, dtype=torch.bfloat16, device="cuda")
    out = guard[32:32 + rows]

    def call():
        cache.attend_into(s["q"], s["ctx"], s["cu"], out, mask=s["mask"], max_nodes=70)
        cache.check_status("skv_tree_attention")

    call()
    want = out.clone()
    with monkeypatch.context() as m:
        m.setattr(B, "lib", lambda: hasty)
        for _ in range(3):
            with pytest.raises(SKVError) as e:
                call()
            assert e.value.name == "TIMEOUT"
    # only rows of requests were written, and the next call is as good as the first
    assert (guard[:32] == 7).all() and (guard[32 + 110:] == 7).all()
    assert torch.equal(s["k"], pools[0]) and torch.equal(s["v"], pools[1])
    assert not cache.workspace[:B.SKV_ATTENTION_ZERO_BYTES].any()
    call()
    assert torch.equal(out, want)
