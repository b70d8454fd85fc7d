"""The paged-cache wrappers refuse tensors of another device than the pools', and calls made
while another device is current (a kernel is launched on the current device and would
reach for the other one's memory). Checked on the host with stand-ins for tensors: one GPU is
enough for everything else."""
import pytest
import torch

from lossless_kv_cache_scalar_gb300 import PagedKV, PageTable
from lossless_kv_cache_scalar_gb300 import _binding as B

DEV = 3


class Stand:
    """What the wrappers ask of a tensor; its address is never read."""

    def __init__(self, *shape, dtype=torch.int32, device=DEV):
        self.t = torch.empty(shape, dtype=dtype, device="meta")
        self.shape, self.dtype, self.device = self.t.shape, dtype, torch.device("cuda", device)
        self.is_cuda = True

    def get_device(self):
        return self.device.index

    def data_ptr(self):
        return 1 << 20

    def __getattr__(self, name):
        return getattr(self.t, name)


class Lib:
    """The C entries, counted."""
    calls = 0

    def __getattr__(self, name):
        def call(*a):
            Lib.calls += 1
            return 0
        return call


@pytest.fixture
def host(monkeypatch):
    import lossless_kv_cache_scalar_gb300.paged as paged
    state = {"current": DEV}
    monkeypatch.setattr(B, "lib", lambda: Lib())
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: state["current"], raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 0, raising=False)
    monkeypatch.setattr(paged._Status, "_new_status",
                        lambda self, device: (setattr(self, "status", None), setattr(self, "_status", 1 << 20),
                                              setattr(self, "_device", device.index)))
    monkeypatch.setattr(paged._Status, "_settle", lambda self: None)
    Lib.calls = 0
    return state


def kv(**kw):
    pool = lambda: Stand(4, 16, 2, 64, dtype=torch.bfloat16)                 # noqa: E731
    c = PagedKV(pool(), pool(), Stand(2, 4), **kw)
    c.workspace, c._workspace, c._workspace_bytes = True, 1 << 20, 1 << 20
    return c


ATTEND = dict(q=((3, 4, 64), torch.bfloat16), ctx_len=((2,), torch.int32), cu_new=((3,), torch.int32), out=((3, 4, 64), torch.bfloat16),
              mask=((3, 1), torch.int64), lse=((3, 4), torch.float32))
APPEND = dict(k=((3, 2, 64), torch.bfloat16), v=((3, 2, 64), torch.bfloat16), slots=((3,), torch.int64), rows=((3,), torch.int32))
MAP = dict(ctx_len=((2,), torch.int32), new_len=((2,), torch.int32), n_pages=((2,), torch.int32), free_pages=((8,), torch.int32),
           free_state=((2,), torch.int32), cu_new=((3,), torch.int32), slots=((5,), torch.int64), n_pages_out=((2,), torch.int32),
           free_state_out=((2,), torch.int32))


def args(spec, away=None):
    return {n: Stand(*s, dtype=d, device=DEV + (n == away)) for n, (s, d) in spec.items()}


@pytest.mark.parametrize("away", [None, *ATTEND])
def test_attend(host, away):
    c = kv()
    before = Lib.calls
    if away is None:
        c.attend_into(**args(ATTEND))
        assert Lib.calls == before + 1
    else:
        with pytest.raises(ValueError):
            c.attend_into(**args(ATTEND, away))
        assert Lib.calls == before


@pytest.mark.parametrize("away", [None, *APPEND])
def test_append(host, away):
    c = kv()
    before = Lib.calls
    if away is None:
        c.append_into(**args(APPEND))
        assert Lib.calls == before + 1
    else:
        with pytest.raises(ValueError):
            c.append_into(**args(APPEND, away))
        assert Lib.calls == before


@pytest.mark.parametrize("away", [None, *MAP])
def test_map(host, away):
    t = PageTable(Stand(2, 4), 16, 8)
    if away is None:
        t.map_into(**args(MAP))
        assert Lib.calls == 1
    else:
        with pytest.raises(ValueError):
            t.map_into(**args(MAP, away))
        assert Lib.calls == 0


@pytest.mark.parametrize("what", ["block_table", "k_scale", "v_pages"])
def test_constructor(host, what):
    a = dict(k_pages=Stand(4, 16, 2, 64, dtype=torch.uint8), v_pages=Stand(4, 16, 2, 64, dtype=torch.uint8), block_table=Stand(2, 4),
             k_scale=Stand(2, dtype=torch.float32), v_scale=Stand(2, dtype=torch.float32))
    PagedKV(**a)
    a[what] = Stand(*a[what].shape, dtype=a[what].dtype, device=DEV + 1)
    with pytest.raises(ValueError):
        PagedKV(**a)


class Stream:
    cuda_stream = 7

    def __init__(self, device):
        self.device_index = device


def test_another_current_device(host):
    c, t = kv(), PageTable(Stand(2, 4), 16, 8)
    before = Lib.calls
    host["current"] = 0
    for call in (lambda: c.attend_into(**args(ATTEND)), lambda: c.append_into(**args(APPEND)), lambda: t.map_into(**args(MAP)),
                 lambda: c.attend_into(**args(ATTEND), stream=Stream(DEV))):
        with pytest.raises(ValueError, match="current device"):
            call()
    host["current"] = DEV
    with pytest.raises(ValueError, match="stream of it"):
        c.attend_into(**args(ATTEND), stream=Stream(0))
    assert Lib.calls == before
    c.attend_into(**args(ATTEND), stream=Stream(DEV))
    assert Lib.calls == before + 1
