"""The wrappers around a serving step refuse tensors of another device than their object's, and calls
made while another device is current. Checked on the host with stand-ins for tensors."""
import pytest
import torch

from lossless_kv_cache_scalar_gb300 import PageTable, Rotary, Verifier
from tests.test_paged_devices import DEV, Lib, Stand, Stream, args, host, kv        # noqa: F401

I32, I64, F32, BF16 = torch.int32, torch.int64, torch.float32, torch.bfloat16

ROTATE = dict(q=((3, 4, 64), BF16), k=((3, 2, 64), BF16), v=((3, 2, 64), BF16), positions=((3,), I32), slots=((3,), I64), q_out=((3, 4, 64), BF16))
MOVE = dict(cu_new=((3,), I32), rows=((5,), I32), slots=((5,), I64), kept=((5,), I64))
COPY = dict(src=((5,), I32), dst=((5,), I32), tokens=((5,), I32))
VERIFY = dict(probs=((5, 9), F32), tokens=((5,), I32), cu_new=((3,), I32), uniform=((5,), F32), accepted=((2,), I32), rows=((5,), I32),
              next_tokens=((2,), I32), parents=((5,), I32), draft_probs=((5, 9), F32), slots=((5,), I64), kept=((5,), I64), ctx_len=((2,), I32),
              ctx_out=((2,), I32))
FORK = dict(parents=((2,), I32), ctx_len=((2,), I32), n_pages=((2,), I32), free_pages=((8,), I32), free_state=((2,), I32), table_out=((2, 4), I32),
            n_pages_out=((2,), I32), ctx_out=((2,), I32), free_state_out=((2,), I32), copy_src=((2,), I32), copy_dst=((2,), I32), copy_tokens=((2,), I32))
COMPACT = dict(n_pages=((2,), I32), free_pages=((8,), I32), free_state=((2,), I32), table_out=((2, 4), I32), free_state_out=((2,), I32),
               copy_src=((8,), I32), copy_dst=((8,), I32))


class FakeRotary:
    def __init__(self, device=DEV, head_dim=64):
        self._device, self.head_dim, self.n_axes, self._ref = device, head_dim, 1, None


def fake_verifier():
    v = Verifier.__new__(Verifier)
    v.n_requests, v.vocab, v.status, v._status, v._device = 2, 9, None, 1 << 20, DEV
    return v


def fake_table():
    t = PageTable(Stand(2, 4), 16, 8)
    t.workspace, t._workspace, t._workspace_bytes = True, 1 << 21, 1 << 20
    return t


def call_of(what):
    if what == "rotate":
        c = kv()
        return lambda **a: c.rotate_append_into(FakeRotary(), **a)
    if what in ("move", "copy"):
        return getattr(kv(), what + "_into")
    if what == "verify":
        return fake_verifier().verify_into
    t = fake_table()

    def call(**a):
        for name in a:                                     # outputs at an address of their own
            if name.endswith("_out"):
                a[name].data_ptr = lambda: 1 << 22
        return getattr(t, what + "_into")(**a)
    return call


CALLS = dict(rotate=ROTATE, move=MOVE, copy=COPY, verify=VERIFY, fork=FORK, compact=COMPACT)


@pytest.mark.parametrize("what,away", [(w, n) for w, spec in CALLS.items() for n in (None, *spec)])
def test_another_device(host, what, away):                 # noqa: F811
    call = call_of(what)
    before = Lib.calls
    if away is None:
        call(**args(CALLS[what]))
        assert Lib.calls == before + 1
    else:
        with pytest.raises(ValueError):
            call(**args(CALLS[what], away))
        assert Lib.calls == before


@pytest.mark.parametrize("what", list(CALLS))
def test_another_current_device(host, what):               # noqa: F811
    call = call_of(what)
    before = Lib.calls
    host["current"] = 0
    with pytest.raises(ValueError, match="current device"):
        call(**args(CALLS[what]))
    host["current"] = DEV
    with pytest.raises(ValueError, match="stream of it"):
        call(**args(CALLS[what]), stream=Stream(0))
    assert Lib.calls == before
    call(**args(CALLS[what]), stream=Stream(DEV))
    assert Lib.calls == before + 1


def test_a_rotary_of_another_device_or_size(host):         # noqa: F811
    c = kv()
    for r in (FakeRotary(DEV + 1), FakeRotary(head_dim=96)):
        with pytest.raises(ValueError, match="Rotary"):
            c.rotate_append_into(r, **args(ROTATE))


def test_host_tensors():
    with pytest.raises(ValueError):
        Rotary(64, [1.0] * 32, device="cpu")
