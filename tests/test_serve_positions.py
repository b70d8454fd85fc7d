"""A Rotary that rotates nothing (norms alone) needs no positions; any other refuses to go without. Checked on the host
with stand-ins for tensors."""
import pytest

from tests.test_paged_devices import DEV, Lib, args, host, kv        # noqa: F401
from tests.test_serve_devices import ROTATE, FakeRotary


@pytest.mark.parametrize("rot_dim", [0, 64])
def test_no_positions(host, rot_dim):                      # noqa: F811
    r = FakeRotary()
    r.rot_dim = rot_dim
    given = dict(args(ROTATE), positions=None)
    before = Lib.calls
    if rot_dim:
        with pytest.raises(ValueError, match="positions"):
            kv().rotate_append_into(r, **given)
        assert Lib.calls == before + 1                     # the pools' own check
    else:
        kv().rotate_append_into(r, **given)
        assert Lib.calls == before + 2
