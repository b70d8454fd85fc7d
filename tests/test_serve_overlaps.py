"""A fork whose new lengths would be written over the arrays that it reads is refused on the host (addresses that are
never read)."""
import pytest

from lossless_kv_cache_scalar_gb300 import _binding as B
from tests.test_paged_refusals import A, BAD
from tests.test_serve_refusals import FORK

APART = dict(FORK, parents=A + 512, ctx_len=A + 1024, n_pages_in=A + 1536, n_pages_out=A + 2048, ctx_out=A + 2560)


@pytest.mark.parametrize("out", ["n_pages_out", "ctx_out"])
@pytest.mark.parametrize("given", ["parents", "ctx_len", "n_pages_in"])
def test_lengths_over_what_is_read(out, given):
    assert B.lib().skv_page_fork(*dict(APART, **{out: APART[given]}).values()) == BAD
