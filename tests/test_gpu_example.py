"""The example of a drafted step runs, and a token's attention as a node of the tree
equals its attention as a single token once its path is accepted."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu


def test_draft_step():
    at = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "draft_step.py")
    spec = importlib.util.spec_from_file_location("draft_step", at)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    out, again, path = m.main()
    a, b = again[0].float(), out[path[-1]].float()
    # weights and outputs rounded to bf16 on both sides: 2^-8 (|o| + A) each, A < 60 for these values
    assert ((a - b).abs() <= 2.0 ** -7 * (b.abs() + 60)).all() and float((a - b).norm() / b.norm()) < 2.0 ** -6
