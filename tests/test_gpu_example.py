"""The served attention block of examples/serve_attention.py runs plan, append and both
attentions between the FP8 projections as a program would."""

import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("kw", [dict(), dict(prompts=(1, 200), chunk=64, hidden=512, q_heads=4, kv_heads=4, head_dim=128, answers=3)])
def test_served_requests_agree_with_whole_prompts(kw):
    """The two runs differ by the e4m3 rounding of keys and values (2^-4 a value at most, about 2.5% in
    the mean square) and of the attention's output before the second projection (the same again):
    the root of the sum of both squares with both runs rounded is under 6%; twice that is allowed."""
    spec = importlib.util.spec_from_file_location("serve_attention", os.path.join(ROOT, "examples", "serve_attention.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    off, steps = m.serve(**kw)
    assert off < 0.12
    assert steps >= 6
