"""The hybrid example end to end: prompt, single tokens, a draft tree's verify and commit, with
the recurrent layers and the attention layers' paged 8-bit cache together."""
import os
import runpy

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_hybrid_example():
    from hybrid_linear_attention_conv_gb300 import build
    build.build()
    run = runpy.run_path(os.path.join(ROOT, "examples", "hybrid_step.py"))["run"]
    error, same = run(1)
    # A key or value within its block's scale is rounded to e4m3: half a step of 2^-3 at most, 2^-4
    # relative, uniform within it: about 2^-4 / sqrt(3) / 1.4 = 0.026 in the 2-norm.  Values' errors
    # reach the output as they are; keys' through logits of order one, as much again.
    assert error < 2 * 2.0 ** -4
    assert same
