"""The example layer end to end: chunked prompts through the cache, then a captured decode step."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# Bound of a sequence's relative output error, by the cache's element rounding: the output is a weighted mean
# of values that are each off by at most u (relative to their block's largest value for the 4-bit types), and the
# weights move by exp(score error).  bf16: u = 2^-8 of weights and values.  E4M3: 2^-4 an element, twice
# (keys and values).  E2M1: a quarter of an element near the top of its grid, an eighth on average, twice.
BOUND = {"bf16": 0.02, "mxfp8": 0.125, "nvfp4": 0.35, "mxfp4": 0.5}


@pytest.mark.parametrize("fmt", sorted(BOUND))
def test_layer(fmt):
    spec = importlib.util.spec_from_file_location("attention_layer", os.path.join(ROOT, "examples", "attention_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    worst, nbytes, y = m.run(fmt, prompts=(300, 17, 2, 64), steps=5)
    assert y.shape == (4, 1024) and bool(y.isfinite().all())
    assert worst < BOUND[fmt], (fmt, worst)
