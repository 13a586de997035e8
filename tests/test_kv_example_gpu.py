"""The serving example: prompts by chunks, captured decode steps, a cache read
back.  Rounding to E2M1 with a block scale leaves an element off by at most a
sixth of its block's largest value (half the widest step, 4 to 6) and a normal
block's relative root mean square below that: 0.17.  MXFP4's power-of-two scale
may be up to twice as wide, 4 to 6 becoming 4 to beyond 6 (clipped): 0.25.
Attention averages values, and its weights move with the keys' error, which for
these random keys reaches about the same size again: twice the bound."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt,bound", [("nvfp4", 0.17), ("mxfp4", 0.25)])
@pytest.mark.parametrize("head_dim,page", [(128, 16), (64, 24)])
def test_serving(fmt, bound, head_dim, page):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import kv_cache_serving
    k, v, out = kv_cache_serving.serve([70, 3, 131], 20, chunk=50, q_heads=8, kv_heads=2, head_dim=head_dim,
                                       page_size=page, format=fmt)
    assert 0.0 < k < bound and 0.0 < v < bound
    assert 0.0 < out < 2 * bound
