"""Results repeat bit for bit in every form of the few-row kernel: two, four and six tiles of the weight a workgroup,
one to four of rows, all types."""
import numpy as np
import pytest
import torch

from test_ffn_gpu import FORMATS, activations, fq, handle, weight  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("kind", ["bf16", "mxfp8", "f32"])
@pytest.mark.parametrize("n,k", [(1024, 4096), (16384, 416), (20000, 416)])
def test_few_rows_repeat(fq, fmt, kind, n, k):
    rng = np.random.default_rng(n)
    w = handle(fq, fmt, weight(rng, fmt, n, k))
    for rows in (1, 9, 16) if kind == "f32" else (1, 9, 16, 17, 32, 33, 48, 49, 64):
        x, _, _ = activations(rng, fq, kind, rows, k)
        first = fq.fp4_linear(x, w), fq.fp4_gated(x, w)
        for _ in range(20):
            assert torch.equal(fq.fp4_linear(x, w), first[0]) and torch.equal(fq.fp4_gated(x, w), first[1])
