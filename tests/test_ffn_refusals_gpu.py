"""What is no tensor is refused as other wrong buffers are."""
import numpy as np
import pytest
import torch

from test_ffn_gpu import fq, handle, weight  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("wrong", ["out", 5, (1, 2), np.zeros((4, 32), dtype=np.float32), [None]], ids=str)
def test_buffers_that_are_no_tensors(fq, wrong):
    w = handle(fq, "mxfp4", weight(np.random.default_rng(0), "mxfp4", 32, 32))
    x, gain = torch.zeros(4, 32, device="cuda"), torch.ones(32, device="cuda")
    for call in (lambda: fq.fp4_linear(x, w, out=wrong), lambda: fq.fp4_linear_backward(x, w, out=wrong),
                 lambda: fq.fp4_gated(x, w, out=wrong), lambda: fq.rms_norm(x, gain, out=wrong),
                 lambda: fq.rms_norm(x, gain, residual=x, summed=wrong),
                 lambda: fq.rms_norm(x, gain, quantize="mxfp8", out=wrong),
                 lambda: fq.fp4_linear(x, w, bias=wrong)):
        with pytest.raises(ValueError):
            call()
