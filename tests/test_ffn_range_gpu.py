"""NVFP4 products where sums without the tensor scale would pass fp32's range, and others without a tensor scale of
ordinary size: results are off by their own roundings alone."""
import numpy as np
import pytest
import torch

import ffn_ref
from test_ffn_gpu import DT, HALF, activations, check, fq, handle, sum_bound, values, weight  # noqa: F401

pytestmark = pytest.mark.gpu


def powers(x, p):
    """x times 2^p, exactly: rows of any kind."""
    if isinstance(x, torch.Tensor):
        return torch.ldexp(x.double(), torch.tensor(float(p), dtype=torch.float64, device=x.device)).to(x.dtype)
    return type(x)(x.codes, (x.scales.int() + p).to(torch.uint8))


# (kernels: few rows in both forms, small tiles in parts, large tiles, the ring with parts and without)
SHAPES = [(3, 96, 320), (16, 64, 8192), (40, 96, 320), (70, 96, 2112), (600, 8200, 4160), (1030, 8200, 192)]


@pytest.mark.parametrize("kind", ["bf16", "f32", "mxfp8"])
@pytest.mark.parametrize("rows,n,k", SHAPES)
@pytest.mark.parametrize("up,g", [(118, 1.37 * 2.0 ** -30), (118, -2.0 ** -100), (-90, 1.9 * 2.0 ** 100), (80, 2.0 ** -126),
                                  (100, 2.0 ** -140), (-100, 1.5 * 2.0 ** 126)])
def test_linear(fq, kind, rows, n, k, up, g):
    print(kind, rows, n, k, up, g, flush=True)
    rng = np.random.default_rng(rows)
    codes, scales, _ = weight(rng, "nvfp4", n, k)
    planes = codes, scales, g
    x, xv, pieces = activations(rng, fq, kind, rows, k)
    y = fq.fp4_linear(powers(x, up), handle(fq, "nvfp4", planes), out_dtype=torch.float32)
    torch.cuda.synchronize()
    w = values("nvfp4", (codes, scales, 1.0)) * float(np.float32(g))
    xv = np.ldexp(xv, up)
    want, S = xv @ w.T, np.abs(xv) @ np.abs(w).T
    assert np.abs(want).max() < 2.0 ** 127 and np.isfinite(want).all()
    check(y, want, sum_bound(S, k, pieces) + HALF[torch.float32] * np.abs(want))


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("rows,n,k", [(3, 96, 320), (90, 2112, 96), (600, 4160, 8256), (1030, 192, 8256)])
def test_backward(fq, kind, rows, n, k):
    rng = np.random.default_rng(rows)
    codes, scales, _ = weight(rng, "nvfp4", n, k)
    g = 1.61 * 2.0 ** -40
    dy, dv, pieces = activations(rng, fq, kind, rows, n)
    dx = fq.fp4_linear_backward(powers(dy, 118), handle(fq, "nvfp4", (codes, scales, g)))
    torch.cuda.synchronize()
    w = values("nvfp4", (codes, scales, 1.0)) * float(np.float32(g))
    dv = np.ldexp(dv, 118)
    want, S = dv @ w, np.abs(dv) @ np.abs(w)
    check(dx, want, sum_bound(S, n, pieces) + HALF[dx.dtype] * np.abs(want))


@pytest.mark.parametrize("rows,f,k", [(3, 48, 320), (40, 48, 320), (70, 48, 2112), (600, 4100, 4160), (1030, 4100, 192)])
def test_gated_products(fq, rows, f, k):
    rng = np.random.default_rng(rows)
    codes, scales, _ = weight(rng, "nvfp4", 2 * f, k)
    g = 1.2 * 2.0 ** -50
    x, xv, pieces = activations(rng, fq, "bf16", rows, k)
    _, p = fq.fp4_gated(powers(x, 118), handle(fq, "nvfp4", (codes, scales, g)), return_products=True)
    torch.cuda.synchronize()
    w = values("nvfp4", (codes, scales, 1.0)) * float(np.float32(g))
    xv = np.ldexp(xv, 118)
    want, S = xv @ w.T, np.abs(xv) @ np.abs(w).T
    check(p, want, sum_bound(S, k, 1) + HALF[torch.float32] * np.abs(want))


@pytest.mark.parametrize("rows", [3, 70, 1030])
@pytest.mark.parametrize("g", [0.0, -0.0, float("inf"), float("nan")])
def test_tensor_scales_that_are_no_numbers(fq, rows, g):
    """Zero gives zeros; infinity and NaN what the product with the sums gives."""
    rng = np.random.default_rng(4)
    n, k = 8200 if rows > 100 else 64, 192
    codes, scales, _ = weight(rng, "nvfp4", n, k)
    x, _, _ = activations(rng, fq, "bf16", rows, k)
    one = fq.fp4_linear(x, handle(fq, "nvfp4", (codes, scales, 1.0)), out_dtype=torch.float32)
    got = fq.fp4_linear(x, handle(fq, "nvfp4", (codes, scales, g)), out_dtype=torch.float32)
    assert torch.equal(torch.nan_to_num(got, nan=7.0), torch.nan_to_num(one * g, nan=7.0))
