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


# fp32 rows enter as three bf16 pieces, cut off.  From 2^-110 on the pieces sum to the row's elements; below, what lies
# under bf16's least number, 2^-133, is lost: less than that of each element.
@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("rows,n,k", [(4, 96, 320), (16, 64, 8192), (80, 96, 2112), (1030, 4200, 192)])
@pytest.mark.parametrize("low", [-109, -118, -126, -140])
def test_smallest_fp32_rows(fq, fmt, rows, n, k, low):
    rng = np.random.default_rng(rows)
    codes, scales, _ = weight(rng, fmt, n, k)
    g = 1.3 * 2.0 ** 90 if fmt == "nvfp4" else None
    if fmt == "mxfp4":
        scales = (scales + 90).astype(np.uint8)
    planes = codes, scales, g
    # magnitudes of all bits, from 2^low to 2^(low + 1)
    x = np.ldexp(rng.choice([-1.0, 1.0], (rows, k)) * rng.uniform(1, 2, (rows, k)), low).astype(np.float32)
    dy = np.ldexp(rng.choice([-1.0, 1.0], (rows, n)) * rng.uniform(1, 2, (rows, n)), low).astype(np.float32)
    h = handle(fq, fmt, planes)
    y, dx = fq.fp4_linear(torch.from_numpy(x).cuda(), h), fq.fp4_linear_backward(torch.from_numpy(dy).cuda(), h)
    torch.cuda.synchronize()
    w = values(fmt, (codes, scales, 1.0 if fmt == "nvfp4" else None)) * (1.0 if g is None else float(np.float32(g)))
    lost = 0.0 if low >= -110 else 2.0 ** -133
    for got, v, a, terms in ((y, x.astype(np.float64), w.T, k), (dx, dy.astype(np.float64), w, n)):
        want, S = v @ a, np.abs(v) @ np.abs(a)
        check(got, want, sum_bound(S, terms, 3) + lost * np.abs(a).sum(0) + HALF[torch.float32] * np.abs(want))


@pytest.mark.parametrize("rows", [3, 40, 70, 1030])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_smallest_mx_elements(fq, rows, kind):
    """MXFP4 elements below bf16's normal range are exact: 2^-128 is the least."""
    rng = np.random.default_rng(7)
    n, k = 4200 if rows > 100 else 96, 192
    codes, _, _ = weight(rng, "mxfp4", n, k)
    scales = rng.integers(0, 3, (n, k // 32), dtype=np.uint8)
    x, xv, pieces = activations(rng, fq, kind, rows, k)
    y = fq.fp4_linear(powers(x, 100), handle(fq, "mxfp4", (codes, scales, None)), out_dtype=torch.float32)
    torch.cuda.synchronize()
    w, xv = values("mxfp4", (codes, scales, None)), np.ldexp(xv, 100)
    want, S = xv @ w.T, np.abs(xv) @ np.abs(w).T
    check(y, want, sum_bound(S, k, pieces) + HALF[torch.float32] * np.abs(want))
