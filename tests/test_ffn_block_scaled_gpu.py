"""MXFP8 rows with MXFP4 weights at sizes of the block-scaled instructions: which calls take them, seen from the
results' errors, and how far they are off."""
import numpy as np
import pytest
import torch

import ffn_ref
from test_ffn_gpu import activations, check, fq, handle, sum_bound, values, weight  # noqa: F401
from test_ffn_tiles_gpu import block_scaled_bound

pytestmark = pytest.mark.gpu


def placed(t, offset):
    space = torch.empty(t.numel() + 64, dtype=torch.uint8, device="cuda")
    space[offset:offset + t.numel()] = t.reshape(-1).cuda()
    return space[offset:offset + t.numel()].view(t.shape)


def spread(rng, fq, rows, n, k):
    """Operands whose blocks' scales and elements spread far, so that products of eight differ in size."""
    planes = weight(rng, "mxfp4", n, k)
    x, xv, _ = activations(rng, fq, "mxfp8", rows, k)
    return planes, x, xv


@pytest.mark.parametrize("codes,scales,x,x_scales", [(1, 0, 0, 0), (8, 0, 0, 0), (0, 1, 0, 0), (0, 2, 0, 0), (0, 0, 4, 0),
                                                     (0, 0, 3, 0), (0, 0, 0, 1), (0, 0, 0, 2)])
def test_planes_that_the_block_scaled_loads_do_not_take(fq, codes, scales, x, x_scales):
    """Codes off 16 bytes or scales off 4: fp32 sums, so the bound of fp32 sums."""
    rng = np.random.default_rng(14)
    rows, n, k = 2049, 2050, 256
    planes, a, xv = spread(rng, fq, rows, n, k)
    w = fq.Fp4Weight("mxfp4", placed(torch.from_numpy(planes[0]), codes), placed(torch.from_numpy(planes[1]), scales))
    y = fq.fp4_linear(fq.Mx8Result(placed(a.codes, x), placed(a.scales, x_scales)), w)
    torch.cuda.synchronize()
    v = values("mxfp4", planes)
    want, S = xv @ v.T, np.abs(xv) @ np.abs(v).T
    check(y, want, sum_bound(S, k, 1) + 2.0 ** -8 * np.abs(want))


def test_fp32_results_have_fp32_sums(fq):
    """What a caller asks for who wants no less, whatever lies where: the linear layer's and the gated pair's."""
    rng = np.random.default_rng(15)
    rows, n, k = 2048, 2048, 512
    planes, x, xv = spread(rng, fq, rows, n, k)
    w = handle(fq, "mxfp4", planes)
    y = fq.fp4_linear(x, w, out_dtype=torch.float32)
    _, p = fq.fp4_gated(x, w, return_products=True)
    torch.cuda.synchronize()
    v = values("mxfp4", planes)
    want, S = xv @ v.T, np.abs(xv) @ np.abs(v).T
    for got in (y, p):
        check(got, want, sum_bound(S, k, 1) + 2.0 ** -24 * np.abs(want))


@pytest.mark.parametrize("rows,f,k", [(2048, 1024, 512), (2090, 1025, 640)])
def test_gated_with_and_without_fp32_products(fq, rows, f, k):
    """The two take different kernels at these sizes: h may differ by the block-scaled sums' error, and no more."""
    rng = np.random.default_rng(16)
    planes, x, xv = spread(rng, fq, rows, 2 * f, k)
    w = handle(fq, "mxfp4", planes)
    alone = fq.fp4_gated(x, w)
    kept, p = fq.fp4_gated(x, w, return_products=True)
    torch.cuda.synchronize()
    v = values("mxfp4", planes)
    sums, S = xv @ v.T, np.abs(xv) @ np.abs(v).T
    g, u = sums[:, :f], sums[:, f:]
    want = ffn_ref.gated(g, u)
    for h, tol in ((alone, block_scaled_bound(S, k)), (kept, sum_bound(S, k, 1))):
        tg, tu = tol[:, :f], tol[:, f:]
        # SiLU's slope is at most 1.1
        check(h, want, 1.1 * tg * (np.abs(u) + tu) + (np.abs(g) + tg) * tu + (8 * 2.0 ** -24 + 2.0 ** -8) * np.abs(want))
    check(p, sums, sum_bound(S, k, 1) + 2.0 ** -24 * np.abs(sums))
    # over the whole output both are bf16's rounding off
    for h in (alone, kept):
        assert np.linalg.norm(h.double().cpu().numpy() - want) <= 2.0 ** -8 * np.linalg.norm(want)
