"""Gradients of the gated pair and the layers as a training program joins them."""
import numpy as np
import pytest
import torch

import ffn_ref
from test_ffn_gpu import check, fq, handle, sum_bound, values, weight  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,f,k", [(5, 96, 320), (1030, 1024, 448)])
def test_one_rounding_with_fp32_gradients(fq, rows, f, k):
    """dh in fp32: dproducts keep fp32 sums' bits, and dx rounded to bf16 is off by that rounding alone."""
    rng = np.random.default_rng(rows)
    planes = weight(rng, "nvfp4", 2 * f, k)
    w = handle(fq, "nvfp4", planes)
    x = torch.from_numpy(rng.standard_normal((rows, k))).bfloat16().cuda()
    dh = torch.from_numpy(0.01 * rng.standard_normal((rows, f))).bfloat16().cuda()
    _, p = fq.fp4_gated(x, w, return_products=True)
    dx, dp = fq.fp4_gated_backward(dh.float(), p, w)
    dx16, dp16 = fq.fp4_gated_backward(dh, p, w)
    torch.cuda.synchronize()
    pv, v = p.double().cpu().numpy(), values("nvfp4", planes)
    want_dp = np.concatenate(ffn_ref.gated_grad(dh.double().cpu().numpy(), pv[:, :f], pv[:, f:]), 1)
    want, S = want_dp @ v, np.abs(want_dp) @ np.abs(v)
    err = lambda a: np.linalg.norm(a.double().cpu().numpy() - want) / np.linalg.norm(want)  # noqa: E731
    # each of the 2 f terms by dproducts' few fp32 roundings (s, 1 - s, three products, a sum; g cancels nothing of
    # 1 + g (1 - s) but near its zero, where it is 2^-22 of what cancels: within 16 of 2^-24 of |dh u| (1 + |g|))
    dhv, g, u = np.abs(dh.double().cpu().numpy()), np.abs(pv[:, :f]), np.abs(pv[:, f:])
    slack = np.concatenate([dhv * u * (1 + g), dhv * g], 1) @ np.abs(v) * 16 * 2.0 ** -24
    check(dx, want, sum_bound(S, 2 * f, 3) + slack + 2.0 ** -24 * np.abs(want))
    check(dx.bfloat16(), want, sum_bound(S, 2 * f, 3) + slack + 2.0 ** -8 * np.abs(want))
    assert dp.dtype == dx.dtype == torch.float32 and dp16.dtype == dx16.dtype == torch.bfloat16
    assert err(dx.bfloat16()) < err(dx16) < 2 * 2.0 ** -8
