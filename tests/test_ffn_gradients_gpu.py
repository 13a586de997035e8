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


def functions(fq):
    """A user's joints of forward and backward calls."""

    class Linear(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, w, bias):
            ctx.w = w
            return fq.fp4_linear(x, w, bias=bias)

        @staticmethod
        def backward(ctx, dy):
            return fq.fp4_linear_backward(dy.contiguous(), ctx.w), None, dy.sum(0)

    class Gated(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, w):
            h, products = fq.fp4_gated(x, w, return_products=True)
            ctx.save_for_backward(products)
            ctx.w = w
            return h

        @staticmethod
        def backward(ctx, dh):
            return fq.fp4_gated_backward(dh.contiguous(), ctx.saved_tensors[0], ctx.w)[0], None

    class Norm(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, residual, gain):
            r = fq.rms_norm(x, gain, residual=residual, return_rstd=True)
            ctx.save_for_backward(r.summed, gain, r.rstd)
            return r.out, r.summed

        @staticmethod
        def backward(ctx, dy, ds):
            dx, dgain = fq.rms_norm_backward(dy.contiguous(), *ctx.saved_tensors, dsummed=ds.contiguous())
            return dx, dx, dgain

    return Linear.apply, Gated.apply, Norm.apply


@pytest.mark.parametrize("rows", [6, 40, 150])
def test_block_under_autograd(fq, rows):
    """A block with low-rank adapters around frozen 4-bit weights, in fp32: all gradients against those of the same block
    in 64 bits, and as far as differences of it tell."""
    rng = np.random.default_rng(rows)
    d, f, r = 128, 160, 8
    up, down = weight(rng, "nvfp4", 2 * f, d), weight(rng, "mxfp4", d, f)
    t = {k: torch.from_numpy(a).float() for k, a in dict(
        x=rng.standard_normal((rows, d)), res=rng.standard_normal((rows, d)), gain=1 + 0.2 * rng.standard_normal(d),
        bias=rng.standard_normal(d), a=0.1 * rng.standard_normal((d, r)), b=0.1 * rng.standard_normal((r, d)),
        out=0.01 * rng.standard_normal((rows, d))).items()}
    scale = 1 / np.abs(values("nvfp4", up)).sum(1).max(), 1 / np.abs(values("mxfp4", down)).sum(1).max()
    norm_up, norm_down = values("nvfp4", up), values("mxfp4", down)

    def block(v, linear, gated, norm):
        y, s = norm(v["x"] * 1, v["res"], v["gain"])
        h = gated(y * scale[0] + y @ v["a"] @ v["b"])
        return s + linear(h * scale[1], v["bias"])

    linear, gated, norm = functions(fq)
    wu, wd = handle(fq, "nvfp4", up), handle(fq, "mxfp4", down)
    mine = {k: a.cuda().requires_grad_(k != "out") for k, a in t.items()}
    with torch.no_grad():
        assert not fq.fp4_linear(mine["x"], handle(fq, "mxfp4", weight(rng, "mxfp4", 32, d))).requires_grad
    got = block(mine, lambda h, b: linear(h, wd, b), lambda y: gated(y, wu), norm)
    assert got.requires_grad
    (got * mine["out"]).sum().backward()

    exact = {k: a.double().requires_grad_(k != "out") for k, a in t.items()}
    vu, vd = torch.from_numpy(norm_up), torch.from_numpy(norm_down)

    def norm64(x, res, gain):
        s = x + res
        return s / (s.square().mean(1, keepdim=True) + 1e-6).sqrt() * gain, s

    def gated64(y):
        p = y @ vu.t()
        return p[:, :f] * torch.sigmoid(p[:, :f]) * p[:, f:]

    def loss(v):
        return (block(v, lambda h, b: h @ vd.t() + b, gated64, norm64) * v["out"]).sum()

    loss(exact).backward()
    # fp32 throughout: each of some ten operations in a row is off by sum_bound of its terms (2^-23 (f / 32 + 41) of its
    # magnitudes), and magnitudes exceed results by the condition of the sums, sqrt of some hundred terms
    tol = 10 * 2.0 ** -23 * (3 * (2 * f / 32 + 1) + 40) * 16
    for k in t:
        if k == "out":
            continue
        want, have = exact[k].grad, mine[k].grad.double().cpu()
        assert (have - want).norm() <= tol * want.norm(), k
        # along a direction, from differences in 64 bits: the third derivative's part is the step's square
        way = torch.randn(want.shape, generator=torch.Generator().manual_seed(1)).double()
        step = 1e-4
        plus, minus = ({**exact, k: (exact[k] + sign * step * way).detach()} for sign in (1, -1))
        slope = ((loss(plus) - loss(minus)) / (2 * step)).item()
        along = (have * way).sum().item()
        assert abs(slope - along) <= (tol + 1e-4) * (want.abs() * way.abs()).sum().item(), k
