"""Linear layers over 4-bit weights, the gated pair, the norm and their
gradients on the GPU against 64-bit arithmetic."""
import numpy as np
import pytest
import torch

import ffn_ref

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def fq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import fp4_block_scaled_row_amd as m
    m.load()
    return m


# Tolerances.  Operands are exact, so a sum of `terms` products is off by its fp32 additions alone: one rounding, 2^-24
# of a partial sum and 2^-23 where the instruction cuts it off, for each 32 products (and for each of the three pieces
# of an fp32 operand) and for each join.  A partial sum is at most S, the sum of the products' magnitudes.
def sum_bound(S, terms, pieces):
    return (pieces * (terms / 32 + 1) + 40) * 2.0 ** -23 * S


# The result's rounding: half a step of its type, relative.  (bf16's subnormal range is not reached.)
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def check(got, want, bound, what=""):
    got = got.double().cpu().numpy()
    assert got.shape == want.shape
    assert np.array_equal(np.isnan(got), np.isnan(want)), what + ": NaN in other places"
    fine = np.isfinite(want)
    assert np.array_equal(got[~fine & ~np.isnan(want)], want[~fine & ~np.isnan(want)]), what + ": infinities differ"
    err, tol = np.abs(got - want)[fine], np.broadcast_to(bound, want.shape)[fine]
    worst = np.max(err - tol, initial=-1.0)
    assert worst <= 0, "%s: off by %g more than the bound" % (what, worst)


def weight(rng, fmt, n, k):
    codes = rng.integers(0, 256, (n, k // 2), dtype=np.uint8)
    span = (0x18, 0x49) if fmt == "nvfp4" else (118, 124)
    scales = rng.integers(*span, (n, k // ffn_ref.BLOCK[fmt]), dtype=np.uint8)
    return codes, scales, 0.0371 if fmt == "nvfp4" else None


def handle(fq, fmt, planes):
    codes, scales, g = planes
    return fq.Fp4Weight(fmt, torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda(),
                        None if g is None else torch.tensor([g], device="cuda"))


def values(fmt, planes):
    codes, scales, g = planes
    return ffn_ref.row_values(fmt, codes, scales, 1.0 if g is None else np.float32(g))


def activations(rng, fq, kind, rows, k):
    """(what the call takes, float64 values, pieces of the kind)."""
    x = rng.standard_normal((rows, k)) * np.where(rng.random(k) > 0.95, 20, 1)
    if kind == "mxfp8":
        codes, scales = ffn_ref.mxfp8_of(x)
        return (fq.Mx8Result(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda()),
                ffn_ref.mxfp8_values(codes, scales), 1)
    t = torch.from_numpy(x).to(DT[kind])
    return t.cuda(), t.double().numpy(), 3 if kind == "f32" else 1


def out_type(kind):
    return torch.float32 if kind == "f32" else torch.bfloat16


def check_linear(fq, fmt, kind, rows, n, k, seed, bias=False):
    print("linear", fmt, kind, rows, n, k, bias, flush=True)
    rng = np.random.default_rng(seed)
    planes = weight(rng, fmt, n, k)
    x, xv, pieces = activations(rng, fq, kind, rows, k)
    w, t = values(fmt, planes), out_type(kind)
    b = torch.from_numpy(rng.standard_normal(n)).to(t) if bias else None
    got = fq.fp4_linear(x, handle(fq, fmt, planes), bias=None if b is None else b.cuda())
    torch.cuda.synchronize()
    assert got.dtype == t
    want = xv @ w.T + (b.double().numpy() if bias else 0.0)
    S = np.abs(xv) @ np.abs(w).T + (np.abs(b.double().numpy()) if bias else 0.0)
    check(got, want, sum_bound(S, k, pieces) + HALF[t] * np.abs(want), "linear")
    if kind == "f32" and k >= 256:
        # the roundings have no direction: sqrt(k / 32 + 8) of them of 2^-24 each, three times that at most; two
        # pieces instead of three would leave 2^-17
        rel = np.linalg.norm(got.double().cpu().numpy() - want) / np.linalg.norm(want)
        assert rel <= 3 * 2.0 ** -24 * np.sqrt(k / 32 + 8)


FORMATS = ["nvfp4", "mxfp4"]
KINDS = ["bf16", "f32", "mxfp8"]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows", [1, 2, 15, 16, 17, 33, 64])
@pytest.mark.parametrize("n,k", [(1, 32), (16, 128), (50, 416), (131, 1312)])
def test_linear_few_rows(fq, fmt, kind, rows, n, k):
    check_linear(fq, fmt, kind, rows, n, k, rows * 7 + n)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows,n,k", [(65, 1, 32), (65, 130, 96), (100, 257, 640), (128, 128, 64), (300, 70, 2080)])
def test_linear_many_rows(fq, fmt, kind, rows, n, k):
    check_linear(fq, fmt, kind, rows, n, k, rows + n, bias=True)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("kind", KINDS)
def test_linear_large_tiles(fq, fmt, kind):
    """Enough tiles that the large ones are taken, with ends inside them."""
    check_linear(fq, fmt, kind, 2090, 8200, 160, 5, bias=True)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [1, 20, 70])
@pytest.mark.parametrize("k", [16, 48, 144, 272, 1360])
def test_linear_half_pieces(fq, kind, rows, k):
    """NVFP4 rows that end in the middle of a lane's 32 elements."""
    check_linear(fq, "nvfp4", kind, rows, 37, k, k, bias=True)


def check_back(fq, fmt, kind, rows, n, k, seed):
    print("back", fmt, kind, rows, n, k, flush=True)
    rng = np.random.default_rng(seed)
    planes = weight(rng, fmt, n, k)
    dy, dv, pieces = activations(rng, fq, kind, rows, n)
    w = values(fmt, planes)
    got = fq.fp4_linear_backward(dy, handle(fq, fmt, planes))
    torch.cuda.synchronize()
    want, S = dv @ w, np.abs(dv) @ np.abs(w)
    check(got, want, sum_bound(S, n, pieces) + HALF[got.dtype] * np.abs(want), "backward")


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("rows,n,k", [(1, 1, 32), (1, 40, 128), (3, 129, 96), (64, 64, 256), (65, 1000, 160),
                                      (200, 77, 416), (130, 515, 1312)])
def test_linear_backward(fq, fmt, kind, rows, n, k):
    check_back(fq, fmt, kind, rows, n, k, rows + n + k)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_linear_backward_large_tiles(fq, fmt, kind):
    check_back(fq, fmt, kind, 2090, 135, 8224, 11)


@pytest.mark.parametrize("k", [16, 48, 144])
def test_linear_backward_half_pieces(fq, k):
    check_back(fq, "nvfp4", "bf16", 33, 70, k, k)


def check_gated(fq, fmt, kind, rows, f, k, seed):
    print("gated", fmt, kind, rows, f, k, flush=True)
    rng = np.random.default_rng(seed)
    planes = weight(rng, fmt, 2 * f, k)
    x, xv, pieces = activations(rng, fq, kind, rows, k)
    w, t = values(fmt, planes) , out_type(kind)
    h, products = fq.fp4_gated(x, handle(fq, fmt, planes), return_products=True)
    alone = fq.fp4_gated(x, handle(fq, fmt, planes))
    torch.cuda.synchronize()
    assert torch.equal(h, alone)
    p, tol = xv @ w.T, sum_bound(np.abs(xv) @ np.abs(w).T, k, pieces)
    assert products.dtype == torch.float32
    check(products, p, tol + 2.0 ** -24 * np.abs(p), "products")
    _, rounded = fq.fp4_gated(x, handle(fq, fmt, planes), return_products=True, products_dtype=torch.bfloat16)
    assert torch.equal(rounded, products.bfloat16())
    g, u = p[:, :f], p[:, f:]
    want = ffn_ref.gated(g, u)
    # |SiLU'| <= 1.1, and 1 + |g| <= ... of it where the sums' errors meet: first order, and the second by 1.1 of both;
    # exponential, sum, quotient and two products: 8 roundings
    bound = 1.1 * tol[:, :f] * (np.abs(u) + tol[:, f:]) + (np.abs(g) + tol[:, :f]) * tol[:, f:] \
        + 8 * 2.0 ** -24 * np.abs(want) + HALF[t] * np.abs(want)
    check(h, want, bound, "gated")


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows,f,k", [(1, 1, 32), (1, 40, 1312), (16, 33, 256), (17, 50, 416), (64, 16, 128),
                                      (65, 70, 96), (130, 257, 672)])
def test_gated(fq, fmt, kind, rows, f, k):
    check_gated(fq, fmt, kind, rows, f, k, rows + f)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("kind", KINDS)
def test_gated_large_tiles(fq, fmt, kind):
    check_gated(fq, fmt, kind, 2090, 4100, 96, 3)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("p_kind", ["bf16", "f32"])
@pytest.mark.parametrize("rows,f,k", [(1, 1, 32), (5, 37, 96), (70, 64, 160), (90, 301, 416)])
def test_gated_backward(fq, fmt, kind, p_kind, rows, f, k):
    print("gated backward", fmt, kind, rows, f, k, flush=True)
    rng = np.random.default_rng(rows + f)
    planes = weight(rng, fmt, 2 * f, k)
    w = values(fmt, planes)
    dh, dhv, pieces = activations(rng, fq, kind, rows, f)
    products = torch.from_numpy(3 * rng.standard_normal((rows, 2 * f))).to(DT[p_kind])
    dx, dp = fq.fp4_gated_backward(dh, products.cuda(), handle(fq, fmt, planes))
    torch.cuda.synchronize()
    p = products.double().numpy()
    dg, du = ffn_ref.gated_grad(dhv, p[:, :f], p[:, f:])
    want = np.concatenate((dg, du), 1)
    # 10 roundings of a factor each; 1 + g (1 - s) is a sum whose terms are at most 1 + |g| (1 - s) for negative g
    g = p[:, :f]
    s = ffn_ref.sigmoid(g)
    terms = np.abs(dhv * p[:, f:]) * s * (1 + np.abs(g) * (1 - s))
    bound = 10 * 2.0 ** -24 * np.concatenate((terms, np.abs(du)), 1) + HALF[DT[kind]] * np.abs(want)
    check(dp, want, bound, "gradient of the products")
    # the product is that of the returned, rounded gradients
    d = dp.double().cpu().numpy()
    check(dx, d @ w, sum_bound(np.abs(d) @ np.abs(w), 2 * f, pieces) + HALF[DT[kind]] * np.abs(d @ w), "gradient of x")


def test_gated_gradient_against_differences(fq):
    """The gradient of sum(dh * h) along a random direction of x, fp32."""
    rng = np.random.default_rng(8)
    rows, f, k = 6, 40, 128
    planes = weight(rng, "nvfp4", 2 * f, k)
    w = handle(fq, "nvfp4", planes)
    x = torch.from_numpy(rng.standard_normal((rows, k))).float().cuda()
    dh = torch.from_numpy(rng.standard_normal((rows, f))).float().cuda()
    along = torch.from_numpy(rng.standard_normal((rows, k))).float().cuda()
    _, products = fq.fp4_gated(x, w, return_products=True)
    dx, _ = fq.fp4_gated_backward(dh, products, w)
    step = 2.0 ** -7
    up, down = ((fq.fp4_gated(x + s * step * along, w).double() * dh.double()).sum() for s in (1, -1))
    want = float((up - down) / (2 * step))
    got = float((dx.double() * along.double()).sum())
    # the difference's own error: step^2 / 6 of the third derivative (SiLU's are below 1, of a direction whose products
    # are about |w| sqrt(k)) and 2^-24 / step of the values
    p = along.double().cpu().numpy() @ values("nvfp4", planes).T
    v = np.abs(dh.double().cpu().numpy())
    both = np.abs(products.double().cpu().numpy())
    third = (v * (np.abs(p[:, :f]) ** 3 * both[:, f:] + 3 * np.abs(p[:, :f]) ** 2 * np.abs(p[:, f:]))).sum()
    size = (v * both[:, :f] * both[:, f:]).sum()
    assert abs(got - want) <= step ** 2 / 6 * third + 2.0 ** -20 / step * size


# ------------------------------------------------------------------------------------------------- norm

EPS = 1e-5


def rows_of(rng, rows, d, t, stride=None):
    x = rng.standard_normal((rows, d)) * np.where(rng.random(d) > 0.97, 15, 1)
    t = torch.from_numpy(x).to(t)
    if stride is None:
        return t.cuda(), t.double().numpy()
    wide = torch.zeros((rows, stride), dtype=t.dtype, device="cuda")
    wide[:, :d] = t.cuda()
    return wide[:, :d], t.double().numpy()


# s and w exact; the sum of squares: at most d / 64 / ... additions in a lane (64) and 10 halvings, all of one sign:
# 74 roundings of its relative error at most, half of it in r, with the quotient, sum, root and quotient: 42; y has 2 more
R_TOL = 42 * 2.0 ** -24
Y_TOL = 44 * 2.0 ** -24


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("w_kind", ["bf16", "f32"])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("rows,d", [(1, 1), (5, 7), (3, 64), (9, 500), (4, 1000), (2, 2048), (3, 4093), (2, 8192),
                                    (1, 8200), (2, 20000), (1, 32768)])
def test_norm(fq, kind, w_kind, residual, rows, d):
    print("norm", kind, w_kind, residual, rows, d, flush=True)
    rng = np.random.default_rng(d)
    t = DT[kind]
    x, xv = rows_of(rng, rows, d, t)
    w = torch.from_numpy(1 + 0.3 * rng.standard_normal(d)).to(DT[w_kind])
    res = rows_of(rng, rows, d, t) if residual else (None, 0.0)
    r = fq.rms_norm(x, w.cuda(), residual=res[0], eps=EPS, return_rstd=True)
    torch.cuda.synchronize()
    s = xv
    if residual:
        want = (x.float() + res[0].float()).to(t)       # (a sum of two is rounded once either way)
        assert torch.equal(r.summed, want)
        s = want.double().cpu().numpy()
    else:
        assert r.summed is None
    y, rstd = ffn_ref.rms_norm(s, w.double().numpy(), EPS)
    check(r.rstd, rstd, R_TOL * rstd, "rstd")
    check(r.out, y, (Y_TOL + HALF[t]) * np.abs(y), "y")


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("rows,d", [(1, 32), (7, 96), (3, 544), (2, 1056), (2, 4096), (3, 8192), (1, 16416)])
def test_norm_mxfp8(fq, kind, rows, d):
    """Bytes of the quantization of y: equal to those of the exact y wherever its error cannot decide, and off by one
    code at most elsewhere."""
    print("norm mxfp8", kind, rows, d, flush=True)
    rng = np.random.default_rng(d + 1)
    x, xv = rows_of(rng, rows, d, DT[kind])
    if rows > 1:
        x[0, :32] = 0
        xv[0, :32] = 0
    w = torch.from_numpy(1 + 0.3 * rng.standard_normal(d)).to(DT[kind])
    r = fq.rms_norm(x, w.cuda(), eps=EPS, quantize="mxfp8")
    back = {t: fq.dequantize("mxfp8", *r.out, out_dtype=t) for t in (torch.float32, torch.bfloat16)}
    torch.cuda.synchronize()
    y, _ = ffn_ref.rms_norm(xv, w.double().numpy(), EPS)
    codes, scales = r.out.codes.cpu().numpy(), r.out.scales.cpu().numpy()
    lo, hi = (ffn_ref.mxfp8_of(y * (1 + e)) for e in (-Y_TOL, Y_TOL))
    assert np.all((scales == lo[1]) | (scales == hi[1]))
    assert np.all((codes == lo[0]) | (codes == hi[0]))
    got = ffn_ref.mxfp8_values(codes, scales)
    for t, v in back.items():
        assert np.array_equal(v.double().cpu().numpy(), got)
    if rows > 1:
        assert np.all(scales[0, 0] == 127) and not codes[0, :32].any()


def test_norm_mxfp8_edges(fq):
    """Blocks of zeros, of the smallest numbers, of values past 448 steps, and those that are not finite."""
    d = 32 * 6
    x = torch.zeros(3, d)
    x[0, 32:64] = 2.0 ** -126
    x[0, 64] = 511.0 / 256
    x[0, 65] = 464.0 / 256
    x[0, 96:128] = torch.linspace(-1, 1, 32)
    x[1, 5] = float("inf")
    x[2, 100] = float("nan")
    w = torch.ones(d)
    w[128:160] = 2.0 ** 100
    x[0, 128:160] = 1.0
    r = fq.rms_norm(x.cuda(), w.cuda(), eps=1.0, quantize="mxfp8")
    plain = fq.rms_norm(x.cuda(), w.cuda(), eps=1.0).out
    torch.cuda.synchronize()
    codes, scales = ffn_ref.mxfp8_of(plain.double().cpu().numpy())
    assert np.array_equal(r.out.codes.cpu().numpy(), codes)
    assert np.array_equal(r.out.scales.cpu().numpy(), scales)
    # (infinity over an infinite mean: NaN; the other elements of its row are zeros)
    assert scales[1, 0] == 255 and np.all(scales[1, 1:] == 127) and np.all(scales[2] == 255)


def check_norm_back(fq, kind, w_kind, rows, d, ds, stride=None):
    print("norm backward", kind, w_kind, rows, d, ds, stride, flush=True)
    rng = np.random.default_rng(rows + d)
    t = DT[kind]
    s, sv = rows_of(rng, rows, d, t, stride)
    dy, dyv = rows_of(rng, rows, d, t, stride)
    extra = rows_of(rng, rows, d, t, stride) if ds else (None, 0.0)
    w = torch.from_numpy(1 + 0.3 * rng.standard_normal(d)).to(DT[w_kind])
    r = fq.rms_norm(s, w.cuda(), eps=EPS, return_rstd=True)
    dx, dw = fq.rms_norm_backward(dy, s, w.cuda(), r.rstd, dsummed=extra[0])
    torch.cuda.synchronize()
    assert dx.dtype == t and dw.dtype == w.dtype
    wv = w.double().numpy()
    want_dx, want_dw = ffn_ref.rms_norm_grad(dyv, sv, wv, EPS)
    want_dx = want_dx + extra[1]
    # each term is off by R_TOL twice (r in hat, and in front) and few roundings; the mean of g hat by the sums' 74
    rs = r.rstd.double().cpu().numpy()[:, None]
    along = (np.abs(dyv * wv * sv).sum(1)[:, None] * rs / d)
    terms = rs * np.abs(dyv * wv) + np.abs(sv) * rs * rs * along
    tol = (4 * R_TOL + 90 * 2.0 ** -24) * terms + 2.0 ** -24 * np.abs(extra[1])
    check(dx, want_dx, tol + HALF[t] * np.abs(want_dx), "dx")
    # rows / parts additions in a thread and as many as parts in the join
    terms = (np.abs(dyv * sv) * rs).sum(0)
    check(dw, want_dw, (R_TOL + (rows + 20) * 2.0 ** -24) * terms + HALF[w.dtype] * np.abs(want_dw), "dw")


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("ds", [False, True])
@pytest.mark.parametrize("rows,d", [(1, 1), (3, 7), (600, 64), (5, 512), (4, 1000), (2, 2048), (700, 2100), (3, 4093),
                                    (2, 8192), (600, 8200), (3, 20000), (2, 32768)])
def test_norm_backward(fq, kind, ds, rows, d):
    check_norm_back(fq, kind, kind, rows, d, ds)


@pytest.mark.parametrize("kind,w_kind", [("bf16", "f32"), ("f32", "bf16")])
def test_norm_backward_mixed(fq, kind, w_kind):
    check_norm_back(fq, kind, w_kind, 40, 333, True, stride=351)


def test_norm_gradient_against_differences(fq):
    rng = np.random.default_rng(4)
    rows, d = 4, 96
    x, w, dy, a, b = (torch.from_numpy(rng.standard_normal(s)).float().cuda()
                      for s in ((rows, d), (d,), (rows, d), (rows, d), (d,)))
    r = fq.rms_norm(x, w, eps=EPS, return_rstd=True)
    dx, dw = fq.rms_norm_backward(dy, x, w, r.rstd)
    step = 2.0 ** -7

    def value(x, w):
        return float((fq.rms_norm(x, w, eps=EPS).out.double() * dy.double()).sum())

    # rows of about one: third derivatives of the direction's size to the third, roundings 2^-24 over the step
    size = float((dy.abs() * w.abs()).sum())
    tol = step ** 2 * 6 * float(a.abs().max()) ** 3 * size + 2.0 ** -20 / step * size
    want = (value(x + step * a, w) - value(x - step * a, w)) / (2 * step)
    assert abs(float((dx.double() * a.double()).sum()) - want) <= tol
    want = (value(x, w + step * b) - value(x, w - step * b)) / (2 * step)
    assert abs(float((dw.double() * b.double()).sum()) - want) <= tol
