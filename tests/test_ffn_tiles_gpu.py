"""Linear layers of so many rows and columns that the kernels of large tiles
run: every count of stages that their rings of buffers pass, ends inside tiles,
parts of the contraction, values that are no numbers, strides."""
import numpy as np
import pytest
import torch

import ffn_ref
from test_ffn_gpu import (FORMATS, HALF, activations, check, check_back, check_gated, check_linear, fq, handle,  # noqa: F401
                          sum_bound, values, weight)

pytestmark = pytest.mark.gpu


# 1030 rows: about one tile of 128 x 256 a CU; 2090: two.
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("rows", [1030, 2090])
@pytest.mark.parametrize("k", [64, 128, 192, 256, 320, 448])
def test_linear(fq, fmt, rows, k):
    check_linear(fq, fmt, "bf16", rows, 8200, k, rows + k, bias=k % 128 == 0)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("rows,f,k", [(1030, 4100, 64), (2090, 4100, 192), (1030, 4097, 320)])
def test_gated(fq, fmt, rows, f, k):
    check_gated(fq, fmt, "bf16", rows, f, k, rows + k)


# (k: 8256 is 64 past a tile; 8224 is no multiple of 64)
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("rows", [1030, 2090])
@pytest.mark.parametrize("n,k", [(64, 8256), (128, 8256), (192, 8256), (256, 8320), (320, 8448), (448, 8256), (128, 8224)])
def test_backward(fq, fmt, rows, n, k):
    check_back(fq, fmt, "bf16", rows, n, k, rows + n)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("rows,n,k", [(600, 8200, 4160), (300, 4100, 12352), (600, 8193, 4224)])
def test_linear_in_parts(fq, fmt, rows, n, k):
    """Few tiles: 2 and 6 parts of the contraction, which do not divide it."""
    check_linear(fq, fmt, "bf16", rows, n, k, rows + k, bias=True)


@pytest.mark.parametrize("fmt", FORMATS)
def test_gated_in_parts(fq, fmt):
    check_gated(fq, fmt, "bf16", 300, 4100, 4160, 3)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("rows,n,k", [(600, 4160, 8256), (1030, 8256, 8256), (300, 12352, 2112)])
def test_backward_in_parts(fq, fmt, rows, n, k):
    check_back(fq, fmt, "bf16", rows, n, k, rows + n)


# The block-scaled instruction adds eight neighbouring products at a time, lined up by the largest exponent among them,
# and drops what lies below 2^-13 of that (256 + 2^-5 is kept, 256 + 2^-6 is 256): less than 2^-13 of the largest
# product for each of the seven others, so 7 2^-13 of the sum of magnitudes in all.  The sums of eights are added in
# fp32: an addition for each 8 products, four times sum_bound's for 32.
def block_scaled_bound(S, k):
    return 7 * 2.0 ** -13 * S + sum_bound(S, k, 4)


@pytest.mark.parametrize("rows,n", [(2090, 2100), (2049, 2049), (2048, 2048)])
@pytest.mark.parametrize("k", [128, 256, 384, 512, 640, 896])
def test_block_scaled(fq, rows, n, k):
    """MXFP8 rows with MXFP4 weights on the instructions that take both; fp32 results of the same are not theirs."""
    print("block-scaled", rows, n, k, flush=True)
    rng = np.random.default_rng(rows + k)
    planes = weight(rng, "mxfp4", n, k)
    x, xv, _ = activations(rng, fq, "mxfp8", rows, k)
    w = values("mxfp4", planes)
    b = torch.from_numpy(rng.standard_normal(n)).bfloat16()
    got = fq.fp4_linear(x, handle(fq, "mxfp4", planes), bias=b.cuda())
    exact = fq.fp4_linear(x, handle(fq, "mxfp4", planes), bias=b.float().cuda(), out_dtype=torch.float32)
    torch.cuda.synchronize()
    want, S = xv @ w.T + b.double().numpy(), np.abs(xv) @ np.abs(w).T + b.double().abs().numpy()
    check(got, want, block_scaled_bound(S, k) + 2.0 ** -8 * np.abs(want), "bf16")
    check(exact, want, sum_bound(S, k, 1) + 2.0 ** -24 * np.abs(want), "fp32")
    # as a whole the results are off by their rounding to bf16: half a step at most, 2^-8
    assert np.linalg.norm(got.double().cpu().numpy() - want) <= 2.0 ** -8 * np.linalg.norm(want)


@pytest.mark.parametrize("rows,f,k", [(2090, 1060, 128), (2090, 1025, 512), (2048, 1024, 640)])
def test_block_scaled_gated(fq, rows, f, k):
    print("block-scaled gated", rows, f, k, flush=True)
    rng = np.random.default_rng(rows + k)
    planes = weight(rng, "mxfp4", 2 * f, k)
    x, xv, _ = activations(rng, fq, "mxfp8", rows, k)
    w = values("mxfp4", planes)
    h, products = fq.fp4_gated(x, handle(fq, "mxfp4", planes), return_products=True, products_dtype=torch.bfloat16)
    assert torch.equal(h, fq.fp4_gated(x, handle(fq, "mxfp4", planes)))
    p, tol = xv @ w.T, block_scaled_bound(np.abs(xv) @ np.abs(w).T, k)
    check(products, p, tol + 2.0 ** -8 * np.abs(p), "products")
    g, u = p[:, :f], p[:, f:]
    want = ffn_ref.gated(g, u)
    # (check_gated's: SiLU's slope is at most 1.1)
    bound = 1.1 * tol[:, :f] * (np.abs(u) + tol[:, f:]) + (np.abs(g) + tol[:, :f]) * tol[:, f:] \
        + 8 * 2.0 ** -24 * np.abs(want) + 2.0 ** -8 * np.abs(want)
    check(h, want, bound, "gated")


@pytest.mark.parametrize("fmt,kind", [("nvfp4", "bf16"), ("mxfp4", "bf16"), ("mxfp4", "mxfp8")])
@pytest.mark.parametrize("rows", [1030, 2090])
def test_no_numbers(fq, fmt, kind, rows):
    """A NaN scale of the weight fills its column, one of a row its row; an infinity stays in its row."""
    rng = np.random.default_rng(8)
    n, k = 8200, 256
    planes = weight(rng, fmt, n, k)
    planes[1][8199, 3] = 0x7F if fmt == "nvfp4" else 0xFF
    planes[1][515, 0] = 0x7F if fmt == "nvfp4" else 0xFF
    x, xv, _ = activations(rng, fq, kind, rows, k)
    if kind == "mxfp8":
        x.scales[rows - 1, 2] = 255
        x.codes[130, 77] = 0x7F
    else:
        x[rows - 1, 77] = float("nan")
        x[130, 77] = float("inf")
    got = fq.fp4_linear(x, handle(fq, fmt, planes))
    torch.cuda.synchronize()
    bad = torch.zeros(rows, n, dtype=torch.bool)
    bad[:, [515, 8199]] = True
    bad[[130, rows - 1]] = True
    g = got.double().cpu()
    if kind == "bf16":
        assert not torch.isfinite(g[130]).any()
        g[130] = float("nan")
    assert torch.equal(torch.isnan(g), bad)
    w = np.nan_to_num(values(fmt, planes))
    want, S = xv @ w.T, np.abs(xv) @ np.abs(w).T
    rows_in, cols_in = np.arange(rows) != 130, np.arange(n) != 515
    rows_in[-1] = cols_in[-1] = False
    pick = np.ix_(rows_in, cols_in)
    bound = sum_bound(S, k, 1) if kind == "bf16" else block_scaled_bound(S, k)
    check(got.cpu()[pick], want[pick], (bound + HALF[got.dtype] * np.abs(want))[pick])


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("rows", [1030, 2090])
def test_no_numbers_backward(fq, fmt, rows):
    rng = np.random.default_rng(9)
    n, k = 192, 8256
    planes = weight(rng, fmt, n, k)
    block = ffn_ref.BLOCK[fmt]
    planes[1][191, k // block - 1] = 0x7F if fmt == "nvfp4" else 0xFF
    dy, _, _ = activations(rng, fq, "bf16", rows, n)
    dy[rows - 1, 70] = float("nan")
    got = fq.fp4_linear_backward(dy, handle(fq, fmt, planes))
    torch.cuda.synchronize()
    bad = torch.zeros(rows, k, dtype=torch.bool)
    bad[:, k - block:] = True
    bad[-1] = True
    assert torch.equal(torch.isnan(got.cpu()), bad)


@pytest.mark.parametrize("rows", [1030, 2090])
@pytest.mark.parametrize("fmt", FORMATS)
def test_strides(fq, fmt, rows):
    """Rows inside a wider buffer: aligned ones, then ones that start between pieces; x of one row for all of them."""
    rng = np.random.default_rng(10)
    n, k = 8200, 192
    planes = weight(rng, fmt, n, k)
    w = handle(fq, fmt, planes)
    x, _, _ = activations(rng, fq, "bf16", rows, k)
    want = fq.fp4_linear(x, w)
    for offset, extra in ((8, 72), (1, 3), (8, 9)):
        wide = torch.full((rows, offset + k + extra), float("nan"), dtype=x.dtype, device="cuda")
        wide[:, offset:offset + k] = x
        got = fq.fp4_linear(wide[:, offset:offset + k], w)
        if offset % 8 == 0 and extra % 8 == 0:
            assert torch.equal(got, want)
        # (another kernel: sums in another order, so the neighbouring bf16 value at most)
        assert (got.float() - want.float()).abs().max() <= 2.0 ** -7 * want.float().abs().max()
    one = fq.fp4_linear(x[:1].expand(rows, k), w)
    assert torch.equal(one, one[:1].expand(rows, n))


@pytest.mark.parametrize("fmt,kind", [("nvfp4", "bf16"), ("mxfp4", "bf16"), ("mxfp4", "mxfp8")])
@pytest.mark.parametrize("rows", [1030, 2090])
def test_nothing_past_the_ends_and_again(fq, fmt, kind, rows):
    """Results go to their places alone, and a second call repeats them bit for bit."""
    rng = np.random.default_rng(11)
    n, k = 8200, 128
    w = handle(fq, fmt, weight(rng, fmt, n, k))
    x, _, _ = activations(rng, fq, kind, rows, k)
    space = torch.full((rows * n + 8192,), 7.0, dtype=torch.bfloat16, device="cuda")
    out = space[4096:4096 + rows * n].view(rows, n)
    fq.fp4_linear(x, w, out=out)
    first = out.clone()
    for _ in range(3):
        out.fill_(3.0)
        fq.fp4_linear(x, w, out=out)
        assert torch.equal(out, first)
    assert (space[:4096] == 7).all() and (space[4096 + rows * n:] == 7).all()


# Few rows of wide weights: two, four and six tiles of the weight a workgroup, the last of them partly there.
@pytest.mark.parametrize("fmt,kind", [("nvfp4", "bf16"), ("mxfp4", "bf16"), ("mxfp4", "mxfp8"), ("nvfp4", "mxfp8")])
@pytest.mark.parametrize("rows", [17, 32, 33, 48])
@pytest.mark.parametrize("n,k", [(8193, 160), (16401, 416), (20001, 96)])
def test_few_rows_wide(fq, fmt, kind, rows, n, k):
    check_linear(fq, fmt, kind, rows, n, k, rows + n, bias=True)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("rows,f,k", [(24, 8200, 160), (40, 8201, 288), (24, 10001, 416), (48, 10007, 160)])
def test_few_rows_wide_gated(fq, fmt, rows, f, k):
    check_gated(fq, fmt, "bf16", rows, f, k, rows + f)


@pytest.mark.parametrize("fmt", FORMATS)
def test_parts_captured_and_on_two_streams(fq, fmt):
    """Calls whose parts lie in memory of the call's own: replayed beside eager ones, and two at once."""
    rng = np.random.default_rng(13)
    n, k = 8200, 4160
    w = handle(fq, fmt, weight(rng, fmt, n, k))
    back = handle(fq, fmt, weight(rng, fmt, k, 8256))
    xs = [activations(rng, fq, "bf16", 600, k)[0] for _ in range(4)]
    want = [(fq.fp4_linear(x, w), fq.fp4_linear_backward(x, back)) for x in xs]
    x = xs[0].clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, dx = fq.fp4_linear(x, w), fq.fp4_linear_backward(x, back)
    for i in (1, 2, 3, 0):
        x.copy_(xs[i])
        graph.replay()
        assert torch.equal(fq.fp4_linear(xs[i - 1], w), want[i - 1][0])      # (eager, while the graph's results wait)
        torch.cuda.synchronize()
        assert torch.equal(y, want[i][0]) and torch.equal(dx, want[i][1])
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for i in range(4):
        for j, s in enumerate(streams):
            with torch.cuda.stream(s):
                a = xs[(i + j) % 4]
                got[j].append((fq.fp4_linear(a, w), fq.fp4_linear_backward(a, back)))
    torch.cuda.synchronize()
    for j in range(2):
        for i in range(4):
            y, dx = got[j][i]
            assert torch.equal(y, want[(i + j) % 4][0]) and torch.equal(dx, want[(i + j) % 4][1])


@pytest.mark.parametrize("which,offset", [("codes", 1), ("codes", 8), ("scales", 1), ("scales", 2), ("x", 4), ("x", 3),
                                          ("x_scales", 1), ("none", 0)])
def test_planes_between_words(fq, which, offset):
    """Planes of many rows that begin anywhere."""
    rng = np.random.default_rng(14)
    rows, n, k = 2049, 2050, 256
    planes = weight(rng, "mxfp4", n, k)
    x, xv, _ = activations(rng, fq, "mxfp8", rows, k)

    def at(t, name):
        space = torch.empty(t.numel() + 64, dtype=torch.uint8, device="cuda")
        o = offset if name == which else 0
        space[o:o + t.numel()] = t.reshape(-1)
        return space[o:o + t.numel()].view(t.shape)

    w = fq.Fp4Weight("mxfp4", at(torch.from_numpy(planes[0]).cuda(), "codes"),
                     at(torch.from_numpy(planes[1]).cuda(), "scales"))
    y = fq.fp4_linear(fq.Mx8Result(at(x.codes, "x"), at(x.scales, "x_scales")), w)
    dy = rng.standard_normal((rows, n))
    dt = torch.from_numpy(dy).bfloat16()
    dx = fq.fp4_linear_backward(dt.cuda(), w)
    z = fq.fp4_linear(torch.from_numpy(xv).bfloat16().cuda(), w)             # (MXFP8 values are exact in bf16)
    torch.cuda.synchronize()
    v = values("mxfp4", planes)
    want, S = xv @ v.T, np.abs(xv) @ np.abs(v).T
    check(y, want, block_scaled_bound(S, k) + 2.0 ** -8 * np.abs(want), "mxfp8")
    check(z, want, sum_bound(S, k, 1) + 2.0 ** -8 * np.abs(want), "bf16")
    d = dt.double().numpy()
    want, S = d @ v, np.abs(d) @ np.abs(v)
    check(dx, want, sum_bound(S, n, 1) + 2.0 ** -8 * np.abs(want), "gradient")
