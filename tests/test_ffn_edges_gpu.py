"""Linear layers, the gated pair and the norm where they can go wrong: values
that are no numbers, empty calls, strides and alignments, buffers of the
caller's, streams, captured calls, refusals, and the operators in a row."""
import numpy as np
import pytest
import torch

import ffn_ref
from test_ffn_gpu import DT, HALF, activations, check, fq, handle, sum_bound, values, weight  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("rows", [3, 70])
def test_weights_that_are_no_numbers(fq, fmt, rows):
    """A NaN scale makes its row of the weight NaN, and only that; backward, its block of columns."""
    rng = np.random.default_rng(1)
    n, k = 70, 320
    planes = weight(rng, fmt, n, k)
    block = ffn_ref.BLOCK[fmt]
    planes[1][37, 5] = 0x7F if fmt == "nvfp4" else 0xFF
    x, xv, _ = activations(rng, fq, "bf16", rows, k)
    dy, dv, _ = activations(rng, fq, "bf16", rows, n)
    w = values(fmt, planes)
    got, back = fq.fp4_linear(x, handle(fq, fmt, planes)), fq.fp4_linear_backward(dy, handle(fq, fmt, planes))
    h = fq.fp4_gated(x, handle(fq, fmt, planes))
    torch.cuda.synchronize()
    assert torch.equal(torch.isnan(got), torch.arange(n, device="cuda").eq(37).expand(rows, n))
    cols = torch.zeros(k, dtype=torch.bool, device="cuda")
    cols[5 * block:6 * block] = True
    assert torch.equal(torch.isnan(back), cols.expand(rows, k))
    assert torch.equal(torch.isnan(h), torch.arange(n // 2, device="cuda").eq(37 - n // 2).expand(rows, n // 2))
    w = np.nan_to_num(w)
    fine = np.arange(n) != 37
    check(got[:, torch.from_numpy(fine).cuda()], (xv @ w.T)[:, fine],
          (sum_bound(np.abs(xv) @ np.abs(w).T, k, 1) + 2.0 ** -8 * np.abs(xv @ w.T))[:, fine])


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [5, 90])
def test_rows_that_are_no_numbers(fq, kind, rows):
    """An infinity or NaN stays in its row; with an infinity the row is infinite or NaN as the sum is."""
    rng = np.random.default_rng(2)
    n, k = 48, 192
    planes = weight(rng, "nvfp4", n, k)
    x, _, pieces = activations(rng, fq, kind, rows, k)
    x[1, 7] = float("inf")
    x[2, 100] = float("nan")
    x[4, 3] = float("-inf")
    xv, w = x.double().cpu().numpy(), values("nvfp4", planes)
    got = fq.fp4_linear(x, handle(fq, "nvfp4", planes))
    torch.cuda.synchronize()
    with np.errstate(invalid="ignore"):
        want = np.stack([(r * w).sum(1) for r in xv])
        S = np.nan_to_num(np.abs(xv), posinf=0) @ np.abs(w).T
    check(got, want, sum_bound(S, k, pieces) + HALF[got.dtype] * np.nan_to_num(np.abs(want), posinf=0), "rows")


@pytest.mark.parametrize("rows", [2, 70])
def test_signalling_nan_of_few_bits(fq, rows):
    """A NaN whose upper 16 bits alone would be an infinity."""
    planes = weight(np.random.default_rng(0), "mxfp4", 32, 64)
    x = torch.ones(rows, 64)
    x.view(torch.int32)[1, 5] = 0x7F800001
    got = fq.fp4_linear(x.cuda(), handle(fq, "mxfp4", planes))
    assert bool(torch.isnan(got[1]).all()) and not bool(torch.isnan(got[0]).any())


@pytest.mark.parametrize("rows", [4, 80])
def test_large_and_small_fp32_rows(fq, rows):
    """fp32's largest values do not pass bf16's range in pieces, and the smallest keep their bits."""
    rng = np.random.default_rng(3)
    n, k = 40, 64
    planes = weight(rng, "mxfp4", n, k)
    planes[1][:] = 100                                   # 2^-27
    x = torch.from_numpy(rng.standard_normal((rows, k))).float()
    x[0] *= 2.0 ** 126 / x[0].abs().max()
    x[0, 0] = torch.finfo(torch.float32).max
    x[1] *= 2.0 ** -70
    w = values("mxfp4", planes)
    got = fq.fp4_linear(x.cuda(), handle(fq, "mxfp4", planes))
    torch.cuda.synchronize()
    xv = x.double().numpy()
    check(got, xv @ w.T, sum_bound(np.abs(xv) @ np.abs(w).T, k, 3), "rows")


@pytest.mark.parametrize("rows", [3, 70])
def test_gates_far_out(fq, rows):
    """SiLU of large negative gates is zero, of large positive ones the gate."""
    f, k = 32, 32
    codes = np.full((2 * f, k // 2), 0x22, dtype=np.uint8)        # ones
    scales = np.full((2 * f, 1), 127, dtype=np.uint8)
    x = torch.zeros(rows, k)
    x[0, 0], x[1, 0] = -1000.0, 1000.0
    w = handle(fq, "mxfp4", (codes, scales, None))
    h, p = fq.fp4_gated(x.cuda(), w, return_products=True)
    dx, dp = fq.fp4_gated_backward(torch.ones(rows, f).cuda(), p, w)
    torch.cuda.synchronize()
    assert h[0].abs().max() == 0 and torch.all(h[1] == 1e6) and h[2].abs().max() == 0
    assert torch.isfinite(dx).all()
    assert dp[0].abs().max() == 0 and torch.all(dp[1] == 1000) and dp[2].abs().max() == 0


def test_empty_calls(fq):
    planes = weight(np.random.default_rng(0), "nvfp4", 6, 32)
    w = handle(fq, "nvfp4", planes)
    x = torch.zeros(0, 32, dtype=torch.bfloat16, device="cuda")
    assert fq.fp4_linear(x, w).shape == (0, 6)
    h, p = fq.fp4_gated(x, w, return_products=True)
    assert h.shape == (0, 3) and p.shape == (0, 6)
    dx, dp = fq.fp4_gated_backward(h, p, w)
    assert dx.shape == (0, 32) and dp.shape == (0, 6)
    assert fq.fp4_linear_backward(torch.zeros(0, 6, device="cuda"), w).shape == (0, 32)
    r = fq.rms_norm(x, torch.ones(32, device="cuda"), return_rstd=True)
    assert r.out.shape == (0, 32) and r.rstd.shape == (0,)
    dx, dw = fq.rms_norm_backward(x, x, torch.ones(32, device="cuda"), r.rstd)
    torch.cuda.synchronize()
    assert dx.shape == (0, 32) and dw.abs().max() == 0
    # no elements to sum over: the bias alone, zeros
    none = fq.Fp4Weight("mxfp4", torch.zeros(5, 0, dtype=torch.uint8, device="cuda"),
                        torch.zeros(5, 0, dtype=torch.uint8, device="cuda"))
    for rows in (2, 70):
        bias = torch.arange(5.0, device="cuda")
        got = fq.fp4_linear(torch.zeros(rows, 0, device="cuda"), none, bias=bias)
        assert torch.equal(got, bias.expand(rows, 5))
    none = fq.Fp4Weight("mxfp4", torch.zeros(0, 32, dtype=torch.uint8, device="cuda"),
                        torch.zeros(0, 2, dtype=torch.uint8, device="cuda"))
    assert fq.fp4_linear_backward(torch.zeros(3, 0, device="cuda"), none).abs().max() == 0
    assert fq.fp4_linear(torch.zeros(3, 64, device="cuda"), none).shape == (3, 0)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [1, 7, 90])
@pytest.mark.parametrize("offset,extra", [(1, 3), (3, 64), (8, 5)])
def test_strides_and_alignment(fq, kind, rows, offset, extra):
    """Rows that lie anywhere, inside a larger matrix full of NaN, give the bits of dense ones; so do weight planes."""
    rng = np.random.default_rng(9)
    n, k = 45, 176
    planes = weight(rng, "nvfp4", n, k)
    dense = handle(fq, "nvfp4", planes)
    moved = []
    for p in planes[:2]:
        buf = torch.zeros(p.size + 64, dtype=torch.uint8, device="cuda")
        at = buf[offset:offset + p.size].view(p.shape)
        at.copy_(torch.from_numpy(p))
        moved.append(at)
    odd = fq.Fp4Weight("nvfp4", *moved, dense.global_scale)
    for cols, call in ((k, fq.fp4_linear), (n, fq.fp4_linear_backward)):
        x, _, _ = activations(rng, fq, kind, rows, cols)
        wide = torch.full((rows * (cols + extra) + offset + 64,), float("nan"), dtype=x.dtype, device="cuda")
        y = wide[offset:offset + rows * (cols + extra)].view(rows, cols + extra)[:, :cols]
        y.copy_(x)
        assert torch.equal(call(x, dense), call(y, odd))
    x, _, _ = activations(rng, fq, kind, 1, k)
    same = x.expand(rows, k)
    assert torch.equal(fq.fp4_linear(same, dense), fq.fp4_linear(same.contiguous(), dense))


@pytest.mark.parametrize("rows", [5, 70])
def test_nothing_is_written_past_the_ends(fq, rows):
    """Outputs inside a larger buffer leave what is around them."""
    rng = np.random.default_rng(4)
    n, k = 38, 80
    w = handle(fq, "nvfp4", weight(rng, "nvfp4", n, k))
    x, _, _ = activations(rng, fq, "bf16", rows, k)
    dy, _, _ = activations(rng, fq, "bf16", rows, n)

    def around(call, shape, dtype):
        size = int(np.prod(shape))
        buf = torch.full((size + 512,), 77.0, device="cuda").to(dtype)
        call(buf[256:256 + size].view(shape))
        torch.cuda.synchronize()
        assert torch.all(buf[:256] == 77) and torch.all(buf[256 + size:] == 77)

    around(lambda o: fq.fp4_linear(x, w, out=o), (rows, n), torch.bfloat16)
    around(lambda o: fq.fp4_linear(x, w, out=o, out_dtype=torch.float32), (rows, n), torch.float32)
    around(lambda o: fq.fp4_gated(x, w, out=o), (rows, n // 2), torch.bfloat16)
    around(lambda o: fq.fp4_linear_backward(dy, w, out=o), (rows, k), torch.bfloat16)
    for d in (7, 100, 2050):
        s = torch.randn(rows, d, device="cuda").bfloat16()
        around(lambda o: fq.rms_norm(s, torch.ones(d, device="cuda"), out=o), (rows, d), torch.bfloat16)
        around(lambda o: fq.rms_norm(s, torch.ones(d, device="cuda"), residual=s, summed=o), (rows, d), torch.bfloat16)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("d", [96, 4096, 9000])
def test_residual_stream_in_place(fq, kind, d):
    x, res = (torch.randn(9, d, device="cuda").to(DT[kind]) for _ in range(2))
    w = torch.rand(d, device="cuda").to(DT[kind])
    want = fq.rms_norm(x, w, residual=res)
    for target in (0, 1):
        a, b = x.clone(), res.clone()
        got = fq.rms_norm(a, w, residual=b, summed=(a, b)[target])
        assert got.summed is (a, b)[target]
        assert torch.equal(got.out, want.out) and torch.equal(got.summed, want.summed)
        assert torch.equal((b, a)[target], (res, x)[target])


def test_calls_repeat_bit_for_bit(fq):
    rng = np.random.default_rng(6)
    w = handle(fq, "nvfp4", weight(rng, "nvfp4", 300, 4096))
    for rows in (1, 60, 200):
        x, _, _ = activations(rng, fq, "bf16", rows, 4096)
        dy, _, _ = activations(rng, fq, "f32", rows, 300)
        first = fq.fp4_linear(x, w), fq.fp4_gated(x, w), fq.fp4_linear_backward(dy, w)
        for _ in range(5):
            again = fq.fp4_linear(x, w), fq.fp4_gated(x, w), fq.fp4_linear_backward(dy, w)
            assert all(torch.equal(a, b) for a, b in zip(first, again))


def block(fq, x, res, norm, up, down, quantize):
    """A feed-forward block: norm, gated products, product back, on the residual stream."""
    r = fq.rms_norm(x, norm, residual=res, quantize=quantize)
    return r.summed, fq.fp4_linear(fq.fp4_gated(r.out, up), down)


def make_block(fq, rng, d, f, rows):
    x, res = (torch.from_numpy(rng.standard_normal((rows, d))).bfloat16().cuda() for _ in range(2))
    norm = torch.from_numpy(1 + 0.2 * rng.standard_normal(d)).bfloat16().cuda()
    up = fq.fp4_weight(fq.quantize_nvfp4(torch.from_numpy(rng.standard_normal((2 * f, d)) / d ** 0.5).float().cuda()))
    down = fq.fp4_weight(fq.quantize_mxfp4(torch.from_numpy(rng.standard_normal((d, f)) / f ** 0.5).bfloat16().cuda()))
    return x, res, norm, up, down


def dense(fq, w):
    return fq.dequantize(w.format, w.codes, w.scales, w.global_scale).double().cpu().numpy()


@pytest.mark.parametrize("rows", [1, 40, 130])
@pytest.mark.parametrize("quantize", [None, "mxfp8"])
def test_block(fq, rows, quantize):
    """The operators one after the other, over weights that the library quantized, against 64 bits from step to step."""
    rng = np.random.default_rng(rows)
    x, res, norm, up, down = make_block(fq, rng, 320, 448, rows)
    s, y = block(fq, x, res, norm, up, down, quantize)
    r = fq.rms_norm(x, norm, residual=res, quantize=quantize)
    a = fq.dequantize("mxfp8", *r.out) if quantize else r.out
    h = fq.fp4_gated(r.out, up)
    torch.cuda.synchronize()
    assert torch.equal(s, r.summed)
    wu, wd = dense(fq, up), dense(fq, down)
    av = a.double().cpu().numpy()
    p = av @ wu.T
    tol = sum_bound(np.abs(av) @ np.abs(wu).T, 320, 1)
    # (dequantize rounds an NVFP4 element once to fp32: 2^-24 of each product)
    tol = tol + 2.0 ** -24 * (np.abs(av) @ np.abs(wu).T)
    g, u, tg, tu = p[:, :448], p[:, 448:], tol[:, :448], tol[:, 448:]
    want = ffn_ref.gated(g, u)
    check(h, want, 1.1 * tg * (np.abs(u) + tu) + (np.abs(g) + tg) * tu + (2.0 ** -8 + 2.0 ** -21) * np.abs(want), "h")
    hv = h.double().cpu().numpy()
    want = hv @ wd.T
    check(y, want, sum_bound(np.abs(hv) @ np.abs(wd).T, 448, 1) + 2.0 ** -8 * np.abs(want), "y")


@pytest.mark.parametrize("rows", [3, 130])
@pytest.mark.parametrize("quantize", [None, "mxfp8"])
def test_block_captured(fq, rows, quantize):
    """Captured and replayed with other inputs in place, eager work between the replays; two graphs, one at a time and
    on two streams at once."""
    rng = np.random.default_rng(5)
    x, res, norm, up, down = make_block(fq, rng, 1024, 512, rows)
    dy = torch.randn(rows, 1024, device="cuda").bfloat16()
    block(fq, x, res, norm, up, down, quantize)
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        xs, rs = x.clone(), res.clone()
        with torch.cuda.graph(graph):
            out = block(fq, xs, rs, norm, up, down, quantize)
            back = fq.fp4_linear_backward(dy, down)
        graphs.append((graph, xs, rs, out, back))
    want_back = fq.fp4_linear_backward(dy, down)
    for step in range(4):
        new = [(torch.randn(rows, 1024, device="cuda").bfloat16(), torch.randn(rows, 1024, device="cuda").bfloat16())
               for _ in graphs]
        want = [block(fq, a, b, norm, up, down, quantize) for a, b in new]
        for (_, xs, rs, _, _), (a, b) in zip(graphs, new):
            xs.copy_(a)
            rs.copy_(b)
        torch.cuda.synchronize()
        if step % 2:
            streams = [torch.cuda.Stream() for _ in graphs]
            for (graph, *_), stream in zip(graphs, streams):
                with torch.cuda.stream(stream):
                    graph.replay()
        else:
            for graph, *_ in graphs:
                graph.replay()
        torch.cuda.synchronize()
        for (_, _, _, out, back), w in zip(graphs, want):
            assert torch.equal(out[0], w[0]) and torch.equal(out[1], w[1]) and torch.equal(back, want_back)


def test_training_step_captured(fq):
    """Forward and backward of norm and gated pair in one graph, while eager ones of the same tensors run."""
    rng = np.random.default_rng(7)
    rows, d, f = 150, 256, 160
    x, res, norm, up, _ = make_block(fq, rng, d, f, rows)
    dh = torch.randn(rows, f, device="cuda").bfloat16()

    def step():
        r = fq.rms_norm(x, norm, residual=res, return_rstd=True)
        h, p = fq.fp4_gated(r.out, up, return_products=True)
        dx, dp = fq.fp4_gated_backward(dh, p, up)
        return (h, dp) + fq.rms_norm_backward(dx, r.summed, norm, r.rstd, dsummed=dx)

    want = step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(3):
        graph.replay()
        eager = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) and torch.equal(c, b) for a, b, c in zip(got, want, eager))


def test_two_streams_at_once(fq):
    """Calls that share sums among workgroups, on two streams: each has memory of its own for them."""
    rng = np.random.default_rng(3)
    w = handle(fq, "mxfp4", weight(rng, "mxfp4", 256, 8192))
    xs = [activations(rng, fq, "bf16", 128, 8192)[0] for _ in range(2)]
    want = [fq.fp4_linear(x, w) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    got = [[], []]
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(fq.fp4_linear(xs[i], w))
    torch.cuda.synchronize()
    assert all(torch.equal(g, want[i]) for i in range(2) for g in got[i])


def test_out_dtypes_and_refusals(fq):
    rng = np.random.default_rng(2)
    n, k = 34, 96
    planes = weight(rng, "mxfp4", n, k)
    w = handle(fq, "mxfp4", planes)
    x, xv, _ = activations(rng, fq, "mxfp8", 5, k)
    got = fq.fp4_linear(x, w, out_dtype=torch.float32)
    assert got.dtype == torch.float32 and torch.equal(got.bfloat16(), fq.fp4_linear(x, w))
    b = torch.zeros(5, k, dtype=torch.bfloat16, device="cuda")
    for bad, error in (
            (lambda: fq.fp4_linear(b[:, 1:], w), ValueError),
            (lambda: fq.fp4_linear(b.half(), w), TypeError),
            (lambda: fq.fp4_linear(b.cpu(), w), ValueError),
            (lambda: fq.fp4_linear(b.t().contiguous().t(), w), ValueError),
            (lambda: fq.fp4_linear(b, w, bias=torch.zeros(n, device="cuda")), ValueError),
            (lambda: fq.fp4_linear(b, w, bias=torch.zeros(n + 1, device="cuda").bfloat16()), ValueError),
            (lambda: fq.fp4_linear(b, w, out=torch.zeros(5, n, device="cuda")), ValueError),
            (lambda: fq.fp4_linear(b, w, out_dtype=torch.float16), TypeError),
            (lambda: fq.fp4_linear(fq.Mx8Result(x.codes[:4], x.scales), w), ValueError),
            (lambda: fq.fp4_linear(fq.Mx8Result(x.codes[:, :64], x.scales), w), ValueError),
            (lambda: fq.fp4_linear(fq.Mx8Result(x.codes.view(torch.int8), x.scales), w), ValueError),
            (lambda: fq.fp4_linear_backward(b, w), ValueError),
            (lambda: fq.fp4_linear_backward(x, w), ValueError),
            (lambda: fq.fp4_gated(b, handle(fq, "mxfp4", weight(rng, "mxfp4", 5, k))), ValueError),
            (lambda: fq.fp4_gated(b, w, return_products=True, products_dtype=torch.float16), TypeError),
            (lambda: fq.fp4_gated_backward(b[:, :17], b[:, :34], w), ValueError),
            (lambda: fq.fp4_gated_backward(b[:, :17], None, w), TypeError),
            (lambda: fq.Fp4Weight("nvfp4", w.codes, w.scales, None), ValueError),
            (lambda: fq.Fp4Weight("mxfp4", w.codes, w.scales[:, :2]), ValueError),
            (lambda: fq.Fp4Weight("mxfp4", w.codes[:, :16], w.scales[:, :1]), ValueError),
            (lambda: fq.rms_norm(b, torch.ones(k - 1, device="cuda")), ValueError),
            (lambda: fq.rms_norm(b, torch.ones(k, device="cuda").half()), TypeError),
            (lambda: fq.rms_norm(b, torch.ones(k, device="cuda"), residual=b.float()), ValueError),
            (lambda: fq.rms_norm(b, torch.ones(k, device="cuda"), summed=b), ValueError),
            (lambda: fq.rms_norm(b, torch.ones(k, device="cuda"), quantize="nvfp4"), ValueError),
            (lambda: fq.rms_norm(b[:, :80], torch.ones(80, device="cuda"), quantize="mxfp8"), ValueError),
            (lambda: fq.rms_norm(b, torch.ones(k, device="cuda"), eps=-1.0), fq.Fp4qError),
            (lambda: fq.rms_norm(torch.zeros(1, 32800, device="cuda"), torch.ones(32800, device="cuda")), fq.Fp4qError),
            (lambda: fq.rms_norm_backward(b, b, torch.ones(k, device="cuda"), torch.ones(4, device="cuda")), ValueError),
            (lambda: fq.rms_norm_backward(b, b.float(), torch.ones(k, device="cuda"), torch.ones(5, device="cuda")),
             ValueError)):
        with pytest.raises(error):
            bad()


def test_same_buffers_again(fq):
    """rms_norm into a former result's buffers, MXFP8 and plain."""
    x = torch.randn(6, 128, device="cuda")
    w = torch.ones(128, device="cuda")
    first = fq.rms_norm(x, w, quantize="mxfp8").out
    again = fq.rms_norm(2 * x, w, quantize="mxfp8", out=first).out
    assert again.codes is first.codes
    assert all(torch.equal(a, b) for a, b in zip(again, fq.rms_norm(2 * x, w, quantize="mxfp8").out))


@pytest.mark.parametrize("policy", ["max6", "four_over_six"])
def test_weights_of_the_quantizers(fq, policy):
    """A product with the identity gives the reconstructed weight."""
    w = torch.randn(50, 64, device="cuda")
    eye = torch.eye(64, device="cuda")
    q = fq.quantize_nvfp4(w, policy=policy)
    want = fq.dequantize("nvfp4", q.codes, q.scales, q.global_scale)
    # (element and scale meet first, then the tensor scale: the reconstruction's own order)
    assert torch.equal(fq.fp4_linear(eye, fq.fp4_weight(q)), want.t())
    assert torch.equal(fq.fp4_linear_backward(torch.eye(50, device="cuda"), fq.fp4_weight(q)), want)
    m = fq.quantize_mxfp4(w)
    want = fq.dequantize("mxfp4", m.codes, m.scales)
    assert torch.equal(fq.fp4_linear(eye, fq.fp4_weight(m)), want.t())


def test_buffers_that_overlap(fq):
    """A caller's buffer that lies in what the call reads is refused; the norm may write over whole dense rows."""
    w = handle(fq, "mxfp4", weight(np.random.default_rng(3), "mxfp4", 64, 64))
    space = torch.zeros(40, 64, dtype=torch.bfloat16, device="cuda")
    x = space[:32]
    for out in (x, space[8:]):
        with pytest.raises(ValueError):
            fq.fp4_linear(x, w, out=out)
        with pytest.raises(ValueError):
            fq.fp4_linear_backward(x, w, out=out)
    with pytest.raises(ValueError):
        fq.fp4_linear(x[:1], w, bias=space[33], out=space[33:34])
    with pytest.raises(ValueError):
        fq.fp4_gated(x, w, out=space.view(-1)[64:64 + 32 * 32].view(32, 32))
    g = torch.ones(64, device="cuda")
    with pytest.raises(ValueError):
        fq.rms_norm(x, g, out=space[8:])
    with pytest.raises(ValueError):
        fq.rms_norm(x, g, residual=x.clone(), out=x, summed=x)
    with pytest.raises(ValueError):
        fq.rms_norm(x, g, residual=space[8:], summed=space[4:36])
    with pytest.raises(ValueError):
        fq.rms_norm(x, g, quantize="mxfp8", out=(x.view(torch.uint8).view(-1)[:2048].view(32, 64),
                                                 torch.empty(32, 2, dtype=torch.uint8, device="cuda")))
    a = torch.randn(300, 5000, device="cuda").bfloat16()
    b, gain = torch.randn_like(a), torch.randn(5000, device="cuda")
    want = fq.rms_norm(a, gain, residual=b)
    a2, b2 = a.clone(), b.clone()
    got = fq.rms_norm(a2, gain, residual=b2, out=a2, summed=b2)
    torch.cuda.synchronize()
    assert got.out.data_ptr() == a2.data_ptr() and torch.equal(a2, want.out) and torch.equal(b2, want.summed)


@pytest.mark.parametrize("rows", [3, 70, 2090])
def test_gradient_of_no_outputs(fq, rows):
    """A weight without rows: zeros, by each kernel."""
    for fmt, block in (("nvfp4", 16), ("mxfp4", 32)):
        g = torch.ones(1, device="cuda") if fmt == "nvfp4" else None
        none = fq.Fp4Weight(fmt, torch.zeros(0, 4128, dtype=torch.uint8, device="cuda"),
                            torch.zeros(0, 8256 // block, dtype=torch.uint8, device="cuda"), g)
        out = torch.full((rows, 8256), 5.0, dtype=torch.bfloat16, device="cuda")
        fq.fp4_linear_backward(torch.zeros(rows, 0, dtype=torch.bfloat16, device="cuda"), none, out=out)
        assert out.abs().max() == 0
