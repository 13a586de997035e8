"""How exact attention over the 4-bit cache is, measured against the outputs' own size: calls as a serving program
makes them (without the log-sum-exp, keys rotated), contexts so long that outputs are far smaller than the values.

Bounds, in root mean square over a call's outputs and relative to the outputs' own.  A bf16 output's own rounding is
computed (the 64-bit result rounded).  What comes on top of it may be at most 2^-11: weights are rounded by 2^-12
of themselves at most (one fp16 piece) with signs of their own, which moves an output by that part of the root of its
squared terms, about its own size; queries in two pieces move a score s by 2^-17 |s| at most (16 bits, bf16) with |s| to
2^4, another 2^-13.  An fp32 output: weights and queries of 22 bits or more, scores to 2^3, fp32 sums over up to 40000
terms with errors of either sign: 2^-22 (1 + 2^3) + 2^-24 * 200, doubled: 2^-15."""
import numpy as np
import pytest
import torch

import kv_ref
from test_kv_gpu import DT, Case, fq  # noqa: F401  (fq: the fixture)

pytestmark = pytest.mark.gpu

ON_TOP = {"bf16": 2.0 ** -11, "f32": 2.0 ** -15}
# (lengths, queries, query heads of 2 cache heads): few rows, more of them, many, long contexts
SHAPES = [([700, 301, 33], [1, 1, 1], 16), ([700, 301, 33], [3, 2, 4], 8), ([300, 87], [40, 33], 8),
          ([333, 210], [140, 70], 4), ([9001, 40000], [1, 1], 8)]


def rms(x):
    return float(np.sqrt(np.mean(np.square(x))))


def call(case, q, new, rotate, **kw):
    cu = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device="cuda")
    return case.fq.kv_cache_attention(q.cuda(), case.cache(), torch.from_numpy(case.table).cuda(),
                                      torch.tensor(case.lens, dtype=torch.int32, device="cuda"),
                                      cu_q=None if max(new) == 1 else cu, max_q=max(new),
                                      rotation="fwht128" if rotate else None, **kw)


def wanted(case, q, new, rotate):
    qd = kv_ref.rotate(q.double().numpy()) if rotate else q.double().numpy()
    at = np.concatenate([[0], np.cumsum(new)])
    return np.concatenate([kv_ref.attention(qd[at[b]:at[b + 1]], *case.tokens(b), case.dim ** -0.5)[0]
                           for b in range(len(new))])


@pytest.mark.parametrize("fmt,dim,rotate", [("nvfp4", 128, True), ("nvfp4", 128, False), ("nvfp4", 256, True),
                                            ("mxfp4", 128, True), ("mxfp4", 128, False), ("mxfp4", 256, False),
                                            ("nvfp4", 64, False), ("mxfp4", 96, False)])
@pytest.mark.parametrize("dtype,q_scale", [("bf16", 1.5), ("bf16", 5.0), ("f32", 1.5)])
@pytest.mark.parametrize("lens,new,q_heads", SHAPES)
def test_error_by_the_outputs_own_size(fq, fmt, dim, rotate, dtype, q_scale, lens, new, q_heads):  # noqa: F811
    case = Case(fq, fmt, dim, 2, lens, 48, seed=len(new) + dim)
    q = (q_scale * torch.from_numpy(case.rng.standard_normal((sum(new), q_heads, dim)))).to(DT[dtype])
    print("attention", fmt, dim, rotate, dtype, q_scale, lens, new, q_heads, flush=True)
    got = call(case, q, new, rotate).double().cpu().numpy()
    want = wanted(case, q, new, rotate)
    own = rms(torch.from_numpy(want).to(DT[dtype]).double().numpy() - want)
    error, bound = rms(got - want), (own ** 2 + (ON_TOP[dtype] * rms(want)) ** 2) ** 0.5
    assert error <= bound, "off by %g of the outputs, own rounding %g, bound %g" % tuple(
        x / rms(want) for x in (error, own, bound))


@pytest.mark.parametrize("fmt,dim,rotate", [("nvfp4", 128, True), ("nvfp4", 128, False), ("mxfp4", 128, True), ("mxfp4", 256, False)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("page", [32, 64])
@pytest.mark.parametrize("lens,new,q_heads", [SHAPES[0], SHAPES[1], ([20000], [1], 32), ([900] * 24, [1] * 24, 32)])
def test_error_with_pages_of_whole_tiles(fq, fmt, dim, rotate, dtype, page, lens, new, q_heads):  # noqa: F811
    """As above where a wave's 32 tokens lie in one page, up to 32 rows a cache head."""
    case = Case(fq, fmt, dim, 1 if len(lens) == 1 else 2, lens, page, seed=page + dim)
    q = (1.5 * torch.from_numpy(case.rng.standard_normal((sum(new), q_heads, dim)))).to(DT[dtype])
    print("attention", fmt, dim, rotate, dtype, page, lens, new, q_heads, flush=True)
    got = call(case, q, new, rotate).double().cpu().numpy()
    want = wanted(case, q, new, rotate)
    own = rms(torch.from_numpy(want).to(DT[dtype]).double().numpy() - want)
    error, bound = rms(got - want), (own ** 2 + (ON_TOP[dtype] * rms(want)) ** 2) ** 0.5
    assert error <= bound, "off by %g of the outputs, own rounding %g, bound %g" % tuple(
        x / rms(want) for x in (error, own, bound))


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("dim", [128, 256])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens,new,q_heads", SHAPES)
def test_log_sum_exps_leave_the_outputs_alone(fq, fmt, dim, dtype, lens, new, q_heads):  # noqa: F811
    """The same bits whether the log-sum-exp is asked for or not."""
    case = Case(fq, fmt, dim, 2, lens, 64, seed=3)
    q = torch.randn(sum(new), q_heads, dim).to(DT[dtype])
    print("attention", fmt, dim, dtype, lens, new, q_heads, flush=True)
    assert torch.equal(call(case, q, new, True), call(case, q, new, True, return_lse=True)[0])


# Scale bytes of MXFP4 values by 32-element block: those of fp16 numbers are 104 to 140
SPANS = {"low edge": [(100, 109)] * 4, "high edge": [(136, 145)] * 4, "far apart": [(20, 24), (122, 127), (60, 66), (180, 184)],
         "one block": [(122, 127)] * 4, "zeros": [(122, 127)] * 4}


@pytest.mark.parametrize("spans", list(SPANS), ids=str)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens,new,q_heads,page", [([700, 301, 33], [1, 1, 1], 8, 32), ([300, 87], [40, 33], 8, 48),
                                                   ([333, 2100], [140, 70], 4, 16), ([500, 90], [200, 90], 12, 64)])
def test_values_of_any_scale(fq, spans, dtype, lens, new, q_heads, page):  # noqa: F811
    """MXFP4 value blocks at the edges of fp16's range and far outside: as exact as others, each block measured by
    its own outputs.  One block alone outside of it, far back in one sequence; blocks of zeros with any scale."""
    case = Case(fq, "mxfp4", 128, 2, lens, page, seed=21)
    case.planes[3][:] = np.stack([case.rng.integers(*s, case.planes[3].shape[:3]) for s in SPANS[spans]], -1)
    if spans == "one block":
        t = lens[0] // 3
        case.planes[3][case.table[0, t // page], 1, t % page, 2] = 150
    if spans == "zeros":
        rows = case.rng.random(case.planes[3].shape) < 0.3
        case.planes[3][rows] = case.rng.integers(0, 253, int(rows.sum()))
        codes = case.planes[2].reshape(*rows.shape, 16)
        codes[rows] &= 0x88
    q = (1.5 * torch.from_numpy(case.rng.standard_normal((sum(new), q_heads, 128)))).to(DT[dtype])
    print("attention", spans, dtype, lens, new, q_heads, page, flush=True)
    got = call(case, q, new, False).double().cpu().numpy().reshape(-1, 4, 32)
    want = wanted(case, q, new, False).reshape(-1, 4, 32)
    for j in range(4):
        g, w = got[:, j], want[:, j]
        own = rms(torch.from_numpy(w).to(DT[dtype]).double().numpy() - w)
        error, bound = rms(g - w), (own ** 2 + (ON_TOP[dtype] * rms(w)) ** 2) ** 0.5
        assert error <= bound, "block %d off by %g of the outputs, own rounding %g, bound %g" % (
            j, error / rms(w), own / rms(w), bound / rms(w))


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("queries", [1, 48])
@pytest.mark.parametrize("score", [12.0625, 14.125, 20.0])
def test_many_small_weights_beside_a_large_one(fq, fmt, queries, score):  # noqa: F811
    """One token scores `score` and has values of zero, 131070 score nothing and have ones: an output is n w / (1 + n w)
    with w = exp(-score).  All of their weights are rounded alike.  fp32: the exponents, to 32 in powers of two, are
    rounded by 2^-20, weights to 22 bits down to 2^-43 of the largest, sums of a lane's hundreds of terms by 2^-24 each:
    2^-19 of the output and 2^17 x 2^-43 of the values, doubled."""
    n, dim, page = 131071, 64, 64
    pages = -(-n // page)
    cache = fq.kv_cache(pages, page, 1, dim, format=fmt)
    one = 0x38 if fmt == "nvfp4" else 127
    cache.k_scales.fill_(one)
    cache.v_scales.fill_(one)
    cache.v_codes.fill_(0x22)                 # ones
    cache.k_codes[0, 0, 0, 0] = 0x02          # the first token's first element
    cache.v_codes[0, 0, 0] = 0
    q = torch.zeros(queries, 4, dim, device="cuda")
    q[:, :, 0] = score
    print("attention", fmt, queries, score, flush=True)
    out = fq.kv_cache_attention(q, cache, torch.arange(pages, dtype=torch.int32, device="cuda")[None],
                                torch.tensor([n], dtype=torch.int32, device="cuda"),
                                cu_q=torch.tensor([0, queries], dtype=torch.int32, device="cuda"), max_q=queries, scale=1.0)
    alike = (n - queries + torch.arange(queries, dtype=torch.float64))[:, None, None] * np.exp(-score)
    want = alike / (1 + alike)
    error = (out.double().cpu() - want).abs()
    print("error", float((error / want).max()), "of the output")
    assert bool((error <= 2.0 ** -18 * want + 2.0 ** -25).all())


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("queries", [1, 3, 48])
@pytest.mark.parametrize("score", [12.0625, 14.125])
@pytest.mark.parametrize("n", [1000, 70000])
def test_a_large_weight_among_few_small_ones(fq, fmt, queries, score, n):  # noqa: F811
    """As above with a large one every 64 tokens, so that every part of a context that is summed by itself has one."""
    dim, page = 64, 64
    pages = -(-n // page)
    cache = fq.kv_cache(pages, page, 1, dim, format=fmt)
    one = 0x38 if fmt == "nvfp4" else 127
    cache.k_scales.fill_(one)
    cache.v_scales.fill_(one)
    cache.v_codes.fill_(0x22)
    cache.k_codes[:, 0, 5, 0] = 0x02
    cache.v_codes[:, 0, 5] = 0
    q = torch.zeros(queries, 4, dim, device="cuda")
    q[:, :, 0] = score
    print("attention", fmt, queries, score, n, flush=True)
    out = fq.kv_cache_attention(q, cache, torch.arange(pages, dtype=torch.int32, device="cuda")[None],
                                torch.tensor([n], dtype=torch.int32, device="cuda"),
                                cu_q=torch.tensor([0, queries], dtype=torch.int32, device="cuda"), max_q=queries, scale=1.0)
    seen = n - queries + 1 + torch.arange(queries, dtype=torch.float64)
    large = torch.floor((seen + 58) / 64)
    small = ((seen - large) * np.exp(-score))[:, None, None]
    want = small / (large[:, None, None] + small)
    error = (out.double().cpu() - want).abs()
    print("error", float((error / want).max()), "of the output")
    assert bool((error <= 2.0 ** -18 * want + 2.0 ** -25 * want.new_tensor(64 / 2 ** 17)).all())
