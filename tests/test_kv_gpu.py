"""The paged 4-bit key/value cache on the GPU against 64-bit arithmetic and
the library's own quantizers."""
import math

import numpy as np
import pytest
import torch

import kv_ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import fp4_block_scaled_row_amd as m
    m.load()
    return m


DT = {"f32": torch.float32, "bf16": torch.bfloat16}
# Tolerances, set from the kernels' arithmetic (relative to a row's largest |v| seen, which bounds |out|):
#   bf16 output: its own rounding 2^-9 of the result; the weights rounded once, 2^-9 (bf16) at most and in the same
#   direction at worst: 2^-8 in all, doubled for fp32 sums over thousands of terms.
#   fp32 output: weights in two pieces 2^-17, scores exact to about 2^-21 |s| with |s| below 2^5: 2^-16, doubled twice.
# lse: the scores' error alone, 2^-21 * 2^5 relative to at most 2^5: 2^-14 absolute.
OUT_TOL = {"bf16": 2.0 ** -7, "f32": 2.0 ** -14}
LSE_TOL = 2.0 ** -13


class Case:
    """A random cache with page tables, and its planes on the CPU."""

    def __init__(self, fq, fmt, dim, heads, lens, page, seed, layout="hnd", spare=3, g=(0.25, 0.375)):
        rng = np.random.default_rng(seed)
        per = max(1, max(-(-n // page) for n in lens))
        pages = len(lens) * per + spare
        self.fmt, self.dim, self.heads, self.page, self.lens = fmt, dim, heads, page, lens
        self.table = rng.permutation(pages)[:len(lens) * per].reshape(len(lens), per).astype(np.int32)
        span = (0x28, 0x41) if fmt == "nvfp4" else (122, 127)
        shape = (pages, heads, page)
        self.planes = []
        for _ in range(2):
            self.planes.append(rng.integers(0, 256, shape + (dim // 2,), dtype=np.uint8))
            self.planes.append(rng.integers(*span, shape + (dim // kv_ref.BLOCK[fmt],), dtype=np.uint8))
        self.g = g
        self.rng = rng
        self.layout = layout
        self.fq = fq

    def cache(self):
        def put(x):
            t = torch.from_numpy(x).cuda()
            if self.layout == "nhd":        # tokens before heads in memory
                t = t.transpose(1, 2).contiguous().transpose(1, 2)
            return t
        return self.fq.KvCache(self.fmt, *(put(x) for x in self.planes),
                               torch.tensor([self.g[0]], device="cuda"), torch.tensor([self.g[1]], device="cuda"))

    def tokens(self, b):
        kc, ks, vc, vs = self.planes
        n = self.lens[b]
        return (kv_ref.tokens_of(self.fmt, kc, ks, self.g[0], self.table[b], n, self.page),
                kv_ref.tokens_of(self.fmt, vc, vs, self.g[1], self.table[b], n, self.page))


def check_attention(case, new, q_heads, dtype, *, causal=True, window=0, rotate=False, scale=None, max_q=None,
                    q_scale=1.5, **kw):
    fq = case.fq
    total = sum(new)
    q = (q_scale * torch.from_numpy(case.rng.standard_normal((total, q_heads, case.dim)))).to(DT[dtype])
    cu = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device="cuda")
    one = all(m == 1 for m in new) and max_q is None
    print("attention", case.fmt, case.dim, case.heads, q_heads, case.lens, new, dtype, causal, window, rotate, flush=True)
    out, lse = fq.kv_cache_attention(q.cuda(), case.cache(), torch.from_numpy(case.table).cuda(),
                                     torch.tensor(case.lens, dtype=torch.int32, device="cuda"),
                                     cu_q=None if one else cu, max_q=max_q or max(new), scale=scale, causal=causal,
                                     window=window, rotation="fwht128" if rotate else None, return_lse=True, **kw)
    torch.cuda.synchronize()
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    qd = q.double().numpy()
    if rotate:
        qd = kv_ref.rotate(qd)
    at = 0
    for b, m in enumerate(new):
        k, v = case.tokens(b)
        want, want_lse = kv_ref.attention(qd[at:at + m], k, v, case.dim ** -0.5 if scale is None else scale, causal,
                                          window)
        got, got_lse = out[at:at + m], lse[at:at + m]
        assert np.array_equal(np.isnan(got), np.isnan(want)), "sequence %d: NaN in other places" % b
        assert np.array_equal(np.isnan(got_lse), np.isnan(want_lse))
        fine = np.isfinite(want)
        bound = OUT_TOL[dtype] * (np.nanmax(np.abs(v), initial=0.0) if v.size else 1.0)
        err = np.max(np.abs(got - want)[fine], initial=0.0)
        assert err <= bound, "sequence %d (n=%d, m=%d): off by %g, bound %g" % (b, case.lens[b], m, err, bound)
        empty = np.isneginf(want_lse)
        assert np.array_equal(empty, np.isneginf(got_lse))
        real = np.isfinite(want_lse)
        err = np.max(np.abs(got_lse - want_lse)[real], initial=0.0)
        assert err <= LSE_TOL, "sequence %d: lse off by %g" % (b, err)
        assert not np.any(got[empty]), "a row that sees nothing is not zero"
        at += m
    return out


# one query each: lengths around every tile edge, none, one, several workgroups' worth
@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("dim", [64, 96, 128, 256])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_decode_lengths(fq, fmt, dim, dtype):
    lens = [0, 1, 2, 15, 16, 17, 31, 32, 33, 127, 128, 129, 300, 1025]
    check_attention(Case(fq, fmt, dim, 2, lens, 24, seed=dim), [1] * len(lens), 8, dtype)


@pytest.mark.parametrize("fmt,dim,rotate", [("nvfp4", 128, True), ("nvfp4", 256, True), ("mxfp4", 128, True),
                                            ("mxfp4", 64, False)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("q_heads,heads", [(3, 3), (5, 1), (16, 1), (17, 1), (40, 2), (64, 1), (80, 1)])
def test_decode_groups(fq, fmt, dim, rotate, dtype, q_heads, heads):
    lens = [257, 40, 0, 513]
    check_attention(Case(fq, fmt, dim, heads, lens, 16, seed=q_heads), [1] * 4, q_heads, dtype, rotate=rotate)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("window", [0, 1, 2, 3, 31, 100])
@pytest.mark.parametrize("new", [[2, 1, 2, 1], [5, 3, 7, 4], [33, 1, 20, 64]])
def test_queries_and_windows(fq, fmt, dtype, window, new):
    lens = [200, 3, 131, 260]       # the second: fewer tokens than queries in two of the cases
    check_attention(Case(fq, fmt, 128, 1, lens, 128, seed=window), new, 8, dtype, window=window)


@pytest.mark.parametrize("fmt,dim", [("nvfp4", 128), ("mxfp4", 128), ("nvfp4", 64), ("mxfp4", 256), ("nvfp4", 96)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("q_heads,heads", [(2, 2), (5, 1)])
def test_long_queries(fq, fmt, dim, dtype, causal, q_heads, heads):
    case = Case(fq, fmt, dim, heads, [150, 0, 331, 64, 40], 40, seed=9)
    check_attention(case, [150, 0, 131, 64, 70], q_heads, dtype, causal=causal)


# ---- writing and reading


def kv_rows(rng, tokens, heads, dim, dtype, kind):
    """Keys or values as a projection leaves them, or with everything that can go wrong in them."""
    x = rng.standard_normal((tokens, heads, dim)) * np.exp2(rng.integers(-3, 3, (1, heads, dim)))
    if kind == "wild":
        x *= np.exp2(rng.integers(-60, 40, (tokens, heads, dim // 32)).repeat(32, -1).astype(float))
        flat = x.reshape(-1, 16)
        for i, v in enumerate((0.0, -0.0, np.inf, -np.inf, np.nan, 1e-45, -1e-45, 3e38)):
            flat[i::37, i] = v
        flat[5::41] = 0.0
        flat[9::43] = -0.0
    return torch.from_numpy(x.astype(np.float32)).to(DT[dtype])


def strided(x, how):
    """The same values with other strides: a slice of a wider matrix, heads before tokens."""
    if how == "slice":
        wide = torch.full((x.shape[0], x.shape[1], x.shape[2] + 32), float("nan"), dtype=x.dtype, device=x.device)
        wide[:, :, 16:16 + x.shape[2]] = x
        return wide[:, :, 16:16 + x.shape[2]]
    if how == "heads":
        return x.transpose(0, 1).contiguous().transpose(0, 1)
    return x


def bits(t):
    return t.contiguous().view(torch.uint8)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("heads,dim,page,rotate", [(2, 128, 16, True), (1, 256, 24, True), (5, 96, 7, False),
                                                   (3, 64, 1, False), (1, 32, 40, False), (2, 1024, 5, True)])
@pytest.mark.parametrize("kind,g", [("plain", (2.0 ** -8, 2.0 ** -9)), ("plain", (0.00321, 0.0123)),
                                    ("wild", (2.0 ** -8, 0.00077)), ("wild", (1e-38, 2.0 ** 101)),
                                    ("wild", (2.0 ** -90, 2.0 ** 80))])
@pytest.mark.parametrize("layout,how", [("hnd", "dense"), ("nhd", "slice"), ("hnd", "heads")])
def test_write_and_read(fq, fmt, dtype, heads, dim, page, rotate, kind, g, layout, how):
    """The cache's bytes are the library's own quantizers' bytes, in the slots asked for and nowhere else; reading
    gives the library's own dequantized values."""
    if fmt == "mxfp4" and g != (2.0 ** -8, 2.0 ** -9) and kind == "plain":
        pytest.skip("no tensor scale")
    rng = np.random.default_rng(heads * dim + page)
    tokens, pages = 61, 61 // page + 4
    k, v = kv_rows(rng, tokens, heads, dim, dtype, kind).cuda(), kv_rows(rng, tokens, heads, dim, dtype, kind).cuda()
    block = kv_ref.BLOCK[fmt]
    planes = []
    for w in (dim // 2, dim // block, dim // 2, dim // block):
        shape = (pages, heads, page, w) if layout == "hnd" else (pages, page, heads, w)
        t = torch.full(shape, 0xA5, dtype=torch.uint8, device="cuda")
        planes.append(t if layout == "hnd" else t.transpose(1, 2))
    (k_amax, kg), (v_amax, vg) = (amax_of(x) for x in g)
    kg, vg = (torch.tensor([x], dtype=torch.float32, device="cuda") for x in (kg, vg))
    cache = fq.KvCache(fmt, *planes, kg, vg)
    slots = rng.permutation(pages * page)[:tokens].astype(np.int64)
    slots[[3, 17]] = -1, pages * page + 5           # skipped
    print("write", fmt, dtype, heads, dim, page, rotate, kind, g, layout, how, flush=True)
    fq.kv_cache_write(cache, strided(k, how), strided(v, how), torch.from_numpy(slots).cuda(),
                      rotation="fwht128" if rotate else None)

    def reference(x, amax, g, rotate):
        x = x.reshape(-1, dim)
        if rotate:
            x = fq.fwht(x, transform_size=128)
        if fmt == "mxfp4":
            r = fq.quantize_mxfp4(x)
            return r.codes.cpu().numpy(), r.scales.cpu().numpy()
        r = nv_with_scale(fq, x, amax)
        assert r.global_scale.item() == g.item()
        return r.codes.cpu().numpy(), r.scales.cpu().numpy()

    kc, ks = reference(k, k_amax, kg, rotate)
    vc, vs = reference(v, v_amax, vg, False)
    for plane, want, width in zip(planes, (kc, ks, vc, vs), (dim // 2, dim // block) * 2):
        got = plane.permute(0, 2, 1, 3).reshape(pages * page, heads, width).cpu().numpy()
        expect = np.full_like(got, 0xA5)
        ok = (slots >= 0) & (slots < pages * page)
        expect[slots[ok]] = want.reshape(tokens, heads, width)[ok]
        assert np.array_equal(got, expect)

    # read back tokens of two sequences: the first 40 slots' worth from position 1 on, and the rest
    table = torch.arange(2 * pages, dtype=torch.int32, device="cuda").reshape(2, pages) % pages
    n0 = min(40, pages * page - 1)
    cu = torch.tensor([0, n0, n0 + 9], dtype=torch.int32, device="cuda")
    starts = torch.tensor([1, 0], dtype=torch.int32, device="cuda")
    for out_dtype in (torch.bfloat16, torch.float32):
        got = fq.kv_cache_read(cache, table, cu, total=n0 + 12, starts=starts, rotation="fwht128" if rotate else None,
                               out_dtype=out_dtype)
        for x, c, s, gs, rot in ((got[0], planes[0], planes[1], kg, rotate), (got[1], planes[2], planes[3], vg, False)):
            c = c.permute(0, 2, 1, 3).reshape(pages * page, -1, dim // 2)
            s = s.permute(0, 2, 1, 3).reshape(pages * page, -1, dim // block)
            rows = torch.cat([torch.arange(1, 1 + n0), torch.arange(9)]).cuda()
            want = fq.dequantize(fmt, c[rows].reshape(-1, dim // 2).contiguous(),
                                 s[rows].reshape(-1, dim // block).contiguous(), gs if fmt == "nvfp4" else None,
                                 out_dtype=torch.float32 if rot else out_dtype)
            if rot:
                want = fq.fwht(want, transform_size=128).to(out_dtype)
            want = want.reshape(-1, heads, dim)
            a, b = x[:n0 + 9], want
            same = (a == b) | (a.isnan() & b.isnan())
            assert bool(same.all()), "values differ in %d places" % int((~same).sum())
            assert not bool(x[n0 + 9:].any()), "rows without a token are not zero"


def amax_of(g):
    """An amax for a tensor scale of about g (quantize_nvfp4 takes the amax and divides it by 2688), and the scale
    that it stands for: not every fp32 number is such a quotient."""
    amax = np.float32(np.float64(np.float32(g)) * 2688.0)
    return amax, float(np.float32(np.float64(amax) / 2688.0))


def nv_with_scale(fq, x, amax):
    return fq.quantize_nvfp4(x, global_amax=torch.tensor([amax], dtype=torch.float32, device=x.device))


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_write_and_read_nothing(fq, fmt):
    cache = fq.kv_cache(4, 16, 2, 64, format=fmt)
    none = torch.zeros((0, 2, 64), dtype=torch.bfloat16, device="cuda")
    fq.kv_cache_write(cache, none, none, torch.zeros(0, dtype=torch.int64, device="cuda"))
    table = torch.zeros((1, 4), dtype=torch.int32, device="cuda")
    k, v = fq.kv_cache_read(cache, table, torch.zeros(2, dtype=torch.int32, device="cuda"), total=0)
    assert k.shape == v.shape == (0, 2, 64)
    out = fq.kv_cache_attention(torch.zeros((0, 4, 64), dtype=torch.bfloat16, device="cuda"), cache, table[:0],
                                torch.zeros(0, dtype=torch.int32, device="cuda"))
    assert out.shape == (0, 4, 64)


def test_read_one_side_only(fq):
    case = Case(fq, "nvfp4", 64, 2, [50], 16, seed=3)
    cache, table = case.cache(), torch.from_numpy(case.table).cuda()
    cu = torch.tensor([0, 50], dtype=torch.int32, device="cuda")
    both = fq.kv_cache_read(cache, table, cu, total=50)
    for side in (0, 1):
        buf = torch.empty_like(both[0])
        out = fq.kv_cache_read(cache, table, cu, total=50, out=(buf, None) if side == 0 else (None, buf))
        assert out[side] is buf and torch.equal(buf, both[side])
