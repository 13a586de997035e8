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
