"""The paged 4-bit key/value cache where it can go wrong: masked garbage, rows
that see nothing, pages that are not there, strides, large planes, streams,
graphs, reused workspaces, and what it refuses."""
import math

import numpy as np
import pytest
import torch

import kv_ref
from test_kv_gpu import Case, check_attention, fq  # noqa: F401  (fq: the fixture)

pytestmark = pytest.mark.gpu

NAN_SCALE = {"nvfp4": (0x7F, 0xFF), "mxfp4": (0xFF, 0xFF)}


class Planted:
    """A generator whose normal numbers are edited before use."""

    def __init__(self, rng, edit):
        self.rng, self.edit = rng, edit

    def standard_normal(self, shape):
        return self.edit(self.rng.standard_normal(shape))


def scale_row(case, plane, b, t):
    """The scale bytes of token t of sequence b, [heads, blocks], to be written."""
    return case.planes[plane][case.table[b, t // case.page], :, t % case.page]


# (queries a sequence, query heads of 2 cache heads): few-row and many-row kernels
SHAPES = [([1, 1, 1], 8), ([3, 2, 4], 8), ([40, 7, 20], 8), ([140, 33, 60], 6)]


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("dim,dtype", [(128, "bf16"), (128, "f32"), (64, "bf16"), (96, "bf16"), (256, "f32")])
@pytest.mark.parametrize("new,q_heads", SHAPES)
def test_masked_garbage(fq, fmt, dim, dtype, new, q_heads):  # noqa: F811
    """NaN scales, the largest scales and all codes behind a sequence's length, before its windows, and in every page
    that no table lists, never reach an output."""
    lens, window = [150, 37, 400], 20
    case = Case(fq, fmt, dim, 2, lens, 24, seed=dim)
    spare = np.setdiff1d(np.arange(case.planes[0].shape[0]), case.table)
    for i, plane in enumerate((1, 3)):
        bad = np.array([NAN_SCALE[fmt][0], NAN_SCALE[fmt][1], 254, 253], dtype=np.uint8)
        case.planes[plane][spare] = bad[i]
        for b, n in enumerate(lens):
            for t in range(n, case.table.shape[1] * case.page):
                scale_row(case, plane, b, t)[:] = bad[(t + i) % 4]
            for t in range(0, n - new[b] - window + 1):     # (NaN alone: the bound goes by the others)
                scale_row(case, plane, b, t)[:] = bad[t % 2]
    check_attention(case, new, q_heads, dtype, window=window)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("dim,dtype", [(128, "bf16"), (96, "f32"), (256, "bf16")])
@pytest.mark.parametrize("new,q_heads", SHAPES)
@pytest.mark.parametrize("plane", [1, 3])
@pytest.mark.parametrize("window", [0, 50])
def test_not_a_number_reaches_its_readers_only(fq, fmt, dim, dtype, new, q_heads, plane, window):  # noqa: F811
    """A NaN block among the last tokens and one far back: a key's makes the rows that see it NaN, a value's the
    block's elements of those rows."""
    lens = [150, 37, 400]
    case = Case(fq, fmt, dim, 2, lens, 24, seed=dim + plane)
    scale_row(case, plane, 0, 148)[0, 1] = NAN_SCALE[fmt][0]
    scale_row(case, plane, 0, 11)[1, 0] = NAN_SCALE[fmt][1]
    scale_row(case, plane, 1, 36)[1, 0] = NAN_SCALE[fmt][0]
    scale_row(case, plane, 2, 380)[0, 0] = NAN_SCALE[fmt][1]
    check_attention(case, new, q_heads, dtype, window=window)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("new,q_heads", SHAPES)
@pytest.mark.parametrize("rotate", [False, True])
def test_queries_that_are_not_numbers(fq, fmt, dtype, new, q_heads, rotate):  # noqa: F811
    """They spoil their own rows; rows of zeros average."""
    case = Case(fq, fmt, 128, 2, [150, 90, 400], 24, seed=7)

    def edit(q):
        q[0, 0, 5] = np.nan
        q[-1, -1, 7] = np.inf
        q[0, 1] = 0.0
        q[-1, 0] = 0.0
        return q

    case.rng = Planted(case.rng, edit)
    check_attention(case, new, q_heads, dtype, rotate=rotate)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("new,q_heads", SHAPES)
@pytest.mark.parametrize("scale,g", [(0.0, (0.25, 0.375)), (-0.0884, (0.25, 0.375)), (0.0884, (1e-30, 1e-12))])
def test_scales_and_small_tensor_scales(fq, fmt, dtype, new, q_heads, scale, g):  # noqa: F811
    """A factor of nothing (0 as such, or zero rows by a small tensor scale) keeps masked tokens out."""
    case = Case(fq, fmt, 128, 2, [150, 37, 400], 24, seed=8, g=g)

    def edit(q):
        q[0, 0] = 0.0
        q[-1] = 0.0
        return q

    case.rng = Planted(case.rng, edit)
    check_attention(case, new, q_heads, dtype, scale=scale)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("new,q_heads", SHAPES)
@pytest.mark.parametrize("page", [1, 24, 128])
def test_pages_that_are_not_there(fq, fmt, new, q_heads, page):  # noqa: F811
    """Table entries outside the cache count as tokens of zeros, for attention and for reading."""
    lens = [150, 37, 400]
    case = Case(fq, fmt, 128, 2, lens, page, seed=page)
    pages = case.planes[0].shape[0]
    for i, wrong in enumerate((-1, pages, 2 ** 31 - 1, -2 ** 31)):
        case.table[i % 3, (5 * i + 1) % case.table.shape[1]] = wrong
    case.table[1, 0] = -7
    check_attention(case, new, q_heads, "bf16")
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    got = fq.kv_cache_read(case.cache(), torch.from_numpy(case.table).cuda(), cu, total=sum(lens),
                           out_dtype=torch.float32)
    want = [case.tokens(b) for b in range(3)]
    for side in (0, 1):
        w = np.concatenate([x[side] for x in want])
        assert np.array_equal(got[side].double().cpu().numpy(), w.astype(np.float32).astype(np.float64))


@pytest.mark.parametrize("fmt,dim", [("nvfp4", 128), ("mxfp4", 128), ("nvfp4", 96), ("mxfp4", 64), ("nvfp4", 256)])
@pytest.mark.parametrize("new,q_heads", SHAPES)
@pytest.mark.parametrize("page", [24, 64])
def test_layouts_and_strides(fq, fmt, dim, new, q_heads, page):  # noqa: F811
    """Tokens before heads in memory, queries that are a slice of a wider matrix, a table that is one of another:
    the same bits."""
    lens = [150, 37, 400]
    case = Case(fq, fmt, dim, 2, lens, page, seed=4)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device="cuda")
    q = torch.randn(sum(new), q_heads, dim, device="cuda").bfloat16()
    wide = torch.full((sum(new), q_heads + 3, dim + 8), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, 1:1 + q_heads, 8:] = q
    table = torch.from_numpy(case.table).cuda()
    wide_table = torch.full((3, table.shape[1] + 5), -1, dtype=torch.int32, device="cuda")
    wide_table[:, :table.shape[1]] = table
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    outs = []
    for layout, qq, tt in (("hnd", q, table), ("nhd", wide[:, 1:1 + q_heads, 8:], wide_table),
                           ("nhd", q.transpose(0, 1).contiguous().transpose(0, 1), wide_table[:, :table.shape[1]])):
        case.layout = layout
        outs.append(fq.kv_cache_attention(qq, case.cache(), tt, n, cu_q=cu, max_q=max(new), return_lse=True))
    for out, lse in outs[1:]:
        assert torch.equal(out, outs[0][0]) and torch.equal(lse, outs[0][1])


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("new,q_heads", [([1, 1], 8), ([40, 7], 8), ([150, 33], 4)])
@pytest.mark.parametrize("page", [24, 32])
def test_large_planes(fq, fmt, new, q_heads, page):  # noqa: F811
    """Offsets past 32 bits: pages 2^30 bytes of codes apart, in planes of 6 GiB."""
    dim, heads, lens, pages = 128, 2, [page + 5, 3 * page], 6
    block = kv_ref.BLOCK[fmt]
    rng = np.random.default_rng(5)
    small, large = [], []
    for width in (dim // 2, dim // block) * 2:
        apart = 2 ** 30 if width == dim // 2 else 2 ** 30 - 4096
        buf = torch.empty(apart * (pages - 1) + page * heads * width, dtype=torch.uint8, device="cuda")
        x = buf.as_strided((pages, heads, page, width), (apart, page * width, width, 1))
        lo, hi = (0, 256) if width == dim // 2 else (120, 126) if fmt == "mxfp4" else (0x28, 0x40)
        y = torch.from_numpy(rng.integers(lo, hi, (pages, heads, page, width), dtype=np.uint8)).cuda()
        x.copy_(y)
        small.append(y)
        large.append(x)
    g = torch.full((1,), 0.25, device="cuda")
    caches = [fq.KvCache(fmt, *p, g, g) for p in (small, large)]
    table = torch.tensor([[5, 0, 3], [4, 5, 2]], dtype=torch.int32, device="cuda")
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, new[0], sum(new)], dtype=torch.int32, device="cuda")
    q = torch.randn(sum(new), q_heads, dim, device="cuda")
    for dtype in (torch.bfloat16, torch.float32):
        a, b = (fq.kv_cache_attention(q.to(dtype), c, table, n, cu_q=cu, max_q=max(new)) for c in caches)
        assert torch.equal(a, b)
    rows = torch.tensor([0, lens[0], sum(lens)], dtype=torch.int32, device="cuda")
    slots = torch.tensor([5 * page + 1, 0, 4 * page + page - 1], dtype=torch.int64, device="cuda")
    k, v = torch.randn(2, 3, heads, dim, device="cuda").bfloat16()
    for _ in range(2):
        a, b = (fq.kv_cache_read(c, table, rows, total=sum(lens)) for c in caches)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        for c in caches:
            fq.kv_cache_write(c, k, v, slots)


# ---- numbers of sequences, ragged queries, long contexts


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("seqs,long_q", [(300, 1), (700, 1), (300, 3), (520, 40)])
def test_many_sequences(fq, fmt, seqs, long_q):  # noqa: F811
    """One query each, or ragged ones, some sequences without any, numbered evenly or by bisection."""
    rng = np.random.default_rng(seqs)
    lens = [int(x) for x in rng.integers(0, 40, seqs)]
    new = [1] * seqs
    if long_q > 1:
        new = [int(x) for x in rng.integers(0, 3, seqs)]
        new[seqs // 2] = long_q
    case = Case(fq, fmt, 64, 1, lens, 16, seed=seqs)
    check_attention(case, new, 4, "bf16")
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    got = fq.kv_cache_read(case.cache(), torch.from_numpy(case.table).cuda(), cu, total=sum(lens),
                           out_dtype=torch.float32)
    want = np.concatenate([case.tokens(b)[0] for b in range(seqs)])
    assert np.array_equal(got[0].double().cpu().numpy(), want.astype(np.float32).astype(np.float64))


@pytest.mark.parametrize("fmt,dim", [("nvfp4", 128), ("mxfp4", 128), ("mxfp4", 256)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens,new,page", [([40000, 3], [1, 1], 64), ([33001, 7000], [2, 3], 16),
                                           ([9001, 30], [21, 30], 48)])
def test_long_contexts(fq, fmt, dim, dtype, lens, new, page):  # noqa: F811
    """Split over many workgroups and joined."""
    check_attention(Case(fq, fmt, dim, 1, lens, page, seed=11), new, 8, dtype, rotate=True)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("max_q", [40, 64, 1000, None])
def test_max_q_is_a_bound(fq, fmt, max_q):  # noqa: F811
    case = Case(fq, fmt, 128, 2, [300, 5, 40], 16, seed=2)
    cu = torch.tensor([0, 3, 3, 43], dtype=torch.int32, device="cuda")
    q = torch.randn(43, 4, 128, device="cuda")
    table = torch.from_numpy(case.table).cuda()
    n = torch.tensor([300, 5, 40], dtype=torch.int32, device="cuda")
    out = fq.kv_cache_attention(q, case.cache(), table, n, cu_q=cu, max_q=max_q).double().cpu().numpy()
    for b, (i, j) in enumerate(((0, 3), (3, 3), (3, 43))):
        k, v = case.tokens(b)
        want, _ = kv_ref.attention(q[i:j].double().cpu().numpy(), k, v, 128 ** -0.5)
        assert np.max(np.abs(out[i:j] - want), initial=0.0) <= 2.0 ** -14 * np.abs(v).max()


@pytest.mark.parametrize("fmt,dim,rotate", [("nvfp4", 64, False), ("mxfp4", 96, False), ("nvfp4", 128, True),
                                            ("mxfp4", 128, True), ("mxfp4", 128, False), ("nvfp4", 256, True),
                                            ("mxfp4", 256, True), ("nvfp4", 256, False)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("queries", [3, 8, 11, 16, 27, 32, 50])
@pytest.mark.parametrize("listed", [0, 140000])
def test_rows_and_listed_tokens(fq, fmt, dim, rotate, dtype, queries, listed):  # noqa: F811
    """4 rows a query, few of them to many, and tables that list no more pages than are needed or a long context's:
    what the choice of kernels goes by."""
    lens, page = [333, 5, 77], 32
    case = Case(fq, fmt, dim, 1, lens, page, seed=queries)
    case.table = np.concatenate([case.table, np.full((3, listed // page), -1, dtype=np.int32)], axis=1)
    check_attention(case, [queries, min(queries, 2), queries - 1], 4, dtype, rotate=rotate)


def test_workspace_serves_any_calls(fq):  # noqa: F811
    """One workspace for calls of both kinds and all sizes, one with more queries than it says among them: each
    result is that with a fresh workspace, and the counters are zero after each."""
    case = Case(fq, "nvfp4", 128, 2, [5000, 37, 900, 0], 16, seed=6)
    cache, table = case.cache(), torch.from_numpy(case.table).cuda()
    n = torch.tensor(case.lens, dtype=torch.int32, device="cuda")
    shared = torch.zeros(256 << 20, dtype=torch.uint8, device="cuda")
    for new, q_heads, max_q in (([1, 1, 1, 1], 8, 1), ([200, 30, 100, 5], 8, 200), ([1, 1, 1, 1], 4, 1),
                                ([3, 1, 2, 4], 8, 1), ([3, 1, 2, 4], 8, 4), ([40, 1, 2, 4], 4, 2),
                                ([40, 1, 2, 4], 4, 40), ([1, 1, 1, 1], 8, 1)):
        cu = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device="cuda")
        q = torch.randn(sum(new), q_heads, 128, device="cuda").bfloat16()
        fresh = torch.zeros_like(shared)
        a, b = (fq.kv_cache_attention(q, cache, table, n, cu_q=cu, max_q=max_q, workspace=w,
                                      out=torch.zeros_like(q)) for w in (shared, fresh))
        assert torch.equal(a, b)
        assert not bool(shared[:1024 * 64].view(torch.int32)[::16].any())


@pytest.mark.parametrize("new,q_heads", SHAPES)
@pytest.mark.parametrize("window", [0, 30])
def test_workspace_bytes(fq, new, q_heads, window):  # noqa: F811
    """A workspace of the size asked for serves; one of 16 bytes less is refused."""
    case = Case(fq, "mxfp4", 128, 2, [150, 37, 400], 16, seed=3)
    cache, table = case.cache(), torch.from_numpy(case.table).cuda()
    n = torch.tensor(case.lens, dtype=torch.int32, device="cuda")
    cu = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device="cuda")
    q = torch.randn(sum(new), q_heads, 128, device="cuda")
    need = fq.kv_cache_attention_workspace_bytes(q, cache, table, max_q=max(new), window=window)
    own = torch.zeros(need, dtype=torch.uint8, device="cuda")
    kw = dict(cu_q=cu, max_q=max(new), window=window)
    assert torch.equal(fq.kv_cache_attention(q, cache, table, n, workspace=own, **kw),
                       fq.kv_cache_attention(q, cache, table, n, **kw))
    with pytest.raises(RuntimeError):
        fq.kv_cache_attention(q, cache, table, n, workspace=own[:-16], **kw)


# ---- streams and graphs


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("queries", [1, 20])
def test_streams(fq, fmt, queries):  # noqa: F811
    """Calls on other streams than the tensors' own, at once on two: the same bits, each stream with its workspace."""
    case = Case(fq, fmt, 128, 2, [3000, 500], 16, seed=1)
    cache, table = case.cache(), torch.from_numpy(case.table).cuda()
    n = torch.tensor(case.lens, dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, queries, 2 * queries], dtype=torch.int32, device="cuda")
    q = torch.randn(2 * queries, 8, 128, device="cuda").bfloat16()
    want = fq.kv_cache_attention(q, cache, table, n, cu_q=cu, max_q=queries)
    read = fq.kv_cache_read(cache, table, torch.tensor([0, 3000, 3500], dtype=torch.int32, device="cuda"), total=3500)
    rows = torch.tensor([0, 3000, 3500], dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(4):
        for s in streams:
            with torch.cuda.stream(s):
                got.append((fq.kv_cache_attention(q, cache, table, n, cu_q=cu, max_q=queries),
                            fq.kv_cache_read(cache, table, rows, total=3500)))
    torch.cuda.synchronize()
    for out, (k, v) in got:
        assert torch.equal(out, want) and torch.equal(k, read[0]) and torch.equal(v, read[1])


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("queries,q_heads", [(1, 8), (3, 8), (40, 4)])
def test_graph(fq, fmt, dtype, queries, q_heads):  # noqa: F811
    """Write, attend and read captured once, replayed with other tokens, lengths, tables and slots in place, eager
    work between: each replay gives the eager bits."""
    seqs, dim, heads, page, pages = 3, 128, 2, 16, 64
    total = seqs * queries
    rng = np.random.default_rng(queries)
    caches = [fq.kv_cache(pages, page, heads, dim, format=fmt, k_global=0.01, v_global=0.01) for _ in range(2)]
    k, v = (torch.zeros(total, heads, dim, dtype=dtype, device="cuda") for _ in range(2))
    q = torch.zeros(total, q_heads, dim, dtype=dtype, device="cuda")
    slots = torch.arange(total, dtype=torch.int64, device="cuda")
    table = torch.zeros(seqs, 12, dtype=torch.int32, device="cuda")
    lens = torch.zeros(seqs, dtype=torch.int32, device="cuda")
    cu = torch.arange(seqs + 1, dtype=torch.int32, device="cuda") * queries
    rows = torch.zeros(seqs + 1, dtype=torch.int32, device="cuda")

    def step(cache, out, read):
        fq.kv_cache_write(cache, k, v, slots, rotation="fwht128")
        fq.kv_cache_attention(q, cache, table, lens, cu_q=cu, max_q=queries, rotation="fwht128", out=out)
        fq.kv_cache_read(cache, table, rows, total=500, rotation="fwht128", out=read)

    def buffers():
        return torch.zeros_like(q), tuple(torch.zeros(500, heads, dim, dtype=torch.bfloat16, device="cuda") for _ in "kv")

    out, read = buffers()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step(caches[0], out, read)      # (makes the stream's workspace)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        step(caches[0], out, read)
    planes = [(c.k_codes, c.k_scales, c.v_codes, c.v_scales) for c in caches]
    for a, b in zip(*planes):
        b.copy_(a)
    for _ in range(5):
        for t in (k, v, q):
            t.copy_(torch.randn(t.shape, device="cuda"))
        n = rng.integers(queries, 12 * page + 1, seqs)
        order = rng.permutation(pages)[:36].reshape(3, 12)
        at = [[int(order[b, t // page]) * page + t % page for t in range(n[b] - queries, n[b])] for b in range(seqs)]
        slots.copy_(torch.tensor(at).reshape(-1))
        table.copy_(torch.from_numpy(order.astype(np.int32)))
        lens.copy_(torch.from_numpy(n.astype(np.int32)))
        rows.copy_(torch.from_numpy(np.concatenate([[0], np.cumsum(n % 150)]).astype(np.int32)))
        want = buffers()
        step(caches[1], *want)
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):     # a larger one: the workspace of the captured call's stream grows
            fq.kv_cache_attention(torch.randn(200, 64, dim, device="cuda"), caches[1], table[:1], lens[:1],
                                  cu_q=torch.tensor([0, 200], dtype=torch.int32, device="cuda"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[0])
        assert torch.equal(read[0], want[1][0]) and torch.equal(read[1], want[1][1])
        for a, b in zip(*planes):
            assert torch.equal(a, b)


def test_capture_without_a_workspace_is_refused(fq):  # noqa: F811
    case = Case(fq, "nvfp4", 64, 1, [10], 16, seed=1)
    cache, table = case.cache(), torch.from_numpy(case.table).cuda()
    n = torch.tensor([10], dtype=torch.int32, device="cuda")
    q = torch.randn(1, 2, 64, device="cuda")
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    from fp4_block_scaled_row_amd import _kv
    with torch.cuda.stream(stream):
        kept = _kv._workspaces.pop((cache._index, stream.cuda_stream), None)
        graph = torch.cuda.CUDAGraph()
        graph.capture_begin(capture_error_mode="relaxed")
        try:
            with pytest.raises(RuntimeError, match="before capturing"):
                fq.kv_cache_attention(q, cache, table, n)
        finally:
            graph.capture_end()
            if kept is not None:
                _kv._workspaces[(cache._index, stream.cuda_stream)] = kept


# ---- refusals


def test_refusals(fq):  # noqa: F811
    cache = fq.kv_cache(8, 16, 2, 128)
    k = torch.zeros(4, 2, 128, dtype=torch.bfloat16, device="cuda")
    slots = torch.zeros(4, dtype=torch.int64, device="cuda")
    table = torch.zeros(2, 4, dtype=torch.int32, device="cuda")
    n = torch.zeros(2, dtype=torch.int32, device="cuda")
    q = torch.zeros(2, 8, 128, dtype=torch.bfloat16, device="cuda")
    cu = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    planes = (cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales)
    g = torch.ones(1, device="cuda")
    bad = [
        (ValueError, lambda: fq.KvCache("if4", *planes, g, g)),
        (ValueError, lambda: fq.KvCache("nvfp4", *planes)),
        (ValueError, lambda: fq.KvCache("nvfp4", *planes, g.cpu(), g)),
        (ValueError, lambda: fq.KvCache("mxfp4", *planes)),
        (ValueError, lambda: fq.KvCache("nvfp4", planes[0].cpu(), *planes[1:], g, g)),
        (ValueError, lambda: fq.KvCache("nvfp4", planes[0].short(), *planes[1:], g, g)),
        (ValueError, lambda: fq.KvCache("nvfp4", planes[0], planes[1], planes[2].transpose(1, 2).contiguous()
                                        .transpose(1, 2), planes[3], g, g)),
        (ValueError, lambda: fq.kv_cache(8, 16, 2, 100)),
        (ValueError, lambda: fq.kv_cache_write(cache, k[:, :1], k[:, :1], slots)),
        (ValueError, lambda: fq.kv_cache_write(cache, k, k.float(), slots)),
        (TypeError, lambda: fq.kv_cache_write(cache, k.half(), k.half(), slots)),
        (ValueError, lambda: fq.kv_cache_write(cache, k, k, slots[:3])),
        (ValueError, lambda: fq.kv_cache_write(cache, k, k, slots.int())),
        (ValueError, lambda: fq.kv_cache_write(cache, k.cpu(), k, slots)),
        (ValueError, lambda: fq.kv_cache_write(cache, k.transpose(0, 2).contiguous().transpose(0, 2), k, slots)),
        (ValueError, lambda: fq.kv_cache_write(cache, k, k, slots, rotation="fwht64")),
        (RuntimeError, lambda: fq.kv_cache_write(fq.kv_cache(8, 16, 2, 96), k[:, :, :96].contiguous(),
                                                 k[:, :, :96].contiguous(), slots, rotation="fwht128")),
        (ValueError, lambda: fq.kv_cache_read(cache, table, cu[:2], total=4)),
        (ValueError, lambda: fq.kv_cache_read(cache, table, cu, total=4, starts=n[:1])),
        (TypeError, lambda: fq.kv_cache_read(cache, table, cu, total=4, out_dtype=torch.float16)),
        (ValueError, lambda: fq.kv_cache_read(cache, table, cu, total=4, out=(k, k.float()))),
        (RuntimeError, lambda: fq.kv_cache_read(cache, table, cu, total=-1, out=(None, None))),
        (ValueError, lambda: fq.kv_cache_attention(q[:1], cache, table, n)),
        (ValueError, lambda: fq.kv_cache_attention(q, cache, table.long(), n)),
        (ValueError, lambda: fq.kv_cache_attention(q, cache, table, n[:1])),
        (ValueError, lambda: fq.kv_cache_attention(q, cache, table, n, cu_q=cu[:2])),
        (ValueError, lambda: fq.kv_cache_attention(q[:, :, :64], cache, table, n)),
        (TypeError, lambda: fq.kv_cache_attention(q.half(), cache, table, n)),
        (ValueError, lambda: fq.kv_cache_attention(q, cache, table, n, out=q.float())),
        (RuntimeError, lambda: fq.kv_cache_attention(q[:, :7].contiguous(), cache, table, n)),
        (RuntimeError, lambda: fq.kv_cache_attention(q, cache, table, n, window=-1)),
        (RuntimeError, lambda: fq.kv_cache_attention(q, cache, table, n, window=4, causal=False)),
        (RuntimeError, lambda: fq.kv_cache_attention(q, cache, table, n, scale=math.inf)),
        (RuntimeError, lambda: fq.kv_cache_attention(q, cache, table, n, cu_q=cu, max_q=-1)),
        (ValueError, lambda: fq.kv_cache_attention(q, cache, table, n, workspace=torch.zeros(1 << 20, dtype=torch.uint8))),
        (RuntimeError, lambda: fq.kv_cache_attention(q, cache, table, n,
                                                     workspace=torch.zeros(64, dtype=torch.uint8, device="cuda"))),
    ]
    for i, (error, call) in enumerate(bad):
        try:
            call()
        except error as e:
            assert "fp4q" in str(e), i
        else:
            raise AssertionError("call %d was not refused" % i)
