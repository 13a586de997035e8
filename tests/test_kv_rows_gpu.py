"""Rows of a cache attention call that no sequence has: padding past the last sequence's queries, and queries past
max_q.  They are zeros and their log-sum-exps minus infinity, whatever was in the buffers."""
import numpy as np
import pytest
import torch

import kv_ref
from test_kv_gpu import DT, OUT_TOL, Case, fq  # noqa: F401  (fq: the fixture)

pytestmark = pytest.mark.gpu


def run(case, q, cu, max_q, out):
    fq = case.fq
    args = (q, case.cache(), torch.from_numpy(case.table).cuda(), torch.tensor(case.lens, dtype=torch.int32, device="cuda"))
    cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
    return fq.kv_cache_attention(*args, cu_q=cu, max_q=max_q, out=out, return_lse=True)


def check(case, q, cu, max_q, out, lse):
    """The rows that sequences have, against 64 bits; the others."""
    qd, got, got_lse = q.double().cpu().numpy(), out.double().cpu().numpy(), lse.double().cpu().numpy()
    given = np.zeros(q.shape[0], dtype=bool)
    for b in range(len(case.lens)):
        m = cu[b + 1] - cu[b]
        rows = slice(cu[b], cu[b] + min(m, max_q))
        given[rows] = True
        k, v = case.tokens(b)
        want, _ = kv_ref.attention(qd[cu[b]:cu[b + 1]], k, v, case.dim ** -0.5)
        error = np.max(np.abs(got[rows] - want[:max_q]), initial=0.0)
        assert error <= OUT_TOL["bf16" if q.dtype == torch.bfloat16 else "f32"] * np.abs(v).max(initial=1.0)
    assert not np.any(got[~given]) and not np.any(np.isnan(got[~given])), "a row that no sequence has is not zero"
    assert np.all(np.isneginf(got_lse[~given]))


@pytest.mark.parametrize("fmt,dim", [("nvfp4", 128), ("mxfp4", 96), ("mxfp4", 256), ("nvfp4", 64)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("new,q_heads,padding", [([1, 2, 1], 6, 1), ([3, 0, 2], 10, 27), ([0, 0, 0], 4, 5),
                                                 ([40, 7, 20], 6, 61), ([140, 33, 60], 10, 300)])
def test_padding(fq, fmt, dim, dtype, new, q_heads, padding):  # noqa: F811
    case = Case(fq, fmt, dim, 2, [150, 37, 400], 24, seed=dim)
    cu = np.concatenate([[0], np.cumsum(new)]).tolist()
    q = torch.randn(cu[-1] + padding, q_heads, dim, device="cuda").to(DT[dtype])
    q[cu[-1]:] = float("nan")
    print("attention", fmt, dim, dtype, new, q_heads, padding, flush=True)
    out, lse = run(case, q, cu, max(new + [1]), torch.full_like(q, float("nan")))
    check(case, q, cu, max(new), out, lse)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("new,q_heads,max_q", [([3, 1, 2], 8, 1), ([40, 1, 2], 6, 2), ([40, 7, 20], 10, 7),
                                               ([300, 5, 130], 10, 129), ([5, 5, 5], 8, 0)])
def test_queries_past_max_q(fq, fmt, dtype, new, q_heads, max_q):  # noqa: F811
    case = Case(fq, fmt, 128, 2, [350, 37, 400], 32, seed=max_q)
    cu = np.concatenate([[0], np.cumsum(new)]).tolist()
    q = torch.randn(cu[-1], q_heads, 128, device="cuda").to(DT[dtype])
    print("attention", fmt, dtype, new, q_heads, max_q, flush=True)
    out, lse = run(case, q, cu, max_q, torch.full_like(q, float("nan")))
    check(case, q, cu, max_q, out, lse)


@pytest.mark.parametrize("queries", [2, 60])
def test_padding_in_a_captured_call(fq, queries):  # noqa: F811
    """A call of a fixed number of rows replayed with other numbers of queries."""
    case = Case(fq, "nvfp4", 128, 2, [150, 90, 400], 16, seed=1)
    cache, table = case.cache(), torch.from_numpy(case.table).cuda()
    lens = torch.tensor(case.lens, dtype=torch.int32, device="cuda")
    q = torch.randn(3 * queries, 8, 128, device="cuda").bfloat16()
    cu, out = torch.zeros(4, dtype=torch.int32, device="cuda"), torch.zeros_like(q)

    def step():
        return fq.kv_cache_attention(q, cache, table, lens, cu_q=cu, max_q=queries, out=out, return_lse=True)

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        _, lse = step()
    for new in ([queries] * 3, [1, queries, 0], [0, 0, 0], [queries // 2, 1, queries]):
        at = np.concatenate([[0], np.cumsum(new)]).tolist()
        cu.copy_(torch.tensor(at, dtype=torch.int32))
        out.fill_(float("nan"))
        lse.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        check(case, q, at, queries, out, lse)
