"""The workspace of cache attention between calls: every counter of every record is zero again, however many levels a
context's pieces are joined in, so that any other call may follow."""
import numpy as np
import pytest
import torch

from test_kv_gpu import Case, fq  # noqa: F401  (fq: the fixture)

pytestmark = pytest.mark.gpu

RECORDS, WORDS, COUNTERS = 1024, 16, 10      # of a workspace's head; a record begins with its counters, five of each kind


@pytest.mark.parametrize("fmt,dim", [("nvfp4", 128), ("mxfp4", 64)])
def test_every_counter_is_zero_after_every_call(fq, fmt, dim):  # noqa: F811
    """Contexts of one to several hundred pieces (levels of 4: up to four of them), ragged batches, many rows between."""
    shared = torch.zeros(256 << 20, dtype=torch.uint8, device="cuda")
    for lens, new, q_heads, heads, page in (([70000], [1], 8, 1, 64), ([30000, 5, 20000], [1, 1, 1], 16, 1, 48),
                                            ([5000, 37, 900, 0], [2, 1, 2, 0], 8, 2, 16), ([3000, 2000], [200, 70], 4, 2, 32),
                                            ([131000], [4], 4, 1, 128), ([9000, 9000, 9000], [7, 3, 1], 8, 4, 64),
                                            ([70000], [1], 8, 1, 64)):
        case = Case(fq, fmt, dim, heads, [16] * len(lens), page, seed=1)
        per = max(-(-n // page) for n in lens)
        table = torch.from_numpy(case.rng.integers(0, case.planes[0].shape[0], (len(lens), per)).astype(np.int32)).cuda()
        n = torch.tensor(lens, dtype=torch.int32, device="cuda")
        cu = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device="cuda")
        q = torch.randn(sum(new), q_heads, dim, device="cuda").bfloat16()
        print("attention", fmt, dim, lens, new, q_heads, heads, page, flush=True)
        cache = case.cache()
        got = fq.kv_cache_attention(q, cache, table, n, cu_q=cu, max_q=max(new), workspace=shared)
        records = shared[:RECORDS * WORDS * 4].view(torch.int32).view(RECORDS, WORDS)
        assert not bool(records[:, :COUNTERS].any())
        want = fq.kv_cache_attention(q, cache, table, n, cu_q=cu, max_q=max(new), workspace=torch.zeros_like(shared))
        assert torch.equal(got, want)
