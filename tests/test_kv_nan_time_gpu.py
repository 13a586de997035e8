"""A value block that is no finite number among the last tokens costs a look at the few tokens that some rows see and
others do not, not at all of a context."""
import pytest
import torch

import kv_ref
from test_kv_gpu import fq  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu


def shortest(call):
    for _ in range(3):
        call()
    times = []
    for _ in range(7):
        begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        begin.record()
        call()
        end.record()
        end.synchronize()
        times.append(begin.elapsed_time(end))
    return min(times)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("seqs,n,queries,q_heads,window", [(64, 7990, 1, 32, 0), (4, 16000, 200, 16, 0),
                                                           (64, 7990, 1, 32, 7001)])
def test_time_with_a_block_that_is_not_a_number(fq, fmt, seqs, n, queries, q_heads, window):  # noqa: F811
    """At most four times as long (11 to 65 times when the whole of a workgroup's tokens was gone through again), and NaN
    for the rows that see it alone."""
    heads, dim, page = 8, 128, 64
    pages = -(-n // page)
    cache = fq.kv_cache(seqs * pages, page, heads, dim, format=fmt)
    for codes, scales in ((cache.k_codes, cache.k_scales), (cache.v_codes, cache.v_scales)):
        codes.random_(0, 256)
        scales.fill_(0x38 if fmt == "nvfp4" else 127)
    table = torch.arange(seqs * pages, dtype=torch.int32, device="cuda").view(seqs, pages)
    lens = torch.full((seqs,), n, dtype=torch.int32, device="cuda")
    cu = torch.arange(seqs + 1, dtype=torch.int32, device="cuda") * queries
    q = torch.randn(seqs * queries, q_heads, dim, device="cuda").bfloat16()
    print("attention", fmt, seqs, n, queries, q_heads, window, flush=True)

    def call():
        return fq.kv_cache_attention(q, cache, table, lens, cu_q=cu, max_q=queries, window=window)

    before = shortest(call)
    want = call()
    last = (n - 1) // page
    cache.v_scales[table[:, last].long(), :, (n - 1) % page, 1] = 0x7F if fmt == "nvfp4" else 0xFF
    after, got = shortest(call), call()
    print("%.1f us, %.1f us" % (1e3 * before, 1e3 * after))
    assert after <= 4 * before
    block = kv_ref.BLOCK[fmt]
    nan = torch.zeros(seqs, queries, q_heads, dim, dtype=torch.bool, device="cuda")
    nan[:, -1, :, block:2 * block] = True           # (the last query alone sees the last token)
    nan = nan.view(got.shape)
    assert bool(got[nan].isnan().all()) and torch.equal(got[~nan], want[~nan])
