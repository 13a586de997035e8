"""Planes whose tokens lie far apart: the offset within a page outermost in memory, as a pool that is filled a token of
every page at a time would have it."""
import numpy as np
import pytest
import torch

import kv_ref
from test_kv_gpu import fq  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt,dim", [("nvfp4", 128), ("mxfp4", 64)])
@pytest.mark.parametrize("apart", [2 ** 27 - 64, 2 ** 27 + 2 ** 24, 2 ** 28])
@pytest.mark.parametrize("new,q_heads", [([1, 1], 8), ([40, 7], 8), ([150, 33], 4)])
def test_token_strides(fq, fmt, dim, apart, new, q_heads):  # noqa: F811
    """Tokens 128 MiB and more apart in pages of 32, 31 strides passing 32 bits: the same bits as from a dense cache."""
    heads, lens, pages, page = 2, [37, 96], 6, 32
    rng = np.random.default_rng(5)
    small, large = [], []
    for width in (dim // 2, dim // kv_ref.BLOCK[fmt]) * 2:
        buf = torch.empty(apart * (page - 1) + pages * heads * width, dtype=torch.uint8, device="cuda")
        x = buf.as_strided((pages, heads, page, width), (heads * width, width, apart, 1))
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
    print("attention", fmt, dim, apart, new, q_heads, flush=True)
    for dtype in (torch.bfloat16, torch.float32):
        a, b = (fq.kv_cache_attention(q.to(dtype), c, table, n, cu_q=cu, max_q=max(new)) for c in caches)
        assert torch.equal(a, b)
    rows = torch.tensor([0, lens[0], sum(lens)], dtype=torch.int32, device="cuda")
    slots = torch.tensor([5 * page + 31, 0, 4 * page + page - 1], dtype=torch.int64, device="cuda")
    k, v = torch.randn(2, 3, heads, dim, device="cuda").bfloat16()
    for _ in range(2):
        a, b = (fq.kv_cache_read(c, table, rows, total=sum(lens)) for c in caches)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        for c in caches:
            fq.kv_cache_write(c, k, v, slots)
